"""Plain FP64 forms of a block's operators between the norms, and how far a
kernel that computes in FP32 and rounds its outputs once may be from them.

The bounds count roundings, as those of the step operators do (u = 2^-24 is
half an FP32 step relative to the value).  In addition:

* a product of K terms on the tensor cores: the terms are exact, every 16 of
  them are added to the sum in a step that may truncate (two half-steps), and
  aligned to the largest of a step before that: 2 (K / 16 + 16) roundings;
* an angle: the phase is exact to 2^-32 of a turn and rounded to FP32 within
  half a turn (pi 2^-25), the sine and cosine are within 2 steps of 2^-23:
  6 u in all, taken as 8;
* the sigmoid of z by the fast exponential, whose argument is rounded after a
  product with log2(e): (|z| + 8) u relative, and of the tanh form's z, itself
  of six roundings, (8 |z| + 8) u.
"""
import math

import torch

from tests.step_reference import COL_CHAIN, ROW_CHAIN, RSTD_REL, U, excess, rounded  # noqa: F401

ANGLE = 8 * U
HEAD_CHAIN = 16 + 5 + 4  # 16 columns of a lane, a butterfly of 5, the roundings of the terms


def mma_chain(k):
    return 2 * (k / 16 + 16)


# ------------------------------------------------------------------------ gated

def act(v, kind):
    """(act, act', the relative error of a kernel's sigmoid)."""
    if kind == "silu":
        z, dz = v, torch.ones_like(v)
        rel = (z.abs().clamp(max=100) + 8) * U
    else:
        k = 2 * math.sqrt(2 / math.pi)
        z, dz = k * (v + 0.044715 * v ** 3), k * (1 + 3 * 0.044715 * v ** 2)
        rel = (8 * z.abs().clamp(max=100) + 8) * U
    s = torch.sigmoid(z)
    return v * s, s + v * s * torch.sigmoid(-z) * dz, rel


def gated_fwd(x, w_gate, w_up, kind):
    """FP64 (h, g, u) with the bounds of a kernel's."""
    x, wg, wu = x.double(), w_gate.double(), w_up.double()
    g, u = x @ wg.t(), x @ wu.t()
    c = mma_chain(x.shape[1]) * U
    eg, eu = c * (x.abs() @ wg.abs().t()), c * (x.abs() @ wu.abs().t())
    a, _, rel = act(g, kind)
    ea = 1.2 * eg + (rel + U) * a.abs() + 1e-36  # |act'| < 1.13
    eh = ea * (u.abs() + eu) + a.abs() * eu + U * (a * u).abs()
    return {"h": (a * u, rounded(a * u, eh)), "g": (g, rounded(g, eg)), "u": (u, rounded(u, eu))}


def _bf16_between(v, err):
    """v rounded to BF16, and how far a value within err of v may be rounded from that."""
    mid, lo, hi = (t.float().to(torch.bfloat16).double() for t in (v, v - err, v + err))
    return mid, torch.maximum((mid - lo).abs(), (hi - mid).abs())


def gated_bwd(dh, x, g, u, w_gate, w_up, kind, two=None):
    """FP64 (dx, dw_gate, dw_up) of the BF16 gradients of g and u, with bounds; `two`: of the gradients as two BF16
    matrices, the rounded values and the rounded rest, which is at most 2^-8 of the value, itself within 2^-8."""
    two = x.shape[0] <= 64 if two is None else two
    dh, x, g, u, wg, wu = (t.double() for t in (dh, x, g, u, w_gate, w_up))
    a, da, rel = act(g, kind)
    # act' = s + v s (1 - s) z': each factor's error, and the cancellation of the two terms where v < 0;
    # 1 - s is off by the error of s, which z' v carries
    s = torch.sigmoid(g if kind == "silu" else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))
    dz = torch.ones_like(g) if kind == "silu" else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g ** 2)
    eda = 3 * (rel + 4 * U) * s * (1 + (g * dz).abs()) + 1e-36 * (1 + (g * dz).abs())
    dg, edg = dh * u * da, (dh * u).abs() * eda + 3 * U * (dh * u * da).abs()
    du, edu = dh * a, dh.abs() * ((rel + U) * a.abs() + 1e-36) + 2 * U * (dh * a).abs()
    if two:
        edg, edu = edg + 2.0 ** -16 * dg.abs(), edu + 2.0 ** -16 * du.abs()
    else:
        (dg, edg), (du, edu) = _bf16_between(dg, edg), _bf16_between(du, edu)
    T, F = (2 * n for n in g.shape) if two else g.shape  # terms of a sum, over both parts
    dx = dg @ wg + du @ wu
    ex = edg @ wg.abs() + edu @ wu.abs() + (mma_chain(2 * F) + 16) * U * (dg.abs() @ wg.abs() + du.abs() @ wu.abs())
    out = {"dx": (dx, rounded(dx, ex))}
    for name, d, e in (("dw_gate", dg, edg), ("dw_up", du, edu)):
        w = d.t() @ x
        out[name] = (w, rounded(w, e.t() @ x.abs() + (mma_chain(T) + 16) * U * (d.abs().t() @ x.abs())))
    return out


# ----------------------------------------------------------------------- rotary

def phases(positions, turns, axes):
    """The angles [T, pairs], from whole numbers modulo 2^64."""
    p = positions.reshape(-1, positions.shape[-1]).long().cpu()
    axes = torch.zeros(turns.numel(), dtype=torch.long) if axes is None else axes.long().cpu()
    return (p[axes].t() * turns.cpu()).double() * (2 * math.pi / 2.0 ** 64)


def turn(v, angle, style, sign=1.0):
    """v [T, heads, D] rotated, and the sum of the magnitudes that went into each value."""
    n = angle.shape[1]
    c, s = angle.cos()[:, None], sign * angle.sin()[:, None]
    at = (slice(0, n), slice(n, 2 * n)) if style == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    a, b = v[..., at[0]], v[..., at[1]]
    out, mag = v.clone(), v.abs()
    out[..., at[0]], out[..., at[1]] = a * c - b * s, b * c + a * s
    mag[..., at[0]] = mag[..., at[1]] = a.abs() + b.abs()
    mag[..., 2 * n:] = v[..., 2 * n:].abs()
    return out, mag


def rotary_fwd(v, angle, w, eps, style):
    """FP64 (y, its bound, rstd) of a [T, heads, D] tensor on the CPU."""
    v, rstd = v.double().cpu(), None
    if w is not None:
        rstd = 1.0 / torch.sqrt((v * v).mean(-1) + eps)
        v = v * rstd[..., None] * w.double().cpu()
    y, mag = turn(v, angle, style)
    err = mag * (ANGLE + 3 * U + (0 if w is None else RSTD_REL + 3 * U))
    return y, rounded(y, err), rstd


def rotary_bwd(dy, angle, v, rstd, w, style):
    """FP64 (dv, its bound, dw, its bound) on the CPU."""
    d, mag = turn(dy.double().cpu(), angle, style, -1.0)
    ed = mag * (ANGLE + 3 * U)
    if w is None:
        return d, rounded(d, ed), None, None
    w, rs = w.double().cpu(), rstd.double().cpu().reshape(d.shape[:2])[..., None]
    vh = v.double().cpu() * rs
    a, D = d * w, d.shape[-1]
    mean = (a * vh).mean(-1, keepdim=True)
    em = (HEAD_CHAIN * U * (a * vh).abs().sum(-1, keepdim=True) + (w * vh * ed).abs().sum(-1, keepdim=True)) / D
    em = em + 2 * U * mean.abs()
    dv = rs * (a - vh * mean)
    edv = rs * (w.abs() * ed + vh.abs() * em + 5 * U * (a.abs() + (vh * mean).abs()))
    terms = d * vh
    edw = ((vh.abs() * ed) + COL_CHAIN * U * terms.abs()).sum((0, 1))
    return dv, rounded(dv, edv), terms.sum((0, 1)), edw


# ---------------------------------------------------------------------- dropout

_LOW = 2 ** 32 - 1


def philox(counter, key):
    """Philox4x32-10 of four 32-bit words (whole numbers), as published."""
    x, k = list(counter), list(key)
    for _ in range(10):
        p0, p1 = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57
        x = [(p1 >> 32) ^ x[1] ^ k[0], p1 & _LOW, (p0 >> 32) ^ x[3] ^ k[1], p0 & _LOW]
        k = [(k[0] + 0x9E3779B9) & _LOW, (k[1] + 0xBB67AE85) & _LOW]
    return x


def kept(rows, H, p, seed, offset):
    """The factor m of each element of [rows, H] in FP64 (whole numbers in 64 bits, which wrap)."""
    b = torch.arange(rows * H // 8, dtype=torch.int64)
    seed, offset = seed % 2 ** 64, offset % 2 ** 64
    x = [b & _LOW, b >> 32, torch.full_like(b, offset & _LOW), torch.full_like(b, offset >> 32)]
    k0, k1 = seed & _LOW, seed >> 32
    for _ in range(10):
        p0, p1 = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57
        x = [((p1 >> 32) & _LOW) ^ x[1] ^ k0, p1 & _LOW, ((p0 >> 32) & _LOW) ^ x[3] ^ k1, p0 & _LOW]
        k0, k1 = (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW
    bits = torch.stack([h for w in x for h in (w & 0xFFFF, w >> 16)], 1).reshape(rows, H)
    cut = round(p * 65536)
    return (bits >= cut).double() * (65536 / (65536 - cut) if cut < 65536 else 0.0)


def dropout_sum(x, m, residual):
    """FP64 (residual + m x, its error before the rounding to BF16)."""
    x = x.double().cpu().reshape(m.shape)
    v = torch.where(m > 0, x, torch.zeros_like(x)) * m
    err = 2 * U * v.abs()
    if residual is not None:
        v = v + residual.double().cpu().reshape(m.shape)
        err = err + U * v.abs()
    return v, err


def dropout_norm_bwd(dy, h, rstd, w, dh, m):
    """FP64 gradients (dresidual, dx, dw) and the bounds of a kernel's, on the CPU."""
    dy, h = dy.double().cpu().reshape(m.shape), h.double().cpu().reshape(m.shape)
    e = torch.zeros_like(h) if dh is None else dh.double().cpu().reshape(m.shape)
    rs, w, H = rstd.double().cpu().reshape(-1, 1), w.double().cpu(), h.shape[-1]
    a, hh = dy * w, h * rs
    mean = (a * hh).mean(-1, keepdim=True)
    em = ROW_CHAIN * U * (a * hh).abs().sum(-1, keepdim=True) / H + 2 * U * mean.abs()
    t = rs * (a - hh * mean) + e
    et = rs * (hh.abs() * em + 5 * U * (a.abs() + (hh * mean).abs())) + U * (t.abs() + e.abs())
    terms = dy * hh
    return {"dresidual": (t, rounded(t, et)), "dx": (m * t, rounded(m * t, m * et + 2 * U * (m * t).abs())),
            "dw": (terms.sum(0), COL_CHAIN * U * terms.abs().sum(0))}
