"""Workloads of a training block's operators between the norms, with their plain forms.

Operators: the gated feed-forward block (both projections, the activation and
the product; forward and backward), the per-head norm of queries and keys with
rotary positions of several axes (forward and backward), and dropout from a
counter-based generator, alone and with the residual addition and the norm
after it (forward and backward).  ``run`` takes one pass through an operator:
through elementary torch operations in 32 bits (``own`` false) or through this
package's entry points (``own`` true).
"""
import functools
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ---------------------------------------------------------------------- cases

def _gated(op, T, H, F, act, save=True, pad=0, name=None):
    c = {"op": op, "T": T, "H": H, "F": F, "act": act, "save": save, "pad": pad}
    return dict(c, name=name) if name else c


def _rotary(op, T, nq, nk, D, sections, style, norm=True, gap=0, far=4096, name=None):
    c = {"op": op, "T": T, "nq": nq, "nk": nk, "D": D, "sections": sections, "style": style, "norm": norm, "gap": gap,
         "far": far}
    return dict(c, name=name) if name else c


def _dropout(op, T, H, p, w32=False, pad=0, name=None):
    c = {"op": op, "T": T, "H": H, "p": p, "w32": w32, "pad": pad}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token (generation inside a training loop): reading the weights once
        _gated("gated_fwd", 1, 2048, 6144, "silu", save=False, name="gated_fwd_t1_h2048"),
        # a decoding batch: still the weights' bytes
        _gated("gated_fwd", 64, 4096, 8192, "gelu", save=False, name="gated_fwd_t64_h4096"),
        # a training batch of a large model, what the backward needs kept
        _gated("gated_fwd", 8192, 4096, 8192, "silu", name="gated_fwd_t8192_h4096"),
        # a short packed batch of odd length and odd widths, rows that are slices of a wider buffer
        _gated("gated_bwd", 333, 1000, 2728, "gelu", pad=24, name="gated_bwd_t333_h1000"),
        # the backward of an ordinary training batch
        _gated("gated_bwd", 8192, 2048, 6144, "silu", name="gated_bwd_t8192_h2048"),
        # one token's heads: a call's latency
        _rotary("rotary_fwd", 1, 24, 4, 256, "64", "half", far=100000, name="rotary_fwd_t1_24x256"),
        # a long-context training batch; queries are slices of heads of 512, a quarter of a head is rotated
        _rotary("rotary_fwd", 32768, 24, 4, 256, "32", "half", gap=256, far=1000000,
                name="rotary_fwd_t32768_24x256"),
        # its backward
        _rotary("rotary_bwd", 32768, 24, 4, 256, "32", "half", gap=256, far=1000000,
                name="rotary_bwd_t32768_24x256"),
        # video tokens of an odd number with time, height and width, adjacent pairs, every head its own key
        _rotary("rotary_bwd", 10007, 16, 16, 128, "16,24,24", "adjacent", far=300, name="rotary_bwd_t10007_video"),
        # a short sequence's residual addition and norm
        _dropout("dropout_norm_fwd", 256, 1536, 0.1, name="dropout_norm_fwd_t256_h1536"),
        # the backward of an ordinary large batch
        _dropout("dropout_norm_bwd", 32768, 4096, 0.1, w32=True, name="dropout_norm_bwd_t32768_h4096"),
        # activations of a packed batch of odd length, slices of a wider buffer
        _dropout("dropout_fwd", 16381, 6144, 0.25, pad=64, name="dropout_fwd_t16381_h6144"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated_fwd", "gated_bwd", "rotary_fwd", "rotary_bwd", "dropout_fwd", "dropout_norm_fwd",
                     "dropout_norm_bwd"])
    if op.startswith("gated"):
        H, F = 8 * _log(rng, 16, 512), 8 * _log(rng, 16, 1024)
        most = (2 ** 38 if op == "gated_fwd" else 10 ** 11) // (H * F)
        T = _log(rng, 1, max(1, min(16384, most)))
        return _gated(op, T, H, F, rng.choice(["silu", "gelu"]), op == "gated_bwd" or rng.random() < 0.5,
                      rng.choice([0, 0, 8, 64]))
    if op.startswith("rotary"):
        D = 16 * rng.randint(2, 16)
        half = 8 * rng.randint(1, D // 16)
        cuts = sorted(rng.randint(1, half - 1) for _ in range(rng.choice([0, 0, 1, 2, 3])))
        ends = sorted(set(cuts)) + [half]
        sections = ",".join(str(b - a) for a, b in zip([0] + ends, ends))
        nk = _log(rng, 1, 16)
        nq = nk * rng.choice([1, 2, 4, 6])
        T = _log(rng, 1, min(65536, int(2.3e8) // ((nq + nk) * D)))
        return _rotary(op, T, nq, nk, D, sections, rng.choice(["half", "adjacent"]), rng.random() < 0.7,
                       rng.choice([0, 0, D, 16]), _log(rng, 100, 2000000))
    H = 8 * _log(rng, 8, 1024)
    T = _log(rng, 1, min(65536, 2 ** 27 // H))
    return _dropout(op, T, H, rng.choice([0.05, 0.1, 0.2, 0.5, rng.uniform(0.01, 0.9)]), rng.random() < 0.5,
                    rng.choice([0, 0, 8, 128]))


# --------------------------------------------------------------------- inputs

def _rows(T, H, pad, g, std=1.0, mean=0.0):
    """BF16 [T, H] of N(mean, std): a slice of a buffer of H + pad columns."""
    buf = torch.empty(T, H + pad, dtype=BF16, device=DEV)
    for a in range(0, T, 8192):
        b = min(T, a + 8192)
        buf[a:b] = (torch.randn(b - a, H + pad, generator=g, device=DEV) * std + mean).to(BF16)
    return buf[:, :H]


def _sections(c):
    return [int(n) for n in c["sections"].split(",")]


def _freqs(c):
    """Each section's ladder of frequencies (radians a position) in turn."""
    return [1.0e4 ** (-i / n) for n in _sections(c) for i in range(n)]


def _prepare_gated(c, s, g):
    T, H, F = c["T"], c["H"], c["F"]
    s["x"] = _rows(T, H, c["pad"], g)
    s["w_gate"] = _rows(F, H, 0, g, H ** -0.5)
    s["w_up"] = _rows(F, H, 0, g, H ** -0.5)
    if c["op"] == "gated_bwd":
        s["g"], s["u"] = _rows(T, F, 0, g), _rows(T, F, 0, g)
        s["dh"] = _rows(T, F, c["pad"], g)


def _prepare_rotary(c, s, g):
    T, nq, nk, D, half = c["T"], c["nq"], c["nk"], c["D"], sum(_sections(c))
    wide = D + c["gap"]
    s["q"] = _rows(T, nq * wide, 0, g, 1.0, 0.5).view(T, nq, wide)[:, :, :D]
    s["k"] = _rows(T, nk * D, 0, g, 1.0, 0.5).view(T, nk, D)
    s["w_q"] = s["w_k"] = None
    if c["norm"]:
        s["w_q"] = 1 + 0.1 * torch.randn(D, generator=g, device=DEV)
        s["w_k"] = (1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(BF16)
    # an axis' positions: where a packed batch's sequences stand
    s["positions"] = torch.randint(0, c["far"], (len(_sections(c)), T), generator=g, device=DEV)
    s["freqs"] = torch.tensor(_freqs(c), dtype=F64, device=DEV)
    s["axes"] = torch.tensor([a for a, n in enumerate(_sections(c)) for _ in range(n)], dtype=torch.int32, device=DEV)
    # the same frequencies in 2^-64 of a turn
    turns = [round(f / (2 * math.pi) * 2 ** 64) for f in _freqs(c)]
    s["turns"] = torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64, device=DEV)
    assert half == len(turns)
    if c["op"] == "rotary_bwd":
        s["dq"] = _rows(T, nq * D, 0, g).view(T, nq, D)
        s["dk"] = _rows(T, nk * D, 0, g).view(T, nk, D)
        s["rstd_q"] = s["rstd_k"] = None
        if c["norm"]:
            s["rstd_q"], s["rstd_k"] = (torch.rsqrt(s[n].float().square().mean(2) + EPS).reshape(-1) for n in "qk")


def _prepare_dropout(c, s, g):
    T, H = c["T"], c["H"]
    s["seed"] = int(torch.randint(0, 2 ** 62, (1,), generator=g, device=DEV))
    s["offset"] = int(torch.randint(0, 2 ** 40, (1,), generator=g, device=DEV))
    if c["op"] == "dropout_fwd":
        s["x"] = _rows(T, H, c["pad"], g)
        return
    s["w"] = (1 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(F32 if c["w32"] else BF16)
    if c["op"] == "dropout_norm_fwd":
        s["x"] = _rows(T, H, c["pad"], g, 0.7)
        s["residual"] = _rows(T, H, 0, g, 1.5)
        return
    s["h"] = _rows(T, H, 0, g, 1.7)
    s["rstd"] = torch.rsqrt(torch.linalg.vector_norm(s["h"], dim=1, dtype=F32).square() / H + EPS)
    s["dy"] = _rows(T, H, 0, g)
    s["dh"] = _rows(T, H, c["pad"], g)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = {"case": c}
    kind = c["op"].split("_")[0]
    {"gated": _prepare_gated, "rotary": _prepare_rotary, "dropout": _prepare_dropout}[kind](c, s, g)
    return s


# ---------------------------------------------------------------- plain forms

def _gated_fwd(s):
    c, x = s["case"], s["x"].float()
    g, u = x @ s["w_gate"].float().t(), x @ s["w_up"].float().t()
    if c["act"] == "silu":
        a = g * torch.sigmoid(g)
    else:
        a = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))
    h = (a * u).to(BF16)
    return (h, g.to(BF16), u.to(BF16)) if c["save"] else h


def _gated_bwd(s):
    c, x = s["case"], s["x"].float()
    g, u, dh = s["g"].float(), s["u"].float(), s["dh"].float()
    if c["act"] == "silu":
        sig = torch.sigmoid(g)
        a, da = g * sig, sig * (1 + g * (1 - sig))
    else:
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (g + 0.044715 * g * g * g))
        a, da = 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)
    dg, du = dh * u * da, dh * a
    dx = dg @ s["w_gate"].float() + du @ s["w_up"].float()
    return dx.to(BF16), (dg.t() @ x).to(BF16), (du.t() @ x).to(BF16)


def _turned(v, cos, sin, style, half):
    """v [T, heads, D] with its first 2 * half columns rotated; cos, sin: [T, half]."""
    c, n = cos[:, None, :], sin[:, None, :]
    head, tail = v[:, :, :2 * half], v[:, :, 2 * half:]
    if style == "half":
        a, b = head[:, :, :half], head[:, :, half:]
        return torch.cat([a * c - b * n, b * c + a * n, tail], 2)
    a, b = head[:, :, 0::2], head[:, :, 1::2]
    return torch.cat([torch.stack([a * c - b * n, b * c + a * n], 3).flatten(2), tail], 2)


def _angles(s):
    angle = s["positions"].to(F64)[s["axes"].long()].t() * s["freqs"]
    return torch.cos(angle).float(), torch.sin(angle).float()


def _rotary_fwd(s):
    c = s["case"]
    cos, sin = _angles(s)

    def one(v, w):
        v, rstd = v.float(), None
        if w is not None:
            rstd = 1.0 / torch.sqrt(v.square().mean(2) + EPS)
            v = v * rstd[:, :, None] * w.float()
        return _turned(v, cos, sin, c["style"], cos.shape[1]).to(BF16), None if rstd is None else rstd.reshape(-1)

    (q, rq), (k, rk) = one(s["q"], s["w_q"]), one(s["k"], s["w_k"])
    return q, k, rq, rk


def _rotary_bwd(s):
    c = s["case"]
    cos, sin = _angles(s)

    def one(dy, v, rstd, w):
        d = _turned(dy.float(), cos, -sin, c["style"], cos.shape[1])
        if w is None:
            return d.to(BF16), None
        hat = v.float() * rstd.view(v.shape[:2])[:, :, None]
        a = d * w.float()
        dv = rstd.view(v.shape[:2])[:, :, None] * (a - hat * (a * hat).mean(2, keepdim=True))
        return dv.to(BF16), (d * hat).sum((0, 1), dtype=F64).float()

    (dq, dwq), (dk, dwk) = one(s["dq"], s["q"], s["rstd_q"], s["w_q"]), one(s["dk"], s["k"], s["rstd_k"], s["w_k"])
    return dq, dk, dwq, dwk


def _kept(s, T, H):
    """The factor of each of [T, H] values: 0, or one over the share that is kept.

    Values 8 b to 8 b + 7, counted row by row, take the 16-bit pieces of the
    Philox4x32-10 block of counter (b, offset) and key (seed), lowest first.
    """
    low = 0xFFFFFFFF
    b = torch.arange(T * H // 8, device=DEV)
    start = (b & low, b >> 32, torch.full_like(b, s["offset"] & low), torch.full_like(b, s["offset"] >> 32))

    def turn(v, r):
        k0, k1 = (s["seed"] + r * 0x9E3779B9) & low, ((s["seed"] >> 32) + r * 0xBB67AE85) & low
        p0, p1 = v[0] * 0xD2511F53, v[2] * 0xCD9E8D57  # whole products of 32 bits, their upper halves below
        return ((p1 >> 32) & low) ^ v[1] ^ k0, p1 & low, ((p0 >> 32) & low) ^ v[3] ^ k1, p0 & low

    v = functools.reduce(turn, range(10), start)
    pieces = torch.stack([x for w in v for x in (w & 0xFFFF, w >> 16)], 1).view(T, H)
    cut = round(s["case"]["p"] * 65536)
    return (pieces >= cut).float() * (65536.0 / (65536 - cut))


def _dropout_fwd(s):
    T, H = s["x"].shape
    return (s["x"].float() * _kept(s, T, H)).to(BF16)


def _dropout_norm_fwd(s):
    T, H = s["x"].shape
    h_new = (s["residual"].float() + s["x"].float() * _kept(s, T, H)).to(BF16)
    h = h_new.float()
    rstd = 1.0 / torch.sqrt(h.square().mean(1) + EPS)
    return (h * rstd[:, None] * s["w"].float()).to(BF16), h_new, rstd


def _dropout_norm_bwd(s):
    T, H = s["h"].shape
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    hat = s["h"].float() * rstd
    a = dy * s["w"].float()
    t = s["dh"].float() + rstd * (a - hat * (a * hat).mean(1, keepdim=True))
    return t.to(BF16), (t * _kept(s, T, H)).to(BF16), (dy * hat).sum(0, dtype=F64).float()


def _plain(s):
    return {"gated_fwd": _gated_fwd, "gated_bwd": _gated_bwd, "rotary_fwd": _rotary_fwd, "rotary_bwd": _rotary_bwd,
            "dropout_fwd": _dropout_fwd, "dropout_norm_fwd": _dropout_norm_fwd,
            "dropout_norm_bwd": _dropout_norm_bwd}[s["case"]["op"]](s)


def run(state):
    s = state
    c = s["case"]
    if not own:
        return _plain(s)
    import bwd_dw_column_gb300 as cake
    if c["op"] == "gated_fwd":
        got = cake.cake_gated_fwd(s["x"], s["w_gate"], s["w_up"], c["act"], save=c["save"])
        return got if c["save"] else got[0]
    if c["op"] == "gated_bwd":
        return cake.cake_gated_bwd(s["dh"], s["x"], s["g"], s["u"], s["w_gate"], s["w_up"], c["act"])
    if c["op"] == "rotary_fwd":
        return cake.cake_rotary_fwd(s["q"], s["k"], s["positions"], s["turns"], s["axes"], s["w_q"], s["w_k"], EPS,
                                    style=c["style"])
    if c["op"] == "rotary_bwd":
        return cake.cake_rotary_bwd(s["dq"], s["dk"], s["positions"], s["turns"], s["axes"], s["q"], s["k"],
                                    s["rstd_q"], s["rstd_k"], s["w_q"], s["w_k"], style=c["style"])
    if c["op"] == "dropout_fwd":
        return cake.cake_dropout_fwd(s["x"], c["p"], s["seed"], s["offset"])
    if c["op"] == "dropout_norm_fwd":
        return cake.cake_dropout_norm_fwd(s["x"], s["residual"], s["w"], c["p"], s["seed"], s["offset"], EPS)
    return cake.cake_dropout_norm_bwd(s["dy"], s["h"], s["rstd"], s["w"], c["p"], s["seed"], s["offset"], dh=s["dh"])


# ----------------------------------------------------------------------- work

def work(case):
    c = case
    T = c["T"]
    if c["op"].startswith("gated"):
        H, F = c["H"], c["F"]
        if c["op"] == "gated_fwd":
            return {"bytes": 2 * (T * H + 2 * F * H + T * F * (3 if c["save"] else 1)), "flops": 4 * T * H * F + 8 * T * F}
        return {"bytes": 2 * (2 * T * H + 4 * F * H + 3 * T * F), "flops": 8 * T * H * F + 16 * T * F}
    if c["op"].startswith("rotary"):
        n, heads = T * (c["nq"] + c["nk"]) * c["D"], T * (c["nq"] + c["nk"])
        known = 8 * T * len(_sections(c)) + (4 * heads if c["norm"] else 0)
        moved = 2 if c["op"] == "rotary_fwd" or not c["norm"] else 3  # without a norm the gradient needs no inputs
        return {"bytes": 2 * n * moved + known, "flops": 10 * n}
    H = c["H"]
    n, w = T * H, H * (4 if c["w32"] else 2)
    if c["op"] == "dropout_fwd":
        return {"bytes": 4 * n, "flops": 2 * n}
    if c["op"] == "dropout_norm_fwd":
        return {"bytes": 8 * n + 4 * T + w, "flops": 8 * n}
    return {"bytes": 10 * n + 4 * T + w + 4 * H, "flops": 16 * n}


# ---------------------------------------------------------------------- exact

def _activated(v, act):
    if act == "silu":
        return v * torch.special.expit(v)
    return v * torch.special.expit(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v.pow(3)))


def _exact_gated(c, s):
    x, wg, wu = (s[k].to(F64) for k in ("x", "w_gate", "w_up"))
    if c["op"] == "gated_fwd":
        g, u = torch.nn.functional.linear(x, wg), torch.nn.functional.linear(x, wu)
        h = _activated(g, c["act"]).mul_(u)
        return (h, g, u) if c["save"] else h
    # differentiated by torch in 64 bits through the activation and the product
    g, u = (s[k].to(F64).requires_grad_() for k in "gu")
    dg, du = torch.autograd.grad(_activated(g, c["act"]) * u, (g, u), s["dh"].to(F64))
    return torch.mm(dg, wg).addmm_(du, wu), torch.mm(x.t(), dg).t(), torch.mm(x.t(), du).t()


def _exact_rotary(c, s):
    half = sum(_sections(c))
    # a rotation is a product of complex numbers of length one
    where = s["positions"].to(F64).index_select(0, s["axes"].long())
    turn = torch.polar(torch.ones_like(where), where * s["freqs"][:, None]).t()[:, None, :]

    def rotated(v):
        head = v[..., :2 * half].unflatten(2, (2, half) if c["style"] == "half" else (half, 2))
        at = 2 if c["style"] == "half" else 3
        z = torch.complex(head.select(at, 0), head.select(at, 1)) * turn
        return torch.cat([torch.stack([z.real, z.imag], at).flatten(2), v[..., 2 * half:]], 2)

    def normed(v, w):
        if w is None:
            return rotated(v), None
        r = (torch.linalg.vector_norm(v, dim=2).square() / c["D"] + EPS).rsqrt()
        return rotated(v * r[:, :, None] * w), r.reshape(-1)

    def parts(n):
        return s[n].to(F64), None if s["w_" + n] is None else s["w_" + n].to(F64)

    if c["op"] == "rotary_fwd":
        (q, rq), (k, rk) = (normed(*parts(n)) for n in "qk")
        return q, k, rq, rk
    got = {}
    for n in "qk":
        v, w = parts(n)
        leaves = [t.requires_grad_() for t in (v, w) if t is not None]
        d = torch.autograd.grad(normed(v, w)[0], leaves, s["d" + n].to(F64))
        got[n] = (d[0], d[1] if w is not None else None)
    return got["q"][0], got["k"][0], got["q"][1], got["k"][1]


def _exact_mask(c, s, T, H):
    """The kept values' factor again, products of 32 bits by 16-bit limbs, a row block at a time."""
    def wide(a, m):
        lo, hi = a & 0xFFFF, torch.bitwise_right_shift(a, 16)
        mid = lo * (m >> 16) + torch.bitwise_right_shift(lo * (m & 0xFFFF), 16)
        mid2 = hi * (m & 0xFFFF) + (mid & 0xFFFF)
        high = hi * (m >> 16) + torch.bitwise_right_shift(mid, 16) + torch.bitwise_right_shift(mid2, 16)
        return high & 0xFFFFFFFF, ((mid2 & 0xFFFF) << 16) | ((lo * (m & 0xFFFF)) & 0xFFFF)

    cut, out = int(math.floor(c["p"] * 65536 + 0.5)), torch.empty(T, H, dtype=F64, device=DEV)
    step = max(1, 2 ** 24 // H)
    for a in range(0, T, step):
        n = min(step, T - a)
        b = torch.arange(a * H // 8, (a + n) * H // 8, device=DEV)
        x, y = b % 2 ** 32, b // 2 ** 32
        z, w = (torch.full_like(b, v) for v in (s["offset"] % 2 ** 32, s["offset"] // 2 ** 32))
        k0, k1 = s["seed"] % 2 ** 32, s["seed"] // 2 ** 32
        for _ in range(10):
            (h0, l0), (h1, l1) = wide(x, 0xD2511F53), wide(z, 0xCD9E8D57)
            x, y, z, w = h1 ^ y ^ k0, l1, h0 ^ w ^ k1, l0
            k0, k1 = (k0 + 0x9E3779B9) % 2 ** 32, (k1 + 0xBB67AE85) % 2 ** 32
        u = torch.stack([x % 65536, x // 65536, y % 65536, y // 65536, z % 65536, z // 65536, w % 65536, w // 65536], 1)
        out[a:a + n] = torch.where(u.reshape(n, H) < cut, 0.0, 1.0 / (1.0 - cut / 65536.0)).to(F64)
    return out


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"].startswith("gated"):
        return _exact_gated(c, s)
    if c["op"].startswith("rotary"):
        return _exact_rotary(c, s)
    m = _exact_mask(c, s, c["T"], c["H"])
    if c["op"] == "dropout_fwd":
        return s["x"].to(F64) * m
    if c["op"] == "dropout_norm_fwd":
        # the norm is of the stored BF16 sum
        h = torch.addcmul(s["residual"].to(F64), s["x"].to(F64), m)
        v = h.to(BF16).to(F64)
        r = (torch.linalg.vector_norm(v, dim=1).square() / c["H"] + EPS).rsqrt()
        return v * r[:, None] * s["w"].to(F64), h, r
    h, w = s["h"].to(F64).requires_grad_(), s["w"].to(F64).requires_grad_()
    y = h * (h.square().mean(1, keepdim=True) + EPS).rsqrt() * w
    t, dw = torch.autograd.grad(y, (h, w), s["dy"].to(F64))
    t = t + s["dh"].to(F64)
    return t, t * m, dw
