"""Plain FP64 forms of the training-step operators, and how far a kernel that
computes in FP32 and rounds its outputs once may be from them.

The bounds count roundings.  u = 2^-24 is half an FP32 step relative to the
value, a BF16 rounding is at most 2^-8 of the value, and a sum of n terms in
FP32 whose longest chain of additions is c is off by at most c * u * sum|terms|.
A row's sums have chains of at most 64 additions (32 columns of a thread or 16
pairs, two butterflies of 5, 16 warps); a column's sums over rows are
compensated or in blocks of 16 rows, 24 roundings at most with those of the
terms.
"""
import torch

U = 2.0 ** -24
HALF_BF16 = 2.0 ** -8
RSTD_REL = 1e-6
ROW_CHAIN = 64 + 4   # and the roundings of the terms
COL_CHAIN = 24
TINY = 2.0 ** -133   # the smallest BF16 step


def _g(gate, like):
    if gate is None:
        return torch.ones((), dtype=torch.float64)
    g = gate.double()
    return g[..., None] if g.dim() == like.dim() - 1 else g


def sandwich_fwd(z, x, w_post, w_pre, eps, gate, scale):
    """FP64 (h before its rounding, the term added to x, rstd_post)."""
    z = z.double()
    r1 = 1.0 / torch.sqrt((z * z).mean(-1) + eps)
    add = scale * _g(gate, z) * z * r1[..., None] * w_post.double()
    return x.double() + add, add, r1


def norm_fwd(h, w, eps):
    h = h.double()
    r = 1.0 / torch.sqrt((h * h).mean(-1) + eps)
    return h * r[..., None] * w.double(), r


def rounded(v, err):
    """The bound of a value within err of v after one rounding to BF16."""
    return err + HALF_BF16 * (v.abs() + err) + TINY


def sandwich_bwd(dy, h, z, r1, r2, w_post, w_pre, dh, gate, scale):
    """FP64 gradients (dx, dz, dw_post, dw_pre, dgate) and the bounds of a kernel's."""
    dy, h, z = dy.double(), h.double(), z.double()
    e = torch.zeros_like(h) if dh is None else dh.double()
    rp, rn = r1.double().reshape(h.shape[:-1])[..., None], r2.double().reshape(h.shape[:-1])[..., None]
    w1, w2, g = w_post.double(), w_pre.double(), _g(gate, z)
    H = h.shape[-1]
    rows = tuple(range(h.dim() - 1))
    row_gate = gate is not None and gate.dim() == z.dim() - 1
    ge = g if gate is not None and not row_gate else torch.ones((), dtype=torch.float64)
    gr = g if row_gate else torch.ones((), dtype=torch.float64)

    def mean(v):
        return v.mean(-1, keepdim=True)

    a = dy * w2
    k2 = rn ** 3 * mean(a * h)
    t = e + rn * a - k2 * h
    dn = scale * g * t
    b = ge * w1
    dot = (t * b * z).sum(-1, keepdim=True)
    k1 = rp ** 2 * dot / H
    sr = scale * gr * rp
    dz = sr * (b * t - k1 * z)
    dw_pre_terms, dw_post_terms = dy * h * rn, dn * z * rp

    # errors
    d_s1 = ROW_CHAIN * U * (a * h).abs().sum(-1, keepdim=True)
    d_s2 = ROW_CHAIN * U * ((e.abs() + (rn * a).abs()) * (b * z).abs()).sum(-1, keepdim=True)
    s3 = (b * h * z).sum(-1, keepdim=True)
    d_s3 = ROW_CHAIN * U * (b * h * z).abs().sum(-1, keepdim=True)
    d_k2 = rn ** 3 * d_s1 / H + 6 * U * k2.abs()
    d_t = h.abs() * d_k2 + 4 * U * (e.abs() + (rn * a).abs() + (k2 * h).abs())
    d_dot = d_s2 + k2.abs() * d_s3 + d_k2 * (s3.abs() + d_s3) + 2 * U * (dot.abs() + (k2 * s3).abs())
    d_k1 = rp ** 2 * d_dot / H + 6 * U * k1.abs()
    d_dz = sr.abs() * (b.abs() * d_t + z.abs() * d_k1 + 8 * U * ((t * b).abs() + (k1 * z).abs()))
    out = {"dx": (t, rounded(t, d_t)), "dz": (dz, rounded(dz, d_dz)),
           "dw_pre": (dw_pre_terms.sum(rows), COL_CHAIN * U * dw_pre_terms.abs().sum(rows)),
           "dw_post": (dw_post_terms.sum(rows),
                       ((sr * ge * z).abs() * d_t).sum(rows) + COL_CHAIN * U * dw_post_terms.abs().sum(rows))}
    if row_gate:
        v = (scale * rp * dot)[..., 0]
        out["dgate"] = (v, (scale * rp).abs()[..., 0] * d_dot[..., 0] + 6 * U * v.abs())
    elif gate is not None:
        n = z * rp * w1
        v = scale * t * n
        out["dgate"] = (v, rounded(v, (scale * n).abs() * d_t + 6 * U * v.abs()))
    return out


def excess(got, want, allow):
    """The largest error as a share of its bound (0 where both are 0); infinite where got is not finite."""
    got, want = got.detach().double().cpu(), want.cpu()
    err = (got - want).abs()
    share = torch.where(err == 0, torch.zeros_like(err), err / allow.cpu().clamp_min(1e-300))
    return float("inf") if not bool(torch.isfinite(got).all()) else float(share.max()) if share.numel() else 0.0


def grad_norm(grads):
    return sum(float(g.double().square().sum()) for g in grads) ** 0.5


def embedding_bwd(dy, ids, vocab, scale, padding_idx, base=None):
    """FP64 table gradient and the sum of the magnitudes that went into each value, and counts per row."""
    H = dy.shape[-1]
    ids, rows = ids.reshape(-1).long().cpu(), dy.reshape(-1, H).double().cpu()
    live = (ids >= 0) & (ids < vocab)
    if padding_idx is not None:
        live &= ids != padding_idx
    total = torch.zeros(vocab, H, dtype=torch.float64)
    mags, counts = torch.zeros_like(total), torch.zeros(vocab, dtype=torch.float64)
    total.index_add_(0, ids[live], rows[live])
    mags.index_add_(0, ids[live], rows[live].abs())
    counts.index_add_(0, ids[live], torch.ones(int(live.sum()), dtype=torch.float64))
    total, mags = total * scale, mags * abs(scale)
    if base is not None:
        total = total + base.double().cpu()
    return total, mags, counts
