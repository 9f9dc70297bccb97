"""Workloads of the training-step operators around the RMSNorm, with their plain forms.

Operators: the sandwich norm (norm after a block, gate and residual scale,
norm before the next block; forward and backward), the global gradient norm
and clipping over many tensors, and the embedding lookup with its gradient by
sorted tokens.  ``run`` takes one pass through an operator: through elementary
torch operations in 32 bits (``own`` false) or through this package's entry
points (``own`` true).
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ---------------------------------------------------------------------- cases

def _sandwich(op, T, H, gate, w32, pad=0, name=None):
    c = {"op": op, "T": T, "H": H, "gate": gate, "w32": w32, "pad": pad, "scale": 0.5}
    return dict(c, name=name) if name else c


def _grads(op, layers, H, ffn, dtype, extra, to32=False, name=None):
    c = {"op": op, "layers": layers, "H": H, "ffn": ffn, "dtype": dtype, "extra": extra, "to32": to32}
    return dict(c, name=name) if name else c


def _embed(op, T, H, V, dtype, ids, pad=False, accumulate=False, name=None):
    c = {"op": op, "T": T, "H": H, "V": V, "dtype": dtype, "ids": ids, "pad": pad, "accumulate": accumulate}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token between two blocks (generation inside a training loop): a call's latency
        _sandwich("sandwich_fwd", 1, 2048, "none", False, name="sandwich_fwd_t1_h2048"),
        # a large training batch of a wide model, one learned gate value per token, FP32 norm weights
        _sandwich("sandwich_fwd", 16384, 6144, "row", True, name="sandwich_fwd_t16384_h6144_row"),
        # a short sequence: few rows per SM
        _sandwich("sandwich_bwd", 256, 1536, "none", False, name="sandwich_bwd_t256_h1536"),
        # the backward of an ordinary large batch
        _sandwich("sandwich_bwd", 65536, 4096, "row", False, name="sandwich_bwd_t65536_h4096_row"),
        # a packed batch of odd length, an element gate, and rows that are slices of a wider buffer
        _sandwich("sandwich_bwd", 8191, 5120, "elem", True, pad=64, name="sandwich_bwd_t8191_h5120_elem"),
        # the norm weights and biases of a small model: many tiny tensors
        _grads("clip", 6, 256, 0, "mixed", 13, name="clip_small_params"),
        # every gradient of a model of 0.6 G parameters, BF16, clipped into the optimizer's FP32 buffers
        _grads("clip", 12, 2048, 6144, "bf16", 3, to32=True, name="clip_bf16_into_fp32"),
        # the gradient norm of a logging step over 3 G FP32 values
        _grads("norm", 24, 4096, 5120, "fp32", 1, name="norm_fp32_large"),
        # a decoding batch's lookup
        _embed("embed_fwd", 64, 2048, 32000, "bf16", "int64", name="embed_fwd_t64_h2048"),
        # a training batch's lookup in a large table
        _embed("embed_fwd", 65536, 5120, 100003, "bf16", "int64", name="embed_fwd_t65536_h5120"),
        # a table's whole gradient from one short sequence batch: mostly rows without a token
        _embed("embed_bwd", 8192, 2048, 131072, "fp32", "int64", name="embed_bwd_t8192_h2048"),
        # a large batch added to a gradient that is there already (tied weights), with padding tokens
        _embed("embed_bwd", 65536, 4096, 50000, "fp32", "int32", pad=True, accumulate=True,
               name="embed_bwd_t65536_h4096_acc"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sandwich_fwd", "sandwich_bwd", "sandwich_bwd", "clip", "norm", "embed_fwd", "embed_bwd"])
    if op.startswith("sandwich"):
        H = 8 * _log(rng, 32, 1024)
        T = _log(rng, 1, min(65536, 2 ** 28 // H))
        return _sandwich(op, T, H, rng.choice(["none", "row", "elem"]), rng.random() < 0.5, rng.choice([0, 0, 8, 128]))
    if op in ("clip", "norm"):
        H = _log(rng, 40, 4096)
        ffn = rng.choice([0, _log(rng, 40, 8192)])
        most = 1.0e9 if op == "clip" else 2.0e9
        layers = max(1, min(_log(rng, 1, 60), int(most / (4 * H * H + 3 * H * ffn + 2 * H))))
        return _grads(op, layers, H, ffn, rng.choice(["bf16", "fp32", "mixed"]), rng.randint(0, 40),
                      op == "clip" and rng.random() < 0.3)
    H = 8 * _log(rng, 8, 768)
    T = _log(rng, 1, 65536)
    V = _log(rng, 100, 150000)
    V = max(100, min(V, 2 ** 28 // H))
    if op == "embed_fwd":
        T = max(1, min(T, 2 ** 28 // H))
        return _embed(op, T, H, V, rng.choice(["bf16", "fp32"]), rng.choice(["int64", "int32"]))
    T = max(1, min(T, 2 ** 27 // H))
    return _embed(op, T, H, V, rng.choice(["bf16", "fp32"]), rng.choice(["int64", "int32"]), rng.random() < 0.5,
                  rng.random() < 0.5)


# --------------------------------------------------------------------- inputs

def _shapes(c):
    """The parameter shapes of a stack of blocks (the gradients' shapes), and a few odd ones."""
    H, F = c["H"], c["ffn"]
    got = []
    for _ in range(c["layers"]):
        got += [(H,), (H,)]
        if F:
            got += [(H, H)] * 4 + [(F, H), (F, H), (H, F)]
    return got + [(7 * i + 1,) for i in range(c["extra"])]


def _dtype_of(c, i):
    return {"bf16": BF16, "fp32": F32, "mixed": (BF16, F32)[i % 2]}[c["dtype"]]


def _rows(T, H, pad, g, std=1.0, mean=0.0):
    """BF16 [T, H] of N(mean, std): a slice of a buffer of H + pad columns."""
    buf = torch.empty(T, H + pad, dtype=BF16, device=DEV)
    for a in range(0, T, 8192):
        b = min(T, a + 8192)
        buf[a:b] = (torch.randn(b - a, H + pad, generator=g, device=DEV) * std + mean).to(BF16)
    return buf[:, :H]


def _ids(c, g):
    """Token ids, the k-th commonest with a frequency of about 1/k, the places of the common ones spread over the table."""
    V = c["V"]
    rank = (torch.rand(c["T"], generator=g, device=DEV, dtype=F64) * math.log(V + 1.0)).exp().floor().long() - 1
    ids = torch.randperm(V, generator=g, device=DEV)[rank.clamp_(0, V - 1)]
    if c["pad"]:  # about one token in eight is padding
        ids = torch.where(torch.rand(c["T"], generator=g, device=DEV) < 0.125, torch.full_like(ids, V // 2), ids)
    return ids.to(torch.int32 if c["ids"] == "int32" else torch.int64)


def _flat(c, tensors, dtype_of):
    """One zeroed buffer for each type, and each tensor's place in them as a view of its shape."""
    size, at = {}, []
    for t in tensors:
        dt = dtype_of(t)
        at.append((dt, size.get(dt, 0)))
        size[dt] = at[-1][1] + -(-t.numel() // 64) * 64
    flat = {dt: torch.zeros(n, dtype=dt, device=DEV) for dt, n in size.items()}
    return list(flat.values()), [flat[dt][o:o + t.numel()].view(t.shape) for t, (dt, o) in zip(tensors, at)]


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = {"case": c}
    if c["op"].startswith("sandwich"):
        T, H, wt = c["T"], c["H"], F32 if c["w32"] else BF16
        s["z"] = _rows(T, H, c["pad"], g, 0.7)
        s["x"] = _rows(T, H, c["pad"], g, 1.5)
        s["w_post"] = (1 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(wt)
        s["w_pre"] = (1 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(wt)
        s["gate"] = None
        if c["gate"] == "row":
            s["gate"] = torch.sigmoid(torch.randn(T, generator=g, device=DEV))
        elif c["gate"] == "elem":
            s["gate"] = torch.sigmoid(_rows(T, H, c["pad"], g))
        if c["op"] == "sandwich_bwd":
            _, s["h"], s["rstd_post"], s["rstd_pre"] = _sandwich_fwd(s)
            del s["x"]
            s["dy"] = _rows(T, H, c["pad"], g)
            s["dh"] = _rows(T, H, c["pad"], g)
    elif c["op"] in ("clip", "norm"):
        # gradients of different layers differ in size
        s["grads"] = [(torch.randn(shape, generator=g, device=DEV) * 0.02 * (1 + i % 5)).to(_dtype_of(c, i))
                      for i, shape in enumerate(_shapes(c))]
        s["max_norm"] = 1.0
        if c["op"] == "clip":  # the optimizer's flat buffers, each tensor's part on a boundary of 64 values
            s["flat"], s["out"] = _flat(c, s["grads"], lambda t: F32 if c["to32"] else t.dtype)
    else:
        T, H, V, dt = c["T"], c["H"], c["V"], BF16 if c["dtype"] == "bf16" else F32
        s["ids"] = _ids(c, g)
        s["scale"] = math.sqrt(H) if c["op"] == "embed_fwd" else 0.25
        if c["op"] == "embed_fwd":
            s["table"] = torch.empty(V, H, dtype=dt, device=DEV)
            for a in range(0, V, 8192):
                b = min(V, a + 8192)
                s["table"][a:b] = (torch.randn(b - a, H, generator=g, device=DEV) * 0.02).to(dt)
        else:
            s["dy"] = _rows(T, H, 0, g)
            s["padding_idx"] = V // 2 if c["pad"] else None
            s["out"] = (torch.randn(V, H, generator=g, device=DEV).to(dt)) if c["accumulate"] else None
    return s


# ---------------------------------------------------------------- plain forms

def _sandwich_fwd(s):
    z, x = s["z"].float(), s["x"].float()
    rstd_post = 1.0 / torch.sqrt((z * z).mean(1) + EPS)
    n = z * rstd_post[:, None] * s["w_post"].float()
    if s["gate"] is not None:
        n = n * (s["gate"][:, None] if s["gate"].dim() == 1 else s["gate"].float())
    h_new = (x + s["case"]["scale"] * n).to(BF16)
    h = h_new.float()
    rstd_pre = 1.0 / torch.sqrt((h * h).mean(1) + EPS)
    y = (h * rstd_pre[:, None] * s["w_pre"].float()).to(BF16)
    return y, h_new, rstd_post, rstd_pre


def _sandwich_bwd(s):
    scale = s["case"]["scale"]
    hh = s["h"].float() * s["rstd_pre"][:, None]
    dy = s["dy"].float()
    a = dy * s["w_pre"].float()
    t = s["dh"].float() + s["rstd_pre"][:, None] * (a - hh * (a * hh).mean(1, keepdim=True))
    dw_pre = (dy * hh).sum(0, dtype=F64).float()
    zh = s["z"].float() * s["rstd_post"][:, None]
    gate = s["gate"]
    dn = scale * t
    if gate is not None:
        dn = dn * (gate[:, None] if gate.dim() == 1 else gate.float())
    dw_post = (dn * zh).sum(0, dtype=F64).float()
    b = dn * s["w_post"].float()
    dz = s["rstd_post"][:, None] * (b - zh * (b * zh).mean(1, keepdim=True))
    dgate = None
    if gate is not None:
        dgate = scale * t * (zh * s["w_post"].float())
        dgate = dgate.sum(1) if gate.dim() == 1 else dgate.to(BF16)
    return t.to(BF16), dz.to(BF16), dw_post, dw_pre, dgate


def _norm(s):
    return torch.stack([g.float().square().sum(dtype=F64) for g in s["grads"]]).sum().sqrt().float()


def _clip(s):
    norm = _norm(s)
    coef = torch.clamp(s["max_norm"] / (norm + EPS), max=1.0)
    for g, o in zip(s["grads"], s["out"]):
        o.copy_(g.float() * coef)
    return norm, s["flat"]


def _embed_fwd(s):
    return (s["table"][s["ids"].long()].float() * s["scale"]).to(BF16)


def _embed_bwd(s):
    c, ids, dy = s["case"], s["ids"].long(), s["dy"].float() * s["scale"]
    if s["padding_idx"] is not None:
        dy = dy * (ids != s["padding_idx"])[:, None]
    if c["accumulate"] and c["dtype"] == "fp32":
        return s["out"].index_add_(0, ids, dy)
    total = s["out"].float() if c["accumulate"] else torch.zeros(c["V"], c["H"], device=DEV)
    total.index_add_(0, ids, dy)
    return s["out"].copy_(total) if c["accumulate"] else total.to(BF16 if c["dtype"] == "bf16" else F32)


def _plain(s):
    return {"sandwich_fwd": _sandwich_fwd, "sandwich_bwd": _sandwich_bwd, "norm": _norm, "clip": _clip,
            "embed_fwd": _embed_fwd, "embed_bwd": _embed_bwd}[s["case"]["op"]](s)


def run(state):
    s = state
    c = s["case"]
    if not own:
        return _plain(s)
    import bwd_dw_column_gb300 as cake
    if c["op"] == "sandwich_fwd":
        return cake.cake_sandwich_fwd(s["z"], s["x"], s["w_post"], s["w_pre"], EPS, gate=s["gate"], scale=c["scale"])
    if c["op"] == "sandwich_bwd":
        return cake.cake_sandwich_bwd(s["dy"], s["h"], s["z"], s["rstd_post"], s["rstd_pre"], s["w_post"], s["w_pre"],
                                      dh=s["dh"], gate=s["gate"], scale=c["scale"])
    if c["op"] == "norm":
        return cake.cake_grad_norm(s["grads"])
    if c["op"] == "clip":
        return cake.cake_clip_grad_norm(s["grads"], s["max_norm"], EPS, out=s["out"]), s["flat"]
    if c["op"] == "embed_fwd":
        return cake.cake_embedding_fwd(s["ids"], s["table"], s["scale"])
    return cake.cake_embedding_bwd(s["dy"], s["ids"], c["V"], s["scale"], padding_idx=s["padding_idx"], out=s["out"],
                                   accumulate=c["accumulate"], dtype=BF16 if c["dtype"] == "bf16" else F32)


# ----------------------------------------------------------------------- work

def _distinct(c):
    """About how many of V rows T tokens with frequencies of 1/k name (in closed form: sums over doubling ranks)."""
    V, T = c["V"], c["T"]
    total, lo, got = math.log(V + 1.0), 1, 0.0
    while lo <= V:
        hi = min(2 * lo, V + 1)
        n = hi - lo
        share = math.log(hi / lo) / total
        got += n * (1 - math.exp(-T * share / n))
        lo = hi
    return got


def work(case):
    c = case
    if c["op"].startswith("sandwich"):
        T, H = c["T"], c["H"]
        wb = H * (8 if c["w32"] else 4)
        gate = {"none": 0, "row": 4 * T, "elem": 2 * T * H}[c["gate"]]
        if c["op"] == "sandwich_fwd":
            return {"bytes": 8 * T * H + 8 * T + wb + gate, "flops": 12 * T * H}
        return {"bytes": 12 * T * H + 8 * T + wb + 8 * H + 2 * gate, "flops": 30 * T * H}
    if c["op"] in ("clip", "norm"):
        moved = n = 0
        for i, shape in enumerate(_shapes(c)):
            k, size = math.prod(shape), 2 if _dtype_of(c, i) == BF16 else 4
            n += k
            moved += k * size + ((k * (4 if c["to32"] else size)) if c["op"] == "clip" else 0)
        return {"bytes": moved + 4, "flops": (3 if c["op"] == "clip" else 2) * n}
    T, H, V, size = c["T"], c["H"], c["V"], 2 if c["dtype"] == "bf16" else 4
    ids = T * (4 if c["ids"] == "int32" else 8)
    rows = _distinct(c)
    if c["op"] == "embed_fwd":
        return {"bytes": int(ids + rows * H * size + 2 * T * H), "flops": T * H}
    table = 2 * rows * H * size if c["accumulate"] else V * H * size
    live = 0.875 if c["pad"] else 1.0
    return {"bytes": int(ids + 2 * live * T * H + table), "flops": T * H}


# ---------------------------------------------------------------------- exact

def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "sandwich_fwd":
        # vectors of each row divided by their root mean square; the second norm is of the stored BF16 sum
        def unit(v):
            r = torch.linalg.vector_norm(v, dim=1, keepdim=True).square() / c["H"] + EPS
            return v * r.rsqrt(), r.rsqrt()[:, 0]
        nz, r1 = unit(s["z"].to(F64))
        add = nz * s["w_post"].to(F64) * c["scale"]
        if s["gate"] is not None:
            add = add * s["gate"].to(F64).reshape(c["T"], -1)
        h = s["x"].to(F64) + add
        y, r2 = unit(h.to(BF16).to(F64))
        return y * s["w_pre"].to(F64), h, r1, r2
    if c["op"] == "sandwich_bwd":
        # differentiated by torch in 64 bits, first through the second norm, then through the gated sum
        leaf = lambda k: s[k].to(F64).detach().requires_grad_()  # noqa: E731
        h, w2 = leaf("h"), leaf("w_pre")
        y = h * (h.square().mean(1, keepdim=True) + EPS).rsqrt() * w2
        t, dw_pre = torch.autograd.grad(y, (h, w2), s["dy"].to(F64))
        t = t + s["dh"].to(F64)
        del h, y
        z, w1 = leaf("z"), leaf("w_post")
        g = leaf("gate") if s["gate"] is not None else None
        add = z * (z.square().mean(1, keepdim=True) + EPS).rsqrt() * w1 * c["scale"]
        if g is not None:
            add = add * g.reshape(c["T"], -1)
        got = torch.autograd.grad(add, (z, w1) + ((g,) if g is not None else ()), t)
        return t, got[0], got[1], dw_pre, got[2] if g is not None else None
    if c["op"] in ("clip", "norm"):
        norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g, dtype=F64)) ** 2 for g in s["grads"]))
        if c["op"] == "norm":
            return torch.tensor(norm, dtype=F64)
        k = min(1.0, s["max_norm"] / (norm + EPS))
        # one place for each of the output types, in the order in which they come up
        parts = {}
        for g in s["grads"]:
            v = torch.nn.functional.pad(g.reshape(-1), (0, -g.numel() % 64)).to(F64) * k
            parts.setdefault(F32 if c["to32"] else g.dtype, []).append(v)
        return torch.tensor(norm, dtype=F64), [torch.cat(v) for v in parts.values()]
    if c["op"] == "embed_fwd":
        return torch.nn.functional.embedding(s["ids"].long(), s["table"]).to(F64) * s["scale"]
    # rows of equal ids brought together, then each run of rows summed as a difference of running sums, by column blocks
    order = torch.argsort(s["ids"].long(), stable=True)
    ids = s["ids"].long()[order]
    if s["padding_idx"] is not None:
        order, ids = order[ids != s["padding_idx"]], ids[ids != s["padding_idx"]]
    got = s["out"].to(F64) if c["accumulate"] else torch.zeros(c["V"], c["H"], dtype=F64, device=DEV)
    rows, counts = torch.unique_consecutive(ids, return_counts=True)
    ends = counts.cumsum(0)
    for a in range(0, c["H"], 512):
        run_sum = s["dy"][:, a:a + 512][order].to(F64).cumsum(0)
        upto = run_sum[ends - 1]
        part = upto - torch.cat([torch.zeros_like(upto[:1]), upto[:-1]])
        got[rows, a:a + 512] += s["scale"] * part
    return got
