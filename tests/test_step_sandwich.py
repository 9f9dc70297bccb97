"""The sandwich norm against its FP64 form: forward and backward, each gate,
both weight types, odd rows and widths, strided rows, in place, zero rows,
graphs and streams.  The FP64 backward is itself held to finite differences
and to torch's differentiation on the CPU."""
import pytest
import torch

from tests import step_reference as ref

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
EPS = 1e-6


@pytest.fixture(scope="module")
def cake():
    import __graft_entry__
    __graft_entry__.build()
    import bwd_dw_column_gb300 as cake
    yield cake


def case(T, H, gate="none", nh=None, pad=0, w=(torch.bfloat16, torch.float32), seed=0, device="cpu", offset=0.0):
    g = torch.Generator().manual_seed(seed * 7919 + T * 31 + H)
    shape = (T, H) if nh is None else (T, nh, H)

    def rows(std=1.0, mean=0.0):
        buf = torch.randn(*shape[:-1], H + pad, generator=g) * std + mean
        return buf.to(torch.bfloat16).to(device)[..., :H]

    c = {"z": rows(0.7, offset), "x": rows(1.5), "dy": rows(), "dh": rows(),
         "w_post": (1 + 0.1 * torch.randn(H, generator=g)).to(w[0]).to(device),
         "w_pre": (1 + 0.1 * torch.randn(H, generator=g)).to(w[1]).to(device), "gate": None}
    if gate == "row":
        c["gate"] = torch.sigmoid(torch.randn(shape[:-1], generator=g)).to(device)
    elif gate == "elem":
        c["gate"] = torch.sigmoid(rows().float()).to(torch.bfloat16)
    return c


def check_fwd(cake, c, scale, **kw):
    y, h, r1, r2 = cake.cake_sandwich_fwd(c["z"], c["x"], c["w_post"], c["w_pre"], EPS, c["gate"], scale, **kw)
    torch.cuda.synchronize()
    h64, add, r64 = ref.sandwich_fwd(c["z"], c["x"], c["w_post"], c["w_pre"], EPS, c["gate"], scale)
    # x is exact; the added term carries rstd's error, four products and a sum
    err = (add.abs() * (ref.RSTD_REL + 6 * ref.U) + ref.U * h64.abs())
    assert ref.excess(h, h64, ref.rounded(h64, err)) <= 1
    assert float((r1.double().view(r64.shape) / r64 - 1).abs().max()) <= ref.RSTD_REL
    y64, r64 = ref.norm_fwd(h, c["w_pre"], EPS)  # of the h_new that was stored
    assert float((r2.double().view(r64.shape) / r64 - 1).abs().max()) <= ref.RSTD_REL
    assert ref.excess(y, y64, ref.rounded(y64, y64.abs() * (ref.RSTD_REL + 3 * ref.U))) <= 1
    return y, h, r1, r2


def check_bwd(cake, c, scale, with_dh=True, h=None, r=None, **kw):
    if h is None:
        _, h, r1, r2 = cake.cake_sandwich_fwd(c["z"], c["x"], c["w_post"], c["w_pre"], EPS, c["gate"], scale)
    else:
        r1, r2 = r
    dh = c["dh"] if with_dh else None
    got = cake.cake_sandwich_bwd(c["dy"], h, c["z"], r1, r2, c["w_post"], c["w_pre"], dh, c["gate"], scale, **kw)
    torch.cuda.synchronize()
    want = ref.sandwich_bwd(c["dy"], h, c["z"], r1, r2, c["w_post"], c["w_pre"], dh, c["gate"], scale)
    for name, v in zip(("dx", "dz", "dw_post", "dw_pre", "dgate"), got):
        if name in want:
            assert ref.excess(v, *want[name]) <= 1, name
        else:
            assert v is None
    return got


# ------------------------------------------------------------------ the form

@pytest.mark.parametrize("gate", ["none", "row", "elem"])
def test_fp64_backward_is_the_derivative(gate):
    c = case(3, 16, gate, seed=3)
    scale = 0.7
    f64 = lambda t: t.double().detach().requires_grad_()  # noqa: E731
    z, x, w1, w2 = (f64(c[k]) for k in ("z", "x", "w_post", "w_pre"))
    gt = f64(c["gate"]) if c["gate"] is not None else None
    dy, dh = c["dy"].double(), c["dh"].double()

    def loss(z, x, w1, w2, gt):
        h, _, _ = ref.sandwich_fwd(z, x, w1, w2, EPS, gt, scale)
        return (ref.norm_fwd(h, w2, EPS)[0] * dy).sum() + (h * dh).sum()

    leaves = [t for t in (x, z, w1, w2, gt) if t is not None]
    auto = torch.autograd.grad(loss(z, x, w1, w2, gt), leaves)
    h, _, r1 = ref.sandwich_fwd(z, x, w1, w2, EPS, gt, scale)
    _, r2 = ref.norm_fwd(h, w2, EPS)
    want = ref.sandwich_bwd(dy, h, z, r1, r2, w1, w2, dh, gt, scale)
    for name, a in zip(("dx", "dz", "dw_post", "dw_pre", "dgate"), auto):
        assert torch.allclose(want[name][0], a, rtol=1e-10, atol=1e-12), name
    # and by differences of the loss along a direction
    with torch.no_grad():
        for i, t in enumerate(leaves):
            d = torch.randn(t.shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64)
            step = 1e-5
            args = {"z": z, "x": x, "w1": w1, "w2": w2, "gt": gt}
            key = next(k for k, v in args.items() if v is t)
            up, down = (loss(**{**args, key: t + s * step * d}) for s in (1, -1))
            assert abs((up - down) / (2 * step) - (auto[i] * d).sum()) <= 1e-6 * (1 + abs((auto[i] * d).sum()))


# ------------------------------------------------------------------- kernels

SHAPES = [(1, 8), (1, 2048), (2, 64), (5, 256), (7, 264), (33, 520), (3, 1024), (129, 1536), (3, 4104), (17, 5120),
          (2, 6144), (3, 8192), (4, 8192), (305, 7936), (311, 2048), (613, 128)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("gate", ["none", "row", "elem"])
def test_sandwich(cake, T, H, gate):
    c = case(T, H, gate, device=DEV, w=[(torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)][T % 2])
    _, h, r1, r2 = check_fwd(cake, c, 0.5)
    check_bwd(cake, c, 0.5, with_dh=T % 3 != 0, h=h, r=(r1, r2))


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["row", "elem"])
def test_strided_rows_and_heads(cake, gate):
    c = case(37, 320, gate, pad=24, device=DEV)
    c["x"] = case(37, 320, pad=8, device=DEV)["x"]
    check_fwd(cake, c, -1.25)
    check_bwd(cake, c, -1.25)
    c = case(9, 512, gate, nh=3, pad=8, device=DEV)
    out = [torch.full((9, 3, 640), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    views = [o[..., 64:576] for o in out]
    check_fwd(cake, c, 2.0, y=views[0], h_new=views[1])
    check_bwd(cake, c, 2.0, dx=views[0], dz=views[1])
    for o in out:  # what is between the rows stays
        assert bool((o[..., :64] == 7).all()) and bool((o[..., 576:] == 7).all())


@pytest.mark.gpu
def test_permuted_heads(cake):
    # heads outside tokens: the token stride is the smaller one
    c = case(6, 256, "row", nh=4, device=DEV)
    for k in ("z", "x", "dy", "dh"):
        c[k] = c[k].transpose(0, 1).contiguous().transpose(0, 1)
    check_fwd(cake, c, 0.5)
    check_bwd(cake, c, 0.5)


@pytest.mark.gpu
def test_in_place_forward(cake):
    c = case(300, 1536, "row", device=DEV)
    want = [t.clone() for t in cake.cake_sandwich_fwd(c["z"], c["x"], c["w_post"], c["w_pre"], EPS, c["gate"], 0.5)]
    got = cake.cake_sandwich_fwd(c["z"], c["x"], c["w_post"], c["w_pre"], EPS, c["gate"], 0.5, y=c["z"], h_new=c["x"])
    torch.cuda.synchronize()
    assert got[0].data_ptr() == c["z"].data_ptr() and got[1].data_ptr() == c["x"].data_ptr()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [8, 256, 264, 320, 384, 392, 512, 520, 640, 704, 768, 776, 1000, 1024, 1032, 1096, 1152, 1280, 1544,
                               1664, 1920, 2056, 2560, 3584, 4608])
def test_row_widths(cake, H):
    # a CTA's first, middle and last tiles of every layout of warps to rows
    gate = ("none", "row", "elem")[H // 8 % 3]
    c = case(2501 if H <= 256 else 1501, H, gate, device=DEV)
    _, h, r1, r2 = check_fwd(cake, c, 0.5)
    check_bwd(cake, c, 0.5, h=h, r=(r1, r2))


@pytest.mark.gpu
@pytest.mark.parametrize("H", [3080, 4104, 5120, 6144, 7168, 8192])
@pytest.mark.parametrize("gate", ["none", "row", "elem"])
def test_many_rows_over_clusters(cake, H, gate):
    # rows split over 2 and 4 CTAs: 9 tiles of a cluster and more, so that the ring, and the four slots and
    # barriers of the sums that cross between its CTAs, come round several times
    c = case(2999, H, gate, device=DEV, w=[(torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)][H // 8 % 2])
    _, h, r1, r2 = check_fwd(cake, c, 0.5)
    a = check_bwd(cake, c, 0.5, h=h, r=(r1, r2))
    for _ in range(3):
        b = check_bwd(cake, c, 0.5, h=h, r=(r1, r2))
        for s, t in zip(a, b):
            assert s is None and t is None or torch.equal(s, t)  # bit for bit


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4096, 20011])
def test_many_rows(cake, T):
    c = case(T, 768, "row", device=DEV, offset=1.0)
    _, h, r1, r2 = check_fwd(cake, c, 0.5)
    a = check_bwd(cake, c, 0.5, h=h, r=(r1, r2))
    b = check_bwd(cake, c, 0.5, h=h, r=(r1, r2))
    for s, t in zip(a, b):
        assert torch.equal(s, t)  # bit for bit


@pytest.mark.gpu
def test_zero_rows_and_values(cake):
    c = case(6, 512, "elem", device=DEV)
    c["z"][1] = 0      # a block that gives nothing
    c["gate"][2] = 0   # a closed gate
    c["x"][3] = 0
    c["dy"][4] = 0
    check_fwd(cake, c, 0.5)
    check_bwd(cake, c, 0.5)
    for scale in (0.0, 1.0):
        check_bwd(cake, c, scale)


@pytest.mark.gpu
def test_nan_stays_in_its_row(cake):
    c = case(40, 256, "row", device=DEV)
    clean = cake.cake_sandwich_fwd(c["z"], c["x"], c["w_post"], c["w_pre"], EPS, c["gate"], 0.5)
    c["z"][17, 3] = float("nan")
    y, h, r1, r2 = cake.cake_sandwich_fwd(c["z"], c["x"], c["w_post"], c["w_pre"], EPS, c["gate"], 0.5)
    dx, dz, _, _, dg = cake.cake_sandwich_bwd(c["dy"], h, c["z"], r1, r2, c["w_post"], c["w_pre"], c["dh"], c["gate"],
                                              0.5)
    torch.cuda.synchronize()
    keep = [i for i in range(40) if i != 17]
    for a, b in zip((y, h, r1, r2), clean):
        assert torch.equal(a[keep], b[keep]) and bool(torch.isnan(a[17]).any())
    for t in (dx, dz, dg):
        assert bool(torch.isfinite(t[keep]).all())


@pytest.mark.gpu
def test_no_rows(cake):
    c = case(0, 64, "row", device=DEV)
    y, h, r1, r2 = cake.cake_sandwich_fwd(c["z"], c["x"], c["w_post"], c["w_pre"], EPS, c["gate"])
    assert y.shape == (0, 64) and r1.numel() == 0
    dw = torch.full((64,), 5.0, device=DEV)
    got = cake.cake_sandwich_bwd(c["dy"], h, c["z"], r1, r2, c["w_post"], c["w_pre"], gate=c["gate"], dw_post=dw)
    torch.cuda.synchronize()
    assert not dw.any() and not got[3].any() and got[0].shape == (0, 64)


@pytest.mark.gpu
def test_python_refusals(cake):
    c = case(4, 64, device=DEV)
    z, x, w1, w2 = c["z"], c["x"], c["w_post"], c["w_pre"]
    with pytest.raises(ValueError):
        cake.cake_sandwich_fwd(z, x[:3], w1, w2)
    with pytest.raises(ValueError):
        cake.cake_sandwich_fwd(z, x, w1[:32], w2)
    with pytest.raises(ValueError):
        cake.cake_sandwich_fwd(z, x, w1, w2, gate=torch.ones(3, device=DEV))
    with pytest.raises(TypeError):
        cake.cake_sandwich_fwd(z, x, w1, w2, gate=torch.ones(4, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(TypeError):
        cake.cake_sandwich_fwd(z, x, w1, w2, gate=torch.ones(4, 64, device=DEV))
    with pytest.raises(TypeError):
        cake.cake_sandwich_fwd(z.float(), x, w1, w2)
    with pytest.raises(ValueError):
        cake.cake_sandwich_fwd(z, x.cpu(), w1, w2)
    with pytest.raises(cake.CakeError):
        cake.cake_sandwich_fwd(z, x, w1, w2, y=x, h_new=x)
    with pytest.raises(cake.CakeError):
        cake.cake_sandwich_fwd(z, x, w1, w2, eps=-1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["none", "row", "elem"])
def test_autograd_gives_the_entry_points_bits(cake, gate):
    c = case(77, 640, gate, device=DEV)
    leaf = lambda t: None if t is None else t.detach().clone().requires_grad_()  # noqa: E731
    z, x, w1, w2, g = (leaf(c[k]) for k in ("z", "x", "w_post", "w_pre", "gate"))
    y, h = cake.cake_sandwich_norm(z, x, w1, w2, EPS, g, 0.5)
    torch.autograd.backward([y, h], [c["dy"], c["dh"]])
    _, h2, r1, r2 = cake.cake_sandwich_fwd(c["z"], c["x"], c["w_post"], c["w_pre"], EPS, c["gate"], 0.5)
    dx, dz, dwo, dwr, dg = cake.cake_sandwich_bwd(c["dy"], h2, c["z"], r1, r2, c["w_post"], c["w_pre"], c["dh"],
                                                  c["gate"], 0.5)
    torch.cuda.synchronize()
    assert torch.equal(h, h2) and torch.equal(x.grad, dx) and torch.equal(z.grad, dz)
    assert torch.equal(w1.grad, dwo.to(w1.dtype)) and torch.equal(w2.grad, dwr.to(w2.dtype))
    if g is not None:
        assert torch.equal(g.grad, dg)


@pytest.mark.gpu
def test_autograd_with_one_output_used(cake):
    c = case(20, 256, device=DEV)
    for use in (0, 1):
        z, x, w1, w2 = (c[k].detach().clone().requires_grad_() for k in ("z", "x", "w_post", "w_pre"))
        out = cake.cake_sandwich_norm(z, x, w1, w2, EPS, None, 0.5)
        out[use].backward(c["dy"])
        zero = torch.zeros_like(c["dy"])
        _, h, r1, r2 = cake.cake_sandwich_fwd(c["z"], c["x"], c["w_post"], c["w_pre"], EPS, None, 0.5)
        dx, dz, _, _, _ = cake.cake_sandwich_bwd(c["dy"] if use == 0 else zero, h, c["z"], r1, r2, c["w_post"],
                                                 c["w_pre"], None if use == 0 else c["dy"], None, 0.5)
        torch.cuda.synchronize()
        assert torch.equal(x.grad, dx) and torch.equal(z.grad, dz)


@pytest.mark.gpu
def test_broadcast_gate_gradient(cake):
    # one learned gate for all rows: torch sums the rows' gradients of the expanded value
    c = case(50, 512, device=DEV)
    g = torch.tensor(0.3, device=DEV, requires_grad=True)
    y, h = cake.cake_sandwich_norm(c["z"], c["x"], c["w_post"], c["w_pre"], EPS, g.expand(50), 0.5)
    torch.autograd.backward([y, h], [c["dy"], c["dh"]])
    _, hn, r1, r2 = cake.cake_sandwich_fwd(c["z"], c["x"], c["w_post"], c["w_pre"], EPS, g.detach().expand(50), 0.5)
    v, bound = ref.sandwich_bwd(c["dy"], hn, c["z"], r1, r2, c["w_post"], c["w_pre"], c["dh"],
                                g.detach().expand(50), 0.5)["dgate"]
    assert abs(float(g.grad) - float(v.sum())) <= float(bound.sum()) + 50 * ref.U * float(v.abs().sum())


@pytest.mark.gpu
def test_rows_beyond_2_to_31_values(cake):
    # the last rows of a tensor of 2.2e9 values come out as they do by themselves
    T, H, n = 270_000, 8192, 5
    c = case(n, H, "row", device=DEV)
    big = {k: torch.zeros(T, H, dtype=torch.bfloat16, device=DEV) for k in ("z", "x", "dy", "dh")}
    for k, v in big.items():
        v[-n:] = c[k]
    gate = torch.zeros(T, device=DEV)
    gate[-n:] = c["gate"]
    w = (c["w_post"], c["w_pre"])
    got = cake.cake_sandwich_fwd(big["z"], big["x"], *w, EPS, gate, 0.5, y=big["z"].clone(), h_new=big["x"].clone())
    want = cake.cake_sandwich_fwd(c["z"], c["x"], *w, EPS, c["gate"], 0.5)
    for a, b in zip(got, want):
        assert torch.equal(a[-n:], b)
    del want
    y, h, r1, r2 = got
    dx, dz, dwo, dwr, dg = cake.cake_sandwich_bwd(big["dy"], h, big["z"], r1, r2, *w, big["dh"], gate, 0.5, dx=y)
    small = cake.cake_sandwich_bwd(c["dy"], h[-n:], c["z"], r1[-n:], r2[-n:], *w, c["dh"], c["gate"], 0.5)
    for a, b in zip((dx, dz, dg), (small[0], small[1], small[4])):
        assert torch.equal(a[-n:], b)
    # all other rows are zero, so the column sums are these rows' alone, added in another order
    ref_sums = ref.sandwich_bwd(c["dy"], h[-n:], c["z"], r1[-n:], r2[-n:], *w, c["dh"], c["gate"], 0.5)
    assert ref.excess(dwo, *ref_sums["dw_post"]) <= 1 and ref.excess(dwr, *ref_sums["dw_pre"]) <= 1


@pytest.mark.gpu
def test_two_graphs_on_two_streams(cake):
    """Captured calls keep their own workspaces: two graphs replayed at once give what each gives alone."""
    cases = [case(3000, 1536, "row", device=DEV, seed=s) for s in (1, 2)]

    def step(c):
        _, h, r1, r2 = cake.cake_sandwich_fwd(c["z"], c["x"], c["w_post"], c["w_pre"], EPS, c["gate"], 0.5)
        return cake.cake_sandwich_bwd(c["dy"], h, c["z"], r1, r2, c["w_post"], c["w_pre"], c["dh"], c["gate"], 0.5)

    want = [[t.clone() for t in step(c)] for c in cases]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(c))
        graphs.append(g)
    for _ in range(5):
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            for a, b in zip(o, w):
                assert torch.equal(a, b)


@pytest.mark.gpu
def test_given_stream(cake):
    c = case(2000, 1024, "elem", device=DEV)
    want = cake.cake_sandwich_fwd(c["z"], c["x"], c["w_post"], c["w_pre"], EPS, c["gate"], 0.5)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = cake.cake_sandwich_fwd(c["z"], c["x"], c["w_post"], c["w_pre"], EPS, c["gate"], 0.5, stream=s)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["row", "elem"])
@pytest.mark.parametrize("T,nh,H", [(40, None, 640), (9, 4, 264), (300, None, 5120)])
def test_given_outputs(cake, T, nh, H, gate):
    """Every output in a tensor of the caller's, rows strided where they may be, gives the bits of a new one."""
    c = case(T, H, gate, nh=nh, device=DEV)
    args = (c["w_post"], c["w_pre"], EPS, c["gate"], 0.5)
    want = cake.cake_sandwich_fwd(c["z"], c["x"], *args)
    lead = c["z"].shape[:-1]
    rstd = [torch.full(lead, 7.0, device=DEV) for _ in range(2)]
    got = cake.cake_sandwich_fwd(c["z"], c["x"], *args, rstd_post=rstd[0], rstd_pre=rstd[1])
    assert got[2] is rstd[0] and got[3] is rstd[1]
    for a, b in zip(got, want):
        assert torch.equal(a.flatten(), b.flatten())
    _, h, r1, r2 = got
    back = (c["dy"], h, c["z"], r1, r2, c["w_post"], c["w_pre"], c["dh"], c["gate"], 0.5)
    want = check_bwd(cake, c, 0.5, h=h, r=(r1, r2))
    buf = torch.full((*lead, H + 24), 7.0, dtype=torch.bfloat16, device=DEV)
    dgate = buf[..., 16:16 + H] if gate == "elem" else torch.full(lead, 7.0, device=DEV)
    dw = torch.full((2, H), 7.0, device=DEV)
    got = cake.cake_sandwich_bwd(*back, dgate=dgate, dw_post=dw[0], dw_pre=dw[1])
    assert got[4] is dgate and got[2].data_ptr() == dw.data_ptr()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    if gate == "elem":
        assert bool((buf[..., :16] == 7).all()) and bool((buf[..., 16 + H:] == 7).all())
    # the gate's gradient left out
    got = cake.cake_sandwich_bwd(*back, need_dgate=False)
    assert got[4] is None
    for a, b in zip(got[:4], want):
        assert torch.equal(a, b)
    with pytest.raises(ValueError):
        cake.cake_sandwich_bwd(*back, need_dgate=False, dgate=dgate)
    with pytest.raises(ValueError):
        cake.cake_sandwich_bwd(*back, dgate=dgate[:-1])
    with pytest.raises((ValueError, TypeError)):
        cake.cake_sandwich_bwd(*back, dgate=dgate.double())
    with pytest.raises(ValueError):
        cake.cake_sandwich_bwd(*back[:8], None, 0.5, dgate=dgate)
    with pytest.raises(ValueError):
        cake.cake_sandwich_bwd(*back, dw_pre=dw[0, :-1])
    with pytest.raises(ValueError):
        cake.cake_sandwich_fwd(c["z"], c["x"], *args, rstd_post=rstd[0].flatten()[1:])


@pytest.mark.gpu
def test_one_workspace_for_ordered_calls(cake):
    """Calls of several widths, gates and row counts one after another in one workspace that holds garbage."""
    cases = [case(T, H, gate, device=DEV) for T, H, gate in
             [(700, 1536, "none"), (1, 64, "row"), (300, 5120, "elem"), (2000, 264, "row"), (64, 8192, "none")]]
    calls, want, size = [], [], 0
    for c in cases:
        _, h, r1, r2 = cake.cake_sandwich_fwd(c["z"], c["x"], c["w_post"], c["w_pre"], EPS, c["gate"], 0.5)
        calls.append((c["dy"], h, c["z"], r1, r2, c["w_post"], c["w_pre"], c["dh"], c["gate"], 0.5))
        want.append(check_bwd(cake, c, 0.5, h=h, r=(r1, r2)))
        size = max(size, cake.cake_sandwich_bwd_workspace_size(c["z"]))
    ws = torch.full((size,), 0xff, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        got = [cake.cake_sandwich_bwd(*a, workspace=ws) for a in calls]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for a, b in zip(g, w):
                assert a is None and b is None or torch.equal(a, b)
    with pytest.raises(cake.CakeError):
        cake.cake_sandwich_bwd(*calls[2], workspace=ws[:1024])
    with pytest.raises(cake.CakeError):
        cake.cake_sandwich_bwd(*calls[0], workspace=ws[8:])
    with pytest.raises(ValueError):
        cake.cake_sandwich_bwd(*calls[0], workspace=ws[::2])


@pytest.mark.gpu
def test_a_gate_without_a_gradient(cake):
    for gate in ("row", "elem"):
        c = case(33, 520, gate, device=DEV)
        z = c["z"].clone().requires_grad_()
        y, h = cake.cake_sandwich_norm(z, c["x"], c["w_post"], c["w_pre"], EPS, c["gate"], 0.5)
        torch.autograd.backward([y, h], [c["dy"], c["dh"]])
        want = check_bwd(cake, c, 0.5)
        assert torch.equal(z.grad, want[1]) and c["gate"].grad is None


@pytest.mark.gpu
@pytest.mark.parametrize("nh", [None, 3])
def test_tensors_in_columns_of_one_buffer(cake, nh):
    T, H = 33, 320
    c = case(T, H, "elem", nh=nh, device=DEV)
    args = (c["w_post"], c["w_pre"], EPS, c["gate"], 0.5)
    want = cake.cake_sandwich_fwd(c["z"], c["x"], *args)
    back = check_bwd(cake, c, 0.5, h=want[1], r=want[2:])
    lead = c["z"].shape[:-1]
    buf = torch.full((*lead, 2 * H), 7.0, dtype=torch.bfloat16, device=DEV)
    y, h = buf.chunk(2, dim=-1)
    got = cake.cake_sandwich_fwd(c["z"], c["x"], *args, y=y, h_new=h)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    y.copy_(c["z"]), h.copy_(c["x"])  # and in place
    got = cake.cake_sandwich_fwd(y, h, *args, y=y, h_new=h)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    wide = torch.full((*lead, 4 * H), 7.0, dtype=torch.bfloat16, device=DEV)
    dy, dx, dz, dg = wide.chunk(4, dim=-1)
    dy.copy_(c["dy"])
    got = cake.cake_sandwich_bwd(dy, want[1], c["z"], *want[2:], c["w_post"], c["w_pre"], c["dh"], c["gate"], 0.5,
                                 dx=dx, dz=dz, dgate=dg)
    for a, b in zip(got, back):
        assert torch.equal(a, b)
    assert torch.equal(dy, c["dy"])
    with pytest.raises(cake.CakeError):
        cake.cake_sandwich_fwd(c["z"], c["x"], *args, y=buf[..., :H], h_new=buf[..., H - 8:2 * H - 8])
