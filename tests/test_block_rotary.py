"""The per-head norm of queries and keys with rotary positions, against FP64 on
a GB300."""
import pytest
import torch

from tests import block_reference as ref

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF16, F32 = torch.bfloat16, torch.float32
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cake():
    import __graft_entry__
    __graft_entry__.build()
    import bwd_dw_column_gb300 as cake
    yield cake
    assert cake.cake_rmsnorm_device_status() == 0


def check(name, got, want, allow):
    share = ref.excess(got.reshape(want.shape), want, allow)
    assert share <= 1, f"{name}: {share:.3g} of its bound"


def heads(g, T, n, D, gap=0, mean=0.3):
    return (torch.randn(T, n, D + gap, generator=g) + mean).to(BF16).to(DEV)[..., :D]


def weights(g, D, w32):
    return (1 + 0.1 * torch.randn(D, generator=g)).to(F32 if w32 else BF16).to(DEV)


#        T, q heads, k heads, D, sections, style, gap, positions' type, far
CASES = [(1, 24, 4, 256, (128,), "half", 0, torch.int64, 100000),
         (1, 1, 0, 16, (8,), "adjacent", 0, torch.int32, 10),
         (5, 3, 1, 32, (8,), "half", 0, torch.int64, 1 << 20),
         (5, 3, 1, 32, (8,), "adjacent", 16, torch.int32, 1 << 20),
         (77, 6, 2, 64, (32,), "half", 64, torch.int64, 4096),
         (130, 5, 5, 80, (5, 11, 24), "half", 0, torch.int64, 300),
         (131, 4, 2, 96, (16, 16, 8), "adjacent", 8, torch.int64, 300),
         (67, 16, 16, 128, (16, 24, 24), "adjacent", 0, torch.int64, 300),
         (33, 24, 4, 256, (64,), "half", 256, torch.int64, 1 << 30),
         (40, 2, 2, 256, (8, 8, 8, 8), "half", 0, torch.int32, 70000),
         (19, 2, 1, 512, (256,), "adjacent", 0, torch.int64, 1 << 40),
         (21, 3, 1, 384, (64,), "half", 0, torch.int64, 1 << 20),
         (9, 2, 1, 128, (), "half", 0, torch.int64, 5),
         (3000, 8, 2, 64, (32,), "half", 0, torch.int64, 1 << 17)]


def make(cake, case):
    T, nq, nk, D, sections, style, gap, it, far = case
    g = torch.Generator().manual_seed(T + D)
    q, k = heads(g, T, nq, D, gap), heads(g, T, nk, D) if nk else None
    pos = torch.randint(-far if len(sections) == 1 else 0, far, (max(1, len(sections)), T), generator=g).to(it).to(DEV)
    turns, axes = cake.cake_rotary_table(sections, device=DEV)
    if len(sections) <= 1:
        pos, axes = pos[0], None
    return g, q, k, pos, turns, axes, style


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_rotary_fwd(cake, case, norm):
    g, q, k, pos, turns, axes, style = make(cake, case)
    D = q.shape[-1]
    w = [weights(g, D, True), weights(g, D, False)] if norm else [None, None]
    if k is None:
        w[1] = None
    angle = ref.phases(pos, turns, axes)
    got = cake.cake_rotary_fwd(q, k, pos, turns, axes, *w, 1e-6, style=style)
    for v, wv, y, rstd in zip((q, k), w, got[:2], got[2:]):
        if v is None:
            assert y is None and rstd is None
            continue
        want, allow, r64 = ref.rotary_fwd(v, angle, wv, 1e-6, style)
        check("y", y, want, allow)
        if norm:
            check("rstd", rstd, r64, ref.RSTD_REL * r64)
        else:
            assert rstd is None
    # in place, into slices of one buffer: queries and keys of a fused product
    if k is not None:
        T, nq, nk = q.shape[0], q.shape[1], k.shape[1]
        qkv = torch.full((T, (nq + 2 * nk) * D), 7.0, dtype=BF16, device=DEV)
        a, b = qkv[:, :nq * D].view(T, nq, D), qkv[:, nq * D:(nq + nk) * D].view(T, nk, D)
        a.copy_(q)
        b.copy_(k)
        cake.cake_rotary_fwd(a, b, pos, turns, axes, *w, 1e-6, style=style, q_out=a, k_out=b)
        assert torch.equal(a, got[0]) and torch.equal(b, got[1])
        assert bool((qkv[:, (nq + nk) * D:] == 7.0).all())


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_rotary_bwd(cake, case, norm):
    g, q, k, pos, turns, axes, style = make(cake, case)
    D = q.shape[-1]
    w = [weights(g, D, False), weights(g, D, True)] if norm else [None, None]
    if k is None:
        w[1] = None
    dy = [None if v is None else heads(g, *v.shape, gap, 0.0) for v, gap in ((q, 0), (k, 16))]
    rstd = [None if v is None or not norm else (1 / torch.sqrt((v.float() ** 2).mean(-1) + 1e-6)).reshape(-1)
            for v in (q, k)]
    angle = ref.phases(pos, turns, axes)
    got = cake.cake_rotary_bwd(*dy, pos, turns, axes, q, k, *rstd, *w, style=style)
    for d, v, r, wv, dv, dw in zip(dy, (q, k), rstd, w, got[:2], got[2:]):
        if v is None:
            assert dv is None and dw is None
            continue
        want, allow, dw64, edw = ref.rotary_bwd(d, angle, v, r, wv, style)
        check("dv", dv, want, allow)
        if norm:
            check("dw", dw, dw64, edw)
        else:
            assert dw is None
    again = cake.cake_rotary_bwd(*(None if d is None else d.clone() for d in dy), pos, turns, axes, q, k, *rstd, *w,
                                 style=style)
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, again))
    # in place over the incoming gradients
    dy = [None if d is None else d.clone() for d in dy]
    cake.cake_rotary_bwd(*dy, pos, turns, axes, q, k, *rstd, *w, style=style, dq_out=dy[0], dk_out=dy[1])
    assert torch.equal(dy[0], got[0]) and (k is None or torch.equal(dy[1], got[1]))


def test_tables(cake):
    """Ladders of each axis, a shared one and given frequencies; the parts of a turn to the last bit that FP64 has."""
    import math
    turns, axes = cake.cake_rotary_table((2, 3), 100.0, device=DEV)
    assert axes.tolist() == [0, 0, 1, 1, 1]
    want = [100.0 ** -(i / n) for n in (2, 3) for i in range(n)]
    got = [(t % 2 ** 64) / 2 ** 64 * 2 * math.pi for t in turns.tolist()]
    assert all(abs(a - b) < 1e-15 for a, b in zip(got, want))
    shared, _ = cake.cake_rotary_table((2, 3), 100.0, shared=True, device=DEV)
    same, _ = cake.cake_rotary_table((5,), 100.0, device=DEV)
    assert torch.equal(shared, same)
    given, _ = cake.cake_rotary_table((1, 2), freqs=[0.5, -0.25, 7.0], device=DEV)
    assert [round((t if t < 2 ** 63 else t) / 2 ** 64 * 2 * math.pi, 12) for t in given.tolist()][:2] == [0.5, -0.25]
    with pytest.raises(ValueError):
        cake.cake_rotary_table((2,), freqs=[1.0], device=DEV)
    with pytest.raises(ValueError):
        cake.cake_rotary_table((1,), freqs=[float("nan")], device=DEV)


def test_strided_positions_and_zero_angles(cake):
    g = torch.Generator().manual_seed(1)
    q = heads(g, 24, 2, 64)
    turns, axes = cake.cake_rotary_table((8, 8, 16), device=DEV)
    pos = torch.randint(0, 50, (24, 3), generator=g).to(DEV)
    y = cake.cake_rotary_fwd(q, None, pos.t(), turns, axes)[0]
    assert torch.equal(y, cake.cake_rotary_fwd(q, None, pos.t().contiguous(), turns, axes)[0])
    one = torch.tensor([3], device=DEV).expand(24)  # one position for all tokens
    y = cake.cake_rotary_fwd(q, None, one, turns)[0]
    assert torch.equal(y, cake.cake_rotary_fwd(q, None, one.contiguous(), turns)[0])
    assert torch.equal(cake.cake_rotary_fwd(q, None, torch.zeros(24, dtype=torch.int32, device=DEV), turns)[0], q)


def test_an_axis_outside_sets_the_status(cake):
    g = torch.Generator().manual_seed(1)
    q = heads(g, 4, 1, 32)
    turns, axes = cake.cake_rotary_table((8, 8), device=DEV)
    axes[3], axes[12] = 2, -1
    pos = torch.full((2, 4), 5, dtype=torch.int64, device=DEV)
    y = cake.cake_rotary_fwd(q, None, pos, turns, axes)[0]
    assert cake.cake_rmsnorm_device_status(clear=True) == 1
    for i in (3, 12):  # those pairs are not rotated
        assert torch.equal(y[..., [i, 16 + i]], q[..., [i, 16 + i]])
    assert cake.cake_rmsnorm_device_status() == 0


def test_more_tokens_than_lane_groups(cake):
    """Tokens enough that lane groups take several in turn, and offsets past 2^31 bytes."""
    g = torch.Generator(device=DEV).manual_seed(4)
    T, nq, nk, D = 70000, 12, 1, 256
    buf = torch.empty(T, nq, 2 * D, dtype=BF16, device=DEV).normal_(generator=g)
    q, k = buf[..., :D], torch.empty(T, nk, D, dtype=BF16, device=DEV).normal_(generator=g)
    w = torch.rand(D, generator=g, device=DEV) + 0.5
    turns, axes = cake.cake_rotary_table((64,), device=DEV)
    pos = torch.arange(T, device=DEV)
    y, z, rq, rk = cake.cake_rotary_fwd(q, k, pos, turns, None, w, w)
    dq, dk, dwq, dwk = cake.cake_rotary_bwd(y, z, pos, turns, None, q, k, rq, rk, w, w)
    angle = ref.phases(pos, turns, None)
    at = torch.tensor([0, 1, 9727, 9728, 34567, T - 1])
    for v, y_, rs, d in ((q, y, rq, dq), (k, z, rk, dk)):
        n = v.shape[1]
        want, allow, r64 = ref.rotary_fwd(v[at.to(DEV)], angle[at], w, 1e-6, "half")
        check("y", y_[at.to(DEV)], want, allow)
        r = rs.view(T, n)[at.to(DEV)]
        want, allow, _, _ = ref.rotary_bwd(y_[at.to(DEV)], angle[at], v[at.to(DEV)], r, w, "half")
        check("dv", d[at.to(DEV)], want, allow)
    for v, y_, rs, dw in ((q, y, rq, dwq), (k, z, rk, dwk)):
        want, allow = torch.zeros(D, dtype=torch.float64), torch.zeros(D, dtype=torch.float64)
        for a in range(0, T, 10000):
            s = slice(a, a + 10000)
            _, _, dw64, edw = ref.rotary_bwd(y_[s], angle[s], v[s], rs.view(T, -1)[s], w, "half")
            want, allow = want + dw64, allow + edw
        check("dw", dw, want, allow)


def test_autograd(cake):
    g = torch.Generator().manual_seed(6)
    T, D = 50, 64
    q, k = (heads(g, T, n, D).requires_grad_() for n in (6, 2))
    wq, wk = weights(g, D, True).requires_grad_(), weights(g, D, False).requires_grad_()
    turns, axes = cake.cake_rotary_table((8, 12, 12), device=DEV)
    pos = torch.randint(0, 99, (3, T), generator=g).to(DEV)
    dy, dz = heads(g, T, 6, D), heads(g, T, 2, D)
    y, z = cake.cake_rotary(q, k, pos, turns, axes, wq, wk)
    torch.autograd.backward((y, z), (dy, dz))
    _, _, rq, rk = cake.cake_rotary_fwd(q.detach(), k.detach(), pos, turns, axes, wq.detach(), wk.detach())
    want = cake.cake_rotary_bwd(dy, dz, pos, turns, axes, q.detach(), k.detach(), rq, rk, wq.detach(), wk.detach())
    for leaf, v in zip((q, k, wq, wk), want):
        assert leaf.grad.dtype == leaf.dtype and torch.equal(leaf.grad, v.to(leaf.dtype))
    # the keys alone reach the loss, and no norm
    y, z = cake.cake_rotary(q, k, pos, turns, axes)
    gq, gk = torch.autograd.grad(z, (q, k), dz)
    assert not bool(gq.any()) and torch.equal(gk, cake.cake_rotary_bwd(dz, None, pos, turns, axes)[0])


def test_gradients_against_differences(cake):
    """The kernels' gradients against central differences of the FP64 form, at a few places."""
    g = torch.Generator().manual_seed(8)
    T, n, D = 3, 2, 32
    v, dy, w = heads(g, T, n, D), heads(g, T, n, D), weights(g, D, True)
    turns, axes = cake.cake_rotary_table((4, 4), device=DEV)
    pos = torch.randint(0, 99, (2, T), generator=g).to(DEV)
    angle = ref.phases(pos, turns, axes)
    rstd = cake.cake_rotary_fwd(v, None, pos, turns, axes, w)[2]
    dv, _, dw, _ = cake.cake_rotary_bwd(dy, None, pos, turns, axes, v, None, rstd, None, w)

    def loss(v64, w64):
        r = 1 / torch.sqrt((v64 * v64).mean(-1, keepdim=True) + 1e-6)
        return float((ref.turn(v64 * r * w64, angle, "half")[0] * dy.double().cpu()).sum())

    v64, w64, h = v.double().cpu(), w.double().cpu(), 1e-4
    for at in ((0, 0, 0), (1, 1, 9), (2, 0, 20), (2, 1, 31)):
        e = torch.zeros_like(v64)
        e[at] = h
        want = (loss(v64 + e, w64) - loss(v64 - e, w64)) / (2 * h)
        # a BF16 rounding of the result, and the differences' own error (h^2 and cancellation)
        assert abs(float(dv[at]) - want) <= 2.0 ** -8 * abs(want) + 1e-5
    for j in (0, 13, 31):
        e = torch.zeros_like(w64)
        e[j] = h
        want = (loss(v64, w64 + e) - loss(v64, w64 - e)) / (2 * h)
        assert abs(float(dw[j]) - want) <= 1e-5 * (1 + abs(want))


def test_several_axes_with_few_lanes_and_uneven_shares(cake):
    """More axes than a row has lanes, tokens that leave the last lane groups without one, steps that no share divides."""
    g = torch.Generator().manual_seed(11)
    for T, n, D, sections, style in ((6151, 3, 32, (4, 2, 1, 1), "half"), (4099, 17, 48, (8, 8, 8), "adjacent"),
                                     (2051, 5, 16, (2, 3, 3), "half"), (997, 40, 112, (16, 8), "half")):
        q, k = heads(g, T, n, D), heads(g, T, 1, D)
        w = weights(g, D, True)
        turns, axes = cake.cake_rotary_table(sections, 100.0, device=DEV)
        pos = torch.randint(-50, 500, (len(sections), T), generator=g).to(DEV)
        angle = ref.phases(pos, turns, axes)
        y, z, rq, rk = cake.cake_rotary_fwd(q, k, pos, turns, axes, w, w, style=style)
        dq, dk, dwq, dwk = cake.cake_rotary_bwd(y, z, pos, turns, axes, q, k, rq, rk, w, w, style=style)
        for v, y_, rs, dv, dw in ((q, y, rq, dq, dwq), (k, z, rk, dk, dwk)):
            want, allow, r64 = ref.rotary_fwd(v, angle, w, 1e-6, style)
            check("y", y_, want, allow)
            want, allow, dw64, edw = ref.rotary_bwd(y_, angle, v, rs, w, style)
            check("dv", dv, want, allow)
            check("dw", dw, dw64, edw)


def test_autograd_without_keys(cake):
    g = torch.Generator().manual_seed(9)
    q, w = heads(g, 20, 3, 64).requires_grad_(), weights(g, 64, True).requires_grad_()
    turns, _ = cake.cake_rotary_table((32,), device=DEV)
    pos, dy = torch.arange(20, device=DEV), heads(g, 20, 3, 64)
    y, none = cake.cake_rotary(q, None, pos, turns, None, w)
    assert none is None
    y.backward(dy)
    rstd = cake.cake_rotary_fwd(q.detach(), None, pos, turns, None, w.detach())[2]
    dq, _, dw, _ = cake.cake_rotary_bwd(dy, None, pos, turns, None, q.detach(), None, rstd, None, w.detach())
    assert torch.equal(q.grad, dq) and torch.equal(w.grad, dw)


def test_head_major_storage(cake):
    """Heads that step past all tokens: [heads, T, D] in memory."""
    g = torch.Generator().manual_seed(10)
    q = heads(g, 5, 70, 64).transpose(0, 1)  # [70, 5, 64]
    w = weights(g, 64, True)
    turns, _ = cake.cake_rotary_table((32,), device=DEV)
    pos = torch.arange(70, device=DEV)
    want = cake.cake_rotary_fwd(q.contiguous(), None, pos, turns, None, w)
    out = torch.empty(5, 70, 64, dtype=BF16, device=DEV).transpose(0, 1)
    got = cake.cake_rotary_fwd(q, None, pos, turns, None, w, q_out=out)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    cake.cake_rotary_fwd(q, None, pos, turns, None, w, q_out=q)
    assert torch.equal(q, want[0])


def test_norm_of_zero_and_special_rows(cake):
    """A row of zeros is zero (eps), infinities and NaN stay in their row."""
    q = torch.ones(4, 2, 64, dtype=BF16, device=DEV)
    q[1] = 0
    q[2, 0, 5], q[3, 1, 7] = float("nan"), float("inf")
    w = torch.ones(64, device=DEV)
    turns, _ = cake.cake_rotary_table((32,), device=DEV)
    y, _, rstd, _ = cake.cake_rotary_fwd(q, None, torch.arange(4, device=DEV), turns, None, w)
    # 1 / sqrt(1e-6): the constant, the root and the quotient are rounded to FP32, 2.5 u in all
    assert not bool(y[1].any()) and bool(((rstd.view(4, 2)[1] / 1000 - 1).abs() <= ref.RSTD_REL).all())
    finite = torch.isfinite(y.float()).all(-1)
    assert finite.tolist() == [[True, True], [True, True], [False, True], [True, False]]


def test_no_pairs_need_no_positions(cake):
    """Through the C ABI: with pairs = 0 the rotation's pointers are not looked at."""
    import struct

    from bwd_dw_column_gb300.step import _three
    g = torch.Generator().manual_seed(12)
    q, w = heads(g, 9, 3, 32), weights(g, 32, True)
    y, rstd = torch.empty_like(q), torch.empty(27, device=DEV)
    rotation = struct.pack("=qqQQQixxxxqqixxxx", 0, 7, w.data_ptr(), w.data_ptr(), 0, 1, 5, 1, 0)
    view = lambda t: _three(t.data_ptr(), t.stride(0), t.stride(1))  # noqa: E731
    st = cake.load_library().cake_rotary_fwd(9, 3, 0, 32, view(q), None, rotation, w.data_ptr(), 1, None, 0, 1e-6, view(y),
                                             None, rstd.data_ptr(), None, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    want, allow, _ = ref.rotary_fwd(q, torch.zeros(9, 0, dtype=torch.float64), w, 1e-6, "half")
    check("y", y, want, allow)
