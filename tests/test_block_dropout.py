"""Dropout from a counter-based generator, alone, with a residual addition and
with the norm after it, against FP64 on a GB300."""
import pytest
import torch

from tests import block_reference as ref

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF16, F32 = torch.bfloat16, torch.float32
SEED, OFFSET = 0x1234567890ABCDEF, 0xFEDCBA9876543210


@pytest.fixture(scope="module")
def cake():
    import __graft_entry__
    __graft_entry__.build()
    import bwd_dw_column_gb300 as cake
    yield cake
    assert cake.cake_rmsnorm_device_status() == 0


def rows(g, size, pad=0, std=1.0):
    return (torch.randn(*size[:-1], size[-1] + pad, generator=g) * std).to(BF16).to(DEV)[..., :size[-1]]


def check(name, got, want, allow):
    share = ref.excess(got.reshape(want.shape), want, allow)
    assert share <= 1, f"{name}: {share:.3g} of its bound"


def test_the_generator_is_the_published_one():
    """Known answers of Philox4x32-10 (counter and key all zero, all ones, and digits of pi)."""
    ones = 2 ** 32 - 1
    assert ref.philox((0,) * 4, (0, 0)) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    assert ref.philox((ones,) * 4, (ones,) * 2) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]
    assert ref.philox((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0)) == \
        [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]


def test_the_plain_form_lays_the_bits_out_as_documented():
    m = ref.kept(3, 16, 0.3, SEED, OFFSET)
    cut = round(0.3 * 65536)
    words = [0x90ABCDEF, 0x12345678, 0x76543210, 0xFEDCBA98]
    for b in range(6):
        block = ref.philox((b, 0, words[2], words[3]), (words[0], words[1]))
        bits = sum(w << (32 * i) for i, w in enumerate(block))
        for j in range(8):
            assert (float(m.view(-1)[8 * b + j]) > 0) == ((bits >> (16 * j)) % 65536 >= cut)


@pytest.mark.gpu
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.99999, 1.0])
@pytest.mark.parametrize("size,pad", [((1, 8), 0), ((1, 2048), 0), ((7, 72), 8), ((129, 1032), 0), ((33, 8192), 64),
                                      ((5, 3, 256), 256), ((4097, 40), 0)])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout(cake, size, pad, residual, p):
    g = torch.Generator().manual_seed(len(size) + size[-1])
    x, e = rows(g, size, pad), rows(g, size, 0) if residual else None
    n = x.numel() // size[-1]
    m = ref.kept(n, size[-1], p, SEED, OFFSET)
    y = cake.cake_dropout_fwd(x, p, SEED, OFFSET, e)
    want, err = ref.dropout_sum(x, m, e)
    check("y", y, want, ref.rounded(want, err))
    if not residual:
        assert torch.equal(y.cpu().reshape(m.shape) == 0, (m == 0) | (x.cpu().reshape(m.shape) == 0))
        assert torch.equal(cake.cake_dropout_bwd(x, p, SEED, OFFSET), y)
    else:  # in place over either
        for k in (0, 1):
            a = [x.clone(), e.clone()]
            assert torch.equal(cake.cake_dropout_fwd(a[0], p, SEED, OFFSET, a[1], y=a[k]), y)


@pytest.mark.gpu
def test_dropped_elements_take_no_part(cake):
    """A dropped infinity or NaN adds nothing."""
    H = 64
    m = ref.kept(4, H, 0.5, 3, 0) > 0
    x = torch.where(m, torch.ones(4, H), torch.full((4, H), float("nan"))).to(BF16).to(DEV)
    x[0, :8] = torch.where(m[0, :8], 1.0, float("inf")).to(BF16).to(DEV)
    y = cake.cake_dropout_fwd(x, 0.5, 3, 0, torch.ones(4, H, dtype=BF16, device=DEV)).cpu()
    assert torch.equal(y, torch.where(m, 3.0, 1.0).to(BF16))
    y, h, rstd = cake.cake_dropout_norm_fwd(x, torch.ones(4, H, dtype=BF16, device=DEV), torch.ones(H, device=DEV), 0.5,
                                            3)
    assert torch.equal(h.cpu(), torch.where(m, 3.0, 1.0).to(BF16)) and bool(torch.isfinite(y).all())


SHAPES = [((1, 8), 0), ((59, 8), 0), ((203, 24), 8), ((131, 40), 0), ((1, 64), 0), ((77, 120), 0), ((65, 128), 0),
          ((1, 2048), 0), ((37, 72), 8), ((129, 264), 0), ((300, 1032), 0), ((64, 1536), 16),
          ((257, 2048), 0), ((90, 2560), 0), ((45, 4096), 0), ((33, 5128), 8), ((31, 6144), 0), ((13, 6152), 0),
          ((17, 8192), 0), ((9, 3, 256), 256), ((4097, 64), 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("w32", [False, True])
@pytest.mark.parametrize("size,pad", SHAPES)
def test_dropout_norm_fwd(cake, size, pad, w32):
    g = torch.Generator().manual_seed(size[-1])
    H, eps, p = size[-1], 1e-6, 0.2
    x, e = rows(g, size, pad, 0.7), rows(g, size, 0, 1.5)
    w = (1 + 0.1 * torch.randn(H, generator=g)).to(F32 if w32 else BF16).to(DEV)
    n = x.numel() // H
    m = ref.kept(n, H, p, SEED, OFFSET)
    y, h, rstd = cake.cake_dropout_norm_fwd(x, e, w, p, SEED, OFFSET, eps)
    want, err = ref.dropout_sum(x, m, e)
    check("h", h, want, ref.rounded(want, err))
    hd = h.double().cpu().reshape(n, H)
    r64 = 1 / torch.sqrt((hd * hd).mean(1) + eps)
    check("rstd", rstd, r64, ref.RSTD_REL * r64)
    y64 = hd * r64[:, None] * w.double().cpu()
    check("y", y, y64, ref.rounded(y64, y64.abs() * (ref.RSTD_REL + 3 * ref.U)))
    # in place: the residual stream in its own memory, the block's input in the block's output's
    a, b = x.clone(), e.clone()
    y2, h2, r2 = cake.cake_dropout_norm_fwd(a, b, w, p, SEED, OFFSET, eps, y=a, h_new=b)
    assert torch.equal(y2, y) and torch.equal(h2, h) and torch.equal(r2, rstd)


@pytest.mark.gpu
@pytest.mark.parametrize("with_dh", [False, True])
@pytest.mark.parametrize("size,pad", SHAPES)
def test_dropout_norm_bwd(cake, size, pad, with_dh):
    g = torch.Generator().manual_seed(size[-1] + 1)
    H, p = size[-1], 0.3
    h, dy = rows(g, size, 0, 1.7), rows(g, size, pad)
    dh = rows(g, size, 0) if with_dh else None
    w = (1 + 0.1 * torch.randn(H, generator=g)).to(F32 if with_dh else BF16).to(DEV)
    n = h.numel() // H
    rstd = (1 / torch.sqrt((h.float() ** 2).mean(-1) + 1e-6)).reshape(-1)
    m = ref.kept(n, H, p, SEED, OFFSET)
    got = cake.cake_dropout_norm_bwd(dy, h, rstd, w, p, SEED, OFFSET, dh)
    want = ref.dropout_norm_bwd(dy, h, rstd, w, dh, m)
    for name, v in zip(("dresidual", "dx", "dw"), got):
        check(name, v, *want[name])
    again = cake.cake_dropout_norm_bwd(dy, h, rstd, w, p, SEED, OFFSET, dh)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.gpu
def test_more_rows_than_one_turn(cake):
    """Rows enough that every CTA goes round its ring several times, of each kind of width."""
    for T, H in ((20000, 128), (5000, 1536), (1500, 6144)):
        g = torch.Generator(device=DEV).manual_seed(H)
        x, e, dy = (torch.randn(T, H, generator=g, device=DEV).to(BF16) for _ in range(3))
        w = torch.rand(H, generator=g, device=DEV) + 0.5
        m = ref.kept(T, H, 0.25, 5, 6)
        y, h, rstd = cake.cake_dropout_norm_fwd(x, e, w, 0.25, 5, 6)
        want, err = ref.dropout_sum(x, m, e)
        check("h", h, want, ref.rounded(want, err))
        got = cake.cake_dropout_norm_bwd(dy, h, rstd, w, 0.25, 5, 6, e)
        want = ref.dropout_norm_bwd(dy, h, rstd, w, e, m)
        for name, v in zip(("dresidual", "dx", "dw"), got):
            check(name, v, *want[name])


@pytest.mark.gpu
def test_random_numbers_from_the_device(cake):
    """The seed and an offset in memory give the bits of the same numbers on the host, and a replay reads them anew."""
    x = torch.ones(64, 256, dtype=BF16, device=DEV)
    rng = torch.tensor([17, 5], dtype=torch.int64, device=DEV)
    assert torch.equal(cake.cake_dropout_fwd(x, 0.5, rng, 3), cake.cake_dropout_fwd(x, 0.5, 17, 8))
    assert torch.equal(cake.cake_dropout_fwd(x, 0.5, -1, -2), cake.cake_dropout_fwd(x, 0.5, 2 ** 64 - 1, 2 ** 64 - 2))
    y = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cake.cake_dropout_fwd(x, 0.5, rng, 3, y=y)
    for k in (5, 6):
        rng[1] = k
        graph.replay()
        assert torch.equal(y, cake.cake_dropout_fwd(x, 0.5, 17, 3 + k))


@pytest.mark.gpu
def test_offsets_past_31_bits(cake):
    """Rows whose elements lie past 2^31, and their random numbers."""
    T, H = 270000, 8192
    free, _ = torch.cuda.mem_get_info()
    if free < 20 << 30:
        pytest.skip("needs 20 GB of device memory")
    x = torch.zeros(T, H, dtype=BF16, device=DEV)
    x[-3:] = 1
    y = cake.cake_dropout_fwd(x, 0.5, 9)
    low = 2 ** 32 - 1
    for t in (T - 3, T - 1):
        for b in (0, 17, H // 8 - 1):
            e = t * (H // 8) + b
            bits = sum(w << (32 * i) for i, w in enumerate(ref.philox((e & low, e >> 32, 0, 0), (9, 0))))
            want = [2.0 if (bits >> (16 * j)) % 65536 >= 32768 else 0.0 for j in range(8)]
            assert y[t, 8 * b:8 * b + 8].tolist() == want
    assert not bool(y[:-3].any())


@pytest.mark.gpu
def test_the_share_that_is_kept(cake):
    """Of 2^24 elements the share that is dropped is p within six standard deviations, in each of the 8 places."""
    x = torch.ones(2 ** 14, 1024, dtype=BF16, device=DEV)
    for p in (0.1, 0.5):
        d = (cake.cake_dropout_fwd(x, p, 12345) == 0).view(-1, 8).double().mean(0)
        assert float((d - p).abs().max()) < 6 * (p * (1 - p) / 2 ** 21) ** 0.5 + 2.0 ** -16


@pytest.mark.gpu
def test_autograd(cake):
    g = torch.Generator().manual_seed(3)
    x, e = (rows(g, (40, 320)).requires_grad_() for _ in range(2))
    w = (1 + 0.1 * torch.randn(320, generator=g)).to(BF16).to(DEV).requires_grad_()
    y, h = cake.cake_dropout_norm(x, e, w, 0.2, 7, 1)
    z = cake.cake_dropout(y, 0.4, 7, 2, residual=h)
    dz = rows(g, (40, 320))
    z.backward(dz)
    y2, h2, rstd = cake.cake_dropout_norm_fwd(x.detach(), e.detach(), w.detach(), 0.2, 7, 1)
    dres, dx, dw = cake.cake_dropout_norm_bwd(cake.cake_dropout_bwd(dz, 0.4, 7, 2), h2, rstd, w.detach(), 0.2, 7, 1, dz)
    assert torch.equal(x.grad, dx) and torch.equal(e.grad, dres) and torch.equal(w.grad, dw.to(BF16))
    assert torch.equal(z.detach(), cake.cake_dropout_fwd(y2, 0.4, 7, 2, h2))
    # only h's gradient, only x's
    y, h = cake.cake_dropout_norm(x, e.detach(), w, 0.2, 7, 1)
    gx, = torch.autograd.grad(h, x, dz)
    assert torch.equal(gx, cake.cake_dropout_bwd(dz, 0.2, 7, 1))


def test_every_width_has_a_plan_that_fits():
    """For every width: a row's warps hold it, the ring has two stages, all of it fits an SM's shared memory, the
    groups' column sums fit the ring, the barriers and reduction slots the space before it."""
    import ctypes

    import __graft_entry__
    __graft_entry__.build()
    import bwd_dw_column_gb300 as cake
    from bwd_dw_column_gb300.step import _three
    lib, got = cake.load_library(), (ctypes.c_int64 * 9)()
    for H in range(8, 8193, 8):
        for backward, tensors in ((0, 2), (1, 2), (1, 3)):
            for T in (1, 1000, 2 ** 31 - 1):
                assert lib.cake_dropout_norm_plan(_three(T, 1, H), tensors, backward, got) == 0
                vpt, lanes, W, groups, stages, ctas, per_cta, lo, smem = got
                assert 1 <= vpt <= (3 if backward else 2) and 1 <= groups * W <= 16 and 8 * lanes * vpt * W >= H
                assert lanes == 32 or (W == 1 and vpt == 1)
                rows = groups * (32 // lanes)
                assert W == 1 or groups <= 14
                fixed = 1024 + (4 * H + 1023) // 1024 * 1024 + lo
                ring = smem - fixed
                assert 2 <= stages <= 16 and ring >= stages * tensors * rows * H * 2 and smem <= 227 * 1024
                assert groups * 2 * W * 4 <= 400
                if backward:  # a float4 of a pair of columns, of each group; and of each of a thread's pairs
                    assert ring >= rows * H * 8 and lo >= vpt * 4 * 16 * groups * W * 32
                assert (ctas - 1) * per_cta < T <= ctas * per_cta
