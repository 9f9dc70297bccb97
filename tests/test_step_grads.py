"""The global gradient norm and clipping against FP64: mixed types, odd sizes
and alignments, many tensors, values at the ends of the range, not-a-numbers,
in place and into other buffers."""
import math

import pytest
import torch

from tests import step_reference as ref

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF16, F32 = torch.bfloat16, torch.float32
# the FP32 sum of 32 squares: chains of 8 products and 2 additions; the root halves it, and norm is rounded once
NORM_REL = 6 * ref.U
# coef: half of the sum's error, its own rounding; the product rounds once more
SCALE_REL = 8 * ref.U


@pytest.fixture(scope="module")
def cake():
    import __graft_entry__
    __graft_entry__.build()
    import bwd_dw_column_gb300 as cake
    yield cake


def make(sizes, types=(BF16, F32), std=1.0, seed=0, device=None):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n if isinstance(n, tuple) else (n,), generator=g) * std).to(types[i % len(types)]).to(device)
            for i, n in enumerate(sizes)]


def check_norm(cake, grads):
    got = cake.cake_grad_norm(grads)
    assert got.shape == () and got.dtype == F32
    want = ref.grad_norm([g for g in grads if g is not None])
    assert abs(float(got) - want) <= NORM_REL * want, (float(got), want)
    return want


def check_scaled(out, grad, coef):
    want = grad.double() * coef
    if out.dtype == BF16:
        allow = want.abs() * (ref.HALF_BF16 + SCALE_REL) + ref.TINY / 2
    else:
        allow = want.abs() * SCALE_REL + 2.0 ** -150
    assert ref.excess(out, want, allow) <= 1


SIZES = {"one": [1], "tiny": [1, 2, 3, 5, 7, 0, 11], "edge": [8191, 8192, 8193, 16384, 4096, 255, 256, 257],
         "shapes": [(3, 5, 7), (640, 640), (2048,), (1, 1), (0, 4)], "big": [1_300_003, 5, 700_001]}


@pytest.mark.gpu
@pytest.mark.parametrize("types", [(BF16,), (F32,), (BF16, F32)], ids=["bf16", "fp32", "mixed"])
@pytest.mark.parametrize("sizes", list(SIZES))
def test_norm_and_clipping(cake, sizes, types):
    grads = make(SIZES[sizes], types, 0.5, device=DEV)
    norm = check_norm(cake, grads)
    for max_norm in (norm * 0.37, norm * 2):
        coef = min(1.0, max_norm / (norm + 1e-6))
        for out_types in ((BF16,), (F32,), None):
            before = [g.clone() for g in grads]
            out = None if out_types is None else [torch.full(g.shape, 3.0, dtype=out_types[0], device=DEV)
                                                  for g in grads]
            mine = [g.clone() for g in grads]
            got = cake.cake_clip_grad_norm(mine, max_norm, out=out)
            torch.cuda.synchronize()
            assert abs(float(got) - norm) <= NORM_REL * norm
            for g, b, m, o in zip(grads, before, mine, out or mine):
                assert torch.equal(g, b) and (out is None or torch.equal(m, b))  # inputs stay where outputs are given
                check_scaled(o, b, coef)
            if out is None and max_norm > norm:
                for b, m in zip(before, mine):
                    assert torch.equal(b, m)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shift,oshift", [(1, 1), (1, 0), (0, 3), (4, 4), (2, 6)])
def test_any_alignment(cake, dtype, shift, oshift):
    base = make([50_000], (dtype,), device=DEV)[0]
    g = base[shift:shift + 40_001]
    check_norm(cake, [g])
    buf = torch.full((50_000,), 3.0, dtype=dtype, device=DEV)
    o = buf[oshift:oshift + 40_001]
    cake.cake_clip_grad_norm([g], 1.0, out=[o])
    torch.cuda.synchronize()
    check_scaled(o, g, 1.0 / (ref.grad_norm([g]) + 1e-6))
    assert bool((buf[:oshift] == 3).all()) and bool((buf[oshift + 40_001:] == 3).all())
    before = base.clone()
    cake.cake_clip_grad_norm([g], 1.0)  # in place
    torch.cuda.synchronize()
    assert torch.equal(g, o) and torch.equal(base[:shift], before[:shift])
    assert torch.equal(base[shift + 40_001:], before[shift + 40_001:])


@pytest.mark.gpu
@pytest.mark.parametrize("n", [31, 32, 33, 999, 1000, 1001, 2500])
def test_many_tensors(cake, n):
    grads = make([(i * 37) % 501 for i in range(n)], device=DEV, seed=n)
    norm = check_norm(cake, grads)
    before = [g.clone() for g in grads]
    cake.cake_clip_grad_norm(grads, norm / 3)
    torch.cuda.synchronize()
    coef = (norm / 3) / (norm + 1e-6)
    check_scaled(torch.cat([g for g in grads if g.dtype == BF16]), torch.cat([g for g in before if g.dtype == BF16]), coef)
    check_scaled(torch.cat([g for g in grads if g.dtype == F32]), torch.cat([g for g in before if g.dtype == F32]), coef)


@pytest.mark.gpu
@pytest.mark.parametrize("std", [1e-38, 1e-30, 1e-22, 1e-10, 1e10, 1e19, 1e30])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_the_whole_range(cake, std, dtype):
    # squares that FP32 cannot hold, alone and next to ordinary ones
    grads = make([10_000, 33], (dtype,), std, device=DEV)
    check_norm(cake, grads)
    check_norm(cake, grads + make([5000], (F32,), 1.0, seed=1, device=DEV))
    grads[0][1::2] = 0
    check_norm(cake, grads)
    norm = ref.grad_norm(grads)
    before = [g.clone() for g in grads]
    cake.cake_clip_grad_norm(grads, norm / 8, eps=0.0)
    torch.cuda.synchronize()
    for g, b in zip(grads, before):
        check_scaled(g, b, 0.125)


@pytest.mark.gpu
def test_zeros_and_not_finite(cake):
    z = make([5000, 3], device=DEV)
    for t in z:
        t.zero_()
    assert float(cake.cake_grad_norm(z)) == 0.0
    assert float(cake.cake_clip_grad_norm(z, 1.0)) == 0.0 and not any(t.any() for t in z)
    cake.cake_clip_grad_norm(z, 0.0, eps=0.0)  # nothing to scale, and no 0 / 0
    assert not any(t.any() for t in z)
    g = make([9000, 100], device=DEV)
    g[0][8500] = float("inf")
    assert float(cake.cake_grad_norm(g)) == math.inf
    cake.cake_clip_grad_norm(g, 1.0)  # coef 0: finite values vanish, infinity * 0 is NaN
    assert bool(torch.isnan(g[0][8500])) and not g[1].any() and not g[0][:8500].any()
    g = make([9000, 100], device=DEV)
    g[1][7] = float("nan")
    assert math.isnan(float(cake.cake_grad_norm(g)))
    assert math.isnan(float(cake.cake_clip_grad_norm(g, 1.0)))
    assert all(bool(torch.isnan(t).all()) for t in g)


@pytest.mark.gpu
def test_limits_of_max_norm(cake):
    g = make([1000, 20], device=DEV)
    before = [t.clone() for t in g]
    cake.cake_clip_grad_norm(g, math.inf)
    assert all(torch.equal(a, b) for a, b in zip(g, before))
    cake.cake_clip_grad_norm(g, 0.0)
    assert not any(t.any() for t in g)
    with pytest.raises(cake.CakeError):
        cake.cake_clip_grad_norm(before, -1.0)


@pytest.mark.gpu
def test_lists_and_layouts(cake):
    a = make([(30, 40)], (F32,), device=DEV)[0]
    check_norm(cake, [a, None, a])                    # read twice: counted twice
    check_norm(cake, [a.t()])                         # dense in another order
    b = a.t().clone(memory_format=torch.preserve_format)
    assert not b.is_contiguous()
    o = torch.empty_like(b)
    norm = cake.cake_clip_grad_norm([None, b], 1.0, out=[None, o])
    check_scaled(o, b, 1.0 / (float(norm) + 1e-6))
    assert float(cake.cake_grad_norm(a)) == float(cake.cake_grad_norm([a]))
    kept = torch.empty(1, device=DEV)
    assert cake.cake_grad_norm([], norm=kept) is kept and float(kept) == 0.0
    for bad in (lambda: cake.cake_grad_norm([]), lambda: cake.cake_grad_norm([a[:, ::2]]),
                lambda: cake.cake_grad_norm([a[:, :5]]), lambda: cake.cake_clip_grad_norm([a], 1.0, out=[a, a]),
                lambda: cake.cake_clip_grad_norm([b], 1.0, out=[b.contiguous()]),
                lambda: cake.cake_grad_norm([a, a.cpu()]), lambda: cake.cake_clip_grad_norm([a], 1.0, out=[None])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        cake.cake_grad_norm([a.half()])
    with pytest.raises(cake.CakeError):
        cake.cake_clip_grad_norm([a, a], 1.0)
    with pytest.raises(cake.CakeError):
        cake.cake_clip_grad_norm([a, a[3:5]], 1.0)


@pytest.mark.gpu
def test_the_same_bits_every_time_and_in_a_graph(cake):
    grads = make([100_003, 77, 4096, (300, 500)], device=DEV)
    out = [torch.empty_like(g) for g in grads]
    norm = cake.cake_clip_grad_norm(grads, 1.0, out=out)
    want = [norm.clone()] + [o.clone() for o in out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = cake.cake_clip_grad_norm(grads, 1.0, out=out)
    for _ in range(3):
        norm.zero_()
        for o in out:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip([norm] + out, want):
            assert torch.equal(a, b)
    for g in grads:
        g.mul_(2)  # a replay reads the gradients as they are then
    graph.replay()
    torch.cuda.synchronize()
    assert float(norm) == 2 * float(want[0])


@pytest.mark.gpu
def test_more_than_2_to_31_values(cake):
    n = (1 << 31) + 5
    g = torch.zeros(n, dtype=BF16, device=DEV)
    g[-1], g[0], g[1 << 31] = 3.0, 4.0, 12.0
    assert float(cake.cake_grad_norm([g])) == 13.0
    cake.cake_clip_grad_norm([g], 6.5, eps=0.0)
    torch.cuda.synchronize()
    assert [float(g[i]) for i in (0, 1 << 31, n - 1, 1, n - 2)] == [2.0, 6.0, 1.5, 0.0, 0.0]


@pytest.mark.gpu
def test_one_workspace_and_given_norms(cake):
    """Calls of one launch, of many tensors and of several launches, in one workspace that holds garbage."""
    lists = [make([5, 70], device=DEV), make([100_003, 77], device=DEV), make([64 + i % 300 for i in range(2100)],
                                                                              device=DEV)]
    want = [float(cake.cake_grad_norm(g)) for g in lists]
    ws = torch.full((cake.cake_grad_norm_workspace_size(2100),), 0xff, dtype=torch.uint8, device=DEV)
    norms = torch.full((3, 1), 7.0, device=DEV)
    for clip in (False, True):
        for _ in range(3):
            for g, n in zip(lists, norms):
                outs = [torch.empty_like(t) for t in g]
                got = (cake.cake_clip_grad_norm(g, 0.5, out=outs, norm=n, workspace=ws) if clip else
                       cake.cake_grad_norm(g, norm=n, workspace=ws))
                assert got is n
            assert norms.flatten().tolist() == want
    with pytest.raises(cake.CakeError):
        cake.cake_grad_norm(lists[2], workspace=ws[:64])
    with pytest.raises(ValueError):
        cake.cake_grad_norm(lists[0], norm=torch.zeros(2, device=DEV))
    with pytest.raises(ValueError):
        cake.cake_grad_norm(lists[0], norm=torch.zeros(1, dtype=torch.float64, device=DEV))
    with pytest.raises(cake.CakeError):  # the norm in a gradient
        cake.cake_grad_norm(lists[1], norm=lists[1][1][4:5])
