"""Gradients of the gated block where an input or a weight is infinite or NaN: of
few tokens, whose gradients go into the products in two parts, as of many."""
import pytest
import torch

from tests import block_reference as ref

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF16 = torch.bfloat16
INF, NAN = float("inf"), float("nan")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cake():
    import __graft_entry__
    __graft_entry__.build()
    import bwd_dw_column_gb300 as cake
    yield cake
    assert cake.cake_rmsnorm_device_status() == 0


def same(name, got, want, allow):
    """Infinite and NaN where the FP64 form is, within the bound elsewhere."""
    got, want, allow = got.double().cpu(), want.cpu(), allow.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{name}: NaN"
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], want[inf]), f"{name}: infinities"
    fin = torch.isfinite(want)
    assert bool(fin.any()) and bool(((got - want).abs()[fin] <= allow[fin]).all()), name


# 64 tokens and fewer: two parts; 300 tokens: one.  Sums over F of one tile and of split ones.
@pytest.mark.parametrize("T,H,F", [(1, 64, 1000), (2, 72, 136), (33, 264, 520), (64, 64, 4096), (64, 1024, 264),
                                   (65, 72, 136), (300, 136, 264)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_an_infinite_factor_gives_infinities(cake, T, H, F, act):
    gen = torch.Generator(device=DEV).manual_seed(T + H)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(BF16)  # noqa: E731
    x, wg, wu, g, u, dh = r(T, H), r(F, H) * 0.1, r(F, H) * 0.1, r(T, F), r(T, F), r(T, F)
    dh[:, 3] = 0  # and a gradient of zero: 0 times an infinity is NaN
    x[0, 1], x[T - 1, 2], x[T // 2, 5] = INF, -INF, NAN
    wg[7, 9], wu[F - 1, 10], wg[2, 11], wu[0, 13] = INF, -INF, NAN, INF
    wg[5, 13] = INF  # two infinite terms in one sum
    want = ref.gated_bwd(dh, x, g, u, wg, wu, act)
    got = cake.cake_gated_bwd(dh, x, g, u, wg, wu, act)
    for name, v in zip(("dx", "dw_gate", "dw_up"), got):
        same(name, v, *want[name])
    only = cake.cake_gated_bwd(dh, x, g, u, wg, wu, act, need_dx=False)[1:] + \
        cake.cake_gated_bwd(dh, x, g, u, wg, wu, act, need_dw=False)[:1]
    for a, b in zip(only, got[1:] + got[:1]):
        assert torch.equal(torch.nan_to_num(a.float(), 0, 1, 2), torch.nan_to_num(b.float(), 0, 1, 2))
        assert torch.equal(torch.isnan(a), torch.isnan(b))
