"""The gated block of few tokens where a wait runs out although the copying warp had
none to make: every block of k fits the ring, one stage never fills, and the
stages behind it land.  The kernel waits for those copies before it leaves."""
import pytest
import torch

from tests.test_block_waits import runs_out

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def cake():
    import __graft_entry__
    __graft_entry__.build()
    import bwd_dw_column_gb300 as cake
    yield cake
    assert cake.cake_rmsnorm_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,F", [(1, 128, 128), (1, 192, 2000), (16, 1024, 640), (40, 256, 128), (128, 192, 264)])
@pytest.mark.parametrize("save", [False, True])
def test_stages_that_land_behind_one_that_never_fills(cake, T, H, F, save):
    g = torch.Generator(device=DEV).manual_seed(T + H)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF16)  # noqa: E731
    x, wg, wu = r(T, H), r(F, H), r(F, H)
    for _ in range(3):
        runs_out(cake, lambda: [t for t in cake.cake_gated_fwd(x, wg, wu, save=save) if t is not None])
