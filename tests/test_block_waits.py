"""The bounded waits of a block's operators, made to run out from the host: some
bytes that a stage expects never come, and the limit is a few milliseconds.
Every such kernel ends by itself, the device status reads CAKE_ERR_TIMEOUT, and
the next call is right again.  Nothing here faults or hangs the GPU."""
import contextlib
import time

import pytest
import torch

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF16 = torch.bfloat16
TIMEOUT = 5


@pytest.fixture(scope="module")
def cake():
    import __graft_entry__
    __graft_entry__.build()
    import bwd_dw_column_gb300 as cake
    yield cake
    if torch.cuda.is_available():
        assert cake.cake_rmsnorm_device_status() == 0


@contextlib.contextmanager
def waits(cake, limit_us, withhold):
    cake.cake_block_wait_test(limit_us, withhold)
    try:
        yield
    finally:
        cake.cake_block_wait_test()


def test_refusals(cake):
    for bad in ((0, 1), (1000001, 0), (100, 2), (100, -1)):
        with pytest.raises(cake.CakeError):
            cake.cake_block_wait_test(*bad)
    cake.cake_block_wait_test(1000, 1)
    cake.cake_block_wait_test()


def runs_out(cake, call):
    want = [t.clone() for t in call()]
    assert cake.cake_rmsnorm_device_status(clear=True) == 0
    t0 = time.perf_counter()
    try:
        with waits(cake, 2000, 1):
            call()
            torch.cuda.synchronize()
    finally:
        status = cake.cake_rmsnorm_device_status(clear=True)
    assert status == TIMEOUT and time.perf_counter() - t0 < 2.0
    assert all(torch.equal(a, b) for a, b in zip(call(), want))
    assert cake.cake_rmsnorm_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,F", [(1, 64, 128), (40, 2048, 640), (100, 512, 2000), (300, 64, 128), (700, 2048, 1160)])
def test_a_gated_blocks_stage_that_never_fills(cake, T, H, F):
    g = torch.Generator(device=DEV).manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF16)  # noqa: E731
    x, wg, wu, dh = r(T, H), r(F, H), r(F, H), r(T, F)
    runs_out(cake, lambda: cake.cake_gated_fwd(x, wg, wu))
    _, a, b = cake.cake_gated_fwd(x, wg, wu)
    runs_out(cake, lambda: cake.cake_gated_bwd(dh, x, a, b, wg, wu))


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(1, 64), (3000, 64), (2500, 256), (900, 2048), (700, 5120), (300, 8192)])
def test_a_norms_stage_that_never_fills(cake, T, H):
    g = torch.Generator(device=DEV).manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF16)  # noqa: E731
    x, e, dy, w = r(T, H), r(T, H), r(T, H), torch.ones(H, device=DEV)
    runs_out(cake, lambda: cake.cake_dropout_norm_fwd(x, e, w, 0.1, 1))
    _, h, rstd = cake.cake_dropout_norm_fwd(x, e, w, 0.1, 1)
    runs_out(cake, lambda: cake.cake_dropout_norm_bwd(dy, h, rstd, w, 0.1, 1, dh=e))
