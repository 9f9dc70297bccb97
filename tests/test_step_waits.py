"""The bounded waits of the training-step operators, made to run out from the
host: a part of what a kernel waits for never comes (a few bytes that a stage
expects beyond its copies, a flag that nothing sets), and the limit is a few
milliseconds.  Every such kernel ends by itself, the device status reads
CAKE_ERR_TIMEOUT, and the next call is right again.  Nothing here faults or
hangs the GPU."""
import contextlib
import time

import pytest
import torch

from tests.test_step_sandwich import case, check_bwd, check_fwd

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF16 = torch.bfloat16
TIMEOUT, INVALID = 5, 1


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
    cake.cake_step_wait_test(limit_us, withhold)
    try:
        yield
    finally:
        cake.cake_step_wait_test()


def test_refusals(cake):
    for bad in ((0, 1), (1000001, 0), (100, 3), (100, -1)):
        with pytest.raises(cake.CakeError):
            cake.cake_step_wait_test(*bad)
    cake.cake_step_wait_test(1000, 2)
    cake.cake_step_wait_test()


@pytest.mark.gpu
@pytest.mark.parametrize("withhold", [1, 2])
@pytest.mark.parametrize("gate", ["none", "row", "elem"])
@pytest.mark.parametrize("T,H", [(40, 64), (2500, 256), (900, 392), (700, 2048), (600, 2560), (300, 4096), (1000, 8192)])
def test_a_sandwich_norms_stage_that_never_fills(cake, T, H, gate, withhold):
    # rows of part of a CTA's warps, of all, and over clusters of 2 and 4
    c = case(T, H, gate, device=DEV)
    _, h, r1, r2 = check_fwd(cake, c, 0.5)
    assert cake.cake_rmsnorm_device_status(clear=True) == 0
    t0 = time.perf_counter()
    try:
        with waits(cake, 2000, withhold):
            cake.cake_sandwich_fwd(c["z"], c["x"], c["w_post"], c["w_pre"], 1e-6, c["gate"], 0.5)
            torch.cuda.synchronize()
            fwd = cake.cake_rmsnorm_device_status(clear=True)
            cake.cake_sandwich_bwd(c["dy"], h, c["z"], r1, r2, c["w_post"], c["w_pre"], c["dh"], c["gate"], 0.5)
            torch.cuda.synchronize()
    finally:
        bwd = cake.cake_rmsnorm_device_status(clear=True)
    assert (fwd, bwd) == (TIMEOUT, TIMEOUT)
    assert time.perf_counter() - t0 < 2.0
    check_bwd(cake, c, 0.5, h=h, r=(r1, r2))
    assert cake.cake_rmsnorm_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("first", ["timeout", "id"])
def test_a_timeout_is_not_lost_to_an_id_outside_the_table(cake, first):
    c = case(64, 256, device=DEV)
    table = torch.randn(10, 64, device=DEV).to(BF16)
    ids = torch.tensor([3, 10, 9], device=DEV)

    def run_out():
        with waits(cake, 2000, 1):
            cake.cake_sandwich_fwd(c["z"], c["x"], c["w_post"], c["w_pre"])

    try:
        if first == "timeout":
            run_out()
        cake.cake_embedding_fwd(ids, table)
        cake.cake_embedding_bwd(torch.ones(3, 64, dtype=BF16, device=DEV), ids, 10)
        if first == "id":
            run_out()
    finally:
        status = cake.cake_rmsnorm_device_status(clear=True)
    assert status == TIMEOUT
    cake.cake_embedding_fwd(ids, table)
    assert cake.cake_rmsnorm_device_status(clear=True) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,V", [(700, 64, 5000), (8192, 256, 100_000)])
def test_a_zeroing_flag_that_nothing_sets(cake, T, H, V):
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(0, V, (T,), generator=g).to(DEV)
    dy = torch.randn(T, H, generator=g).to(BF16).to(DEV)
    want = cake.cake_embedding_bwd(dy, ids, V)
    out = torch.full((V, H), 7.0, device=DEV)
    try:
        with waits(cake, 2000, 1):
            cake.cake_embedding_bwd(dy, ids, V, out=out)
            torch.cuda.synchronize()
    finally:
        status = cake.cake_rmsnorm_device_status(clear=True)
    assert status == TIMEOUT
    has = torch.zeros(V, dtype=torch.bool, device=DEV)
    has[ids] = True
    assert torch.equal(out[has], want[has]) and bool((out[~has] == 7).all())  # the sums do not wait for the flag
    assert torch.equal(cake.cake_embedding_bwd(dy, ids, V, out=out), want)


@pytest.mark.gpu
def test_a_zeroing_cta_goes_on_or_gives_up_as_a_whole(cake):
    """A flag that a copy of the host sets at about the time at which the limit runs out: a CTA zeroes all of its 8
    rows (4 warps of 2 rows of 8 KB) or none, and no row is left without a report."""
    T, H, V, limit = 300, 1024, 16_000, 1500
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(0, V, (T,), generator=g).to(DEV)
    dy = torch.randn(T, H, generator=g).to(BF16).to(DEV)
    want = cake.cake_embedding_bwd(dy, ids, V)
    has = torch.zeros(V, dtype=torch.bool, device=DEV)
    has[ids] = True
    out = torch.empty(V, H, device=DEV)
    ws = torch.zeros(cake.cake_embedding_bwd_workspace_size(T, V, H), dtype=torch.uint8, device=DEV)
    flag, one, side = ws[8:12].view(torch.int32), torch.ones(1, dtype=torch.int32).pin_memory(), torch.cuda.Stream()
    may, calls = ~has.view(-1, 8), {"whole": 0, "none": 0, "some": 0}
    try:
        for k in range(240):
            out.fill_(7)
            torch.cuda.synchronize()
            with waits(cake, limit, 1):
                cake.cake_embedding_bwd(dy, ids, V, out=out, workspace=ws)
            until = time.perf_counter() + 1e-6 * (limit - 60 + k % 120)
            while time.perf_counter() < until:
                pass
            with torch.cuda.stream(side):
                flag.copy_(one, non_blocking=True)
            status = cake.cake_rmsnorm_device_status(clear=True)
            kept = (out == 7).all(1) & ~has
            assert torch.equal(out[~kept], want[~kept])  # a row is whole or untouched
            assert status == (TIMEOUT if bool(kept.any()) else 0)
            gave_up = kept.view(-1, 8)
            assert torch.equal(gave_up, gave_up.any(1, keepdim=True) & may)
            calls["none" if torch.equal(gave_up, may) else "some" if status else "whole"] += 1
    finally:
        cake.cake_rmsnorm_device_status(clear=True)
    assert torch.equal(cake.cake_embedding_bwd(dy, ids, V, out=out), want)
    print("\nrows zeroed:", calls)
