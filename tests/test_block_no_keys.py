"""Keys without heads, [T, 0, D]: nothing of theirs to turn, and a weight's gradient of zero."""
import pytest
import torch

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF16 = torch.bfloat16
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cake():
    import __graft_entry__
    __graft_entry__.build()
    import bwd_dw_column_gb300 as cake
    yield cake
    assert cake.cake_rmsnorm_device_status() == 0


@pytest.mark.parametrize("T", [0, 1, 50])
def test_their_weights_gradient_is_zero(cake, T):
    D = 64
    gen = torch.Generator().manual_seed(T)
    q, dq = (torch.randn(T, 3, D, generator=gen).to(BF16).to(DEV) for _ in range(2))
    k, pos = torch.empty(T, 0, D, dtype=BF16, device=DEV), torch.arange(T, device=DEV)
    w = (1 + 0.1 * torch.randn(D, generator=gen)).to(DEV)
    turns, _ = cake.cake_rotary_table((32,), device=DEV)
    y, z, rq, rk = cake.cake_rotary_fwd(q, k, pos, turns, None, w, w)
    assert z.shape == k.shape and rk.numel() == 0
    want = cake.cake_rotary_bwd(dq, None, pos, turns, None, q, None, rq, None, w)
    given = torch.full((D,), 7.0, device=DEV)
    for kw in ({"dw_k": given}, {}):
        torch.full((64, D), 7.0, device=DEV)  # what a fresh tensor may find in its memory
        dv, dz, dwq, dwk = cake.cake_rotary_bwd(dq, k, pos, turns, None, q, k, rq, rk, w, w, **kw)
        assert torch.equal(dv, want[0]) and torch.equal(dwq, want[2]) and dz.shape == k.shape
        assert dwk.shape == (D,) and not bool(dwk.any())
    wk = w.clone().requires_grad_()
    q = q.requires_grad_()
    cake.cake_rotary(q, k, pos, turns, None, w, wk)[0].backward(dq)
    assert torch.equal(q.grad, want[0]) and not bool(wk.grad.any())
    if T:  # what is written shares no memory with what is read
        with pytest.raises(cake.CakeError):
            cake.cake_rotary_bwd(dq, k, pos, turns, None, q.detach(), k, rq, rk, w, w, dw_k=w)
