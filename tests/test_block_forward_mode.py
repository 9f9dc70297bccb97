"""The gated block under forward-mode differentiation."""
import pytest
import torch
import torch.autograd.forward_ad as fwd_ad

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def cake():
    import __graft_entry__
    __graft_entry__.build()
    import bwd_dw_column_gb300 as cake
    yield cake
    if torch.cuda.is_available():
        assert cake.cake_rmsnorm_device_status() == 0


def rows(*size, seed=1):
    return torch.randn(*size, generator=torch.Generator().manual_seed(seed)).to(BF16).to(DEV or "cpu")


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("grad", [False, True])
def test_a_tangent_is_not_dropped(cake, monkeypatch, which, grad):
    """The gated block has no forward-mode derivative: a dual tensor raises, as in every other function."""
    from bwd_dw_column_gb300 import block

    def plain(x, wg, wu, act="silu", *, save=True, **kw):
        g, u = x @ wg.t(), x @ wu.t()
        return (torch.nn.functional.silu(g) * u, g, u) if save else (torch.nn.functional.silu(g) * u, None, None)

    monkeypatch.setattr(block, "cake_gated_fwd", plain)
    args = [rows(4, 16), rows(24, 16), rows(24, 16)]
    assert cake.cake_gated(*args).shape == (4, 24)
    with fwd_ad.dual_level(), torch.set_grad_enabled(grad):
        args[which] = fwd_ad.make_dual(args[which], torch.ones_like(args[which]))
        with pytest.raises(NotImplementedError):
            cake.cake_gated(*args)


@pytest.mark.gpu
def test_forward_mode_of_the_kernels(cake):
    args = [rows(4, 16), rows(24, 16), rows(24, 16)]
    want = cake.cake_gated(*args)
    with fwd_ad.dual_level():
        assert torch.equal(cake.cake_gated(*args), want)  # tensors without a tangent are as outside
        with pytest.raises(NotImplementedError):
            cake.cake_gated(fwd_ad.make_dual(args[0], args[0]), *args[1:])
    with pytest.raises(RuntimeError):  # torch's own refusal of a function without setup_context
        torch.func.jvp(lambda x: cake.cake_gated(x, *args[1:]), (args[0],), (args[0],))
