"""The backward of dropout with the norm for rows far from one: with eps = 0, which
is accepted, a row's rstd may be any finite FP32 number."""
import pytest
import torch

from tests import block_reference as ref

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


@pytest.mark.parametrize("T,H", [(5, 32), (9, 64), (7, 128), (6, 512), (40, 2048), (11, 6144)])
@pytest.mark.parametrize("with_dh", [False, True])
def test_rows_of_any_size(cake, T, H, with_dh):
    gen = torch.Generator().manual_seed(H)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    # rows of 1e-21 to 1e15: rstd of 1e21 to 1e-15, whose square is beyond FP32 at the small end
    scale = torch.logspace(-21, 15, T).unsqueeze(1)
    e = (r(T, H) * scale).to(BF16).to(DEV)
    dy, w = r(T, H).to(BF16).to(DEV), (1 + 0.1 * r(H)).to(DEV)
    dh = r(T, H).to(BF16).to(DEV) if with_dh else None
    m = ref.kept(T, H, 0.2, 5, 6)
    _, h, rstd = cake.cake_dropout_norm_fwd(torch.zeros_like(e), e, w, 0.2, 5, 6, 0.0)
    assert torch.equal(h, e) and bool(torch.isfinite(rstd).all()) and float(rstd.max()) > 2.0 ** 64
    want = ref.dropout_norm_bwd(dy, h, rstd, w, dh, m)
    for name, v in zip(("dresidual", "dx", "dw"), cake.cake_dropout_norm_bwd(dy, h, rstd, w, 0.2, 5, 6, dh)):
        assert ref.excess(v.reshape(want[name][0].shape), *want[name]) <= 1, name
