"""Dropout with the norm from a seed in device memory, as a captured training step
has it: the bits of the same numbers on the host, in every form of the kernels;
and the norm's forms at both ends of p."""
import pytest
import torch

from tests import block_reference as ref

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF16 = torch.bfloat16
pytestmark = pytest.mark.gpu

# 4, 8, 16 lanes a row; a row of 1, 2 and (backward) 3 vectors a thread, of one warp and of several
SIZES = [(59, 32), (77, 64), (65, 128), (130, 256), (40, 520), (33, 1536), (45, 4096), (31, 6144), (17, 8192)]


@pytest.fixture(scope="module")
def cake():
    import __graft_entry__
    __graft_entry__.build()
    import bwd_dw_column_gb300 as cake
    yield cake
    assert cake.cake_rmsnorm_device_status() == 0


def rows(g, *size, pad=0):
    return torch.randn(*size[:-1], size[-1] + pad, generator=g).to(BF16).to(DEV)[..., :size[-1]]


@pytest.mark.parametrize("T,H", SIZES)
def test_device_numbers_give_the_hosts_bits(cake, T, H):
    g = torch.Generator().manual_seed(H)
    x, e, dy, dh = rows(g, T, H, pad=8), rows(g, T, H), rows(g, T, H), rows(g, T, H)
    w = (1 + 0.1 * torch.randn(H, generator=g)).to(DEV)
    for seed, k, offset in ((17, 5, 3), (-2 ** 62 + 9, -1, 2 ** 63 + 4)):
        rng = torch.tensor([seed, k], dtype=torch.int64, device=DEV)
        want = cake.cake_dropout_norm_fwd(x, e, w, 0.3, seed, offset + k)
        got = cake.cake_dropout_norm_fwd(x, e, w, 0.3, rng, offset)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        _, h, rstd = want
        for d in (None, dh):
            want = cake.cake_dropout_norm_bwd(dy, h, rstd, w, 0.3, seed, offset + k, d)
            got = cake.cake_dropout_norm_bwd(dy, h, rstd, w, 0.3, rng, offset, d)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        for res in (None, e):  # alone: equally spaced rows, and rows of unlike spacing
            for v in (x, x[:, :H // 2 // 8 * 8], rows(g, T, 3, H, pad=8)[:, :2]):
                r = None if res is None else torch.ones(v.shape, dtype=BF16, device=DEV)
                assert torch.equal(cake.cake_dropout_fwd(v, 0.3, rng, offset, r),
                                   cake.cake_dropout_fwd(v, 0.3, seed, offset + k, r))


@pytest.mark.parametrize("p", [0.0, 1.0, 2.0 ** -17, 1 - 2.0 ** -18])
@pytest.mark.parametrize("T,H", SIZES)
def test_nothing_or_everything_dropped(cake, T, H, p):
    g = torch.Generator().manual_seed(H + 1)
    x, e, dy, dh = (rows(g, T, H) for _ in range(4))
    w = (1 + 0.1 * torch.randn(H, generator=g)).to(BF16).to(DEV)
    m = torch.full((T, H), float(round(p * 65536) == 0), dtype=torch.float64)
    assert torch.equal(ref.kept(T, H, p, 3, 4), m)
    if not bool(m.any()):
        x[:, 5] = float("nan")  # takes no part
    for seed in (3, torch.tensor([3, 0], dtype=torch.int64, device=DEV)):
        y, h, rstd = cake.cake_dropout_norm_fwd(x, e, w, p, seed, 4)
        want, err = ref.dropout_sum(x, m, e)
        assert ref.excess(h, want, ref.rounded(want, err)) <= 1
        hd = h.double().cpu()
        y64 = hd / torch.sqrt((hd * hd).mean(1, keepdim=True) + 1e-6) * w.double().cpu()
        assert ref.excess(y, y64, ref.rounded(y64, y64.abs() * (ref.RSTD_REL + 3 * ref.U))) <= 1
        want = ref.dropout_norm_bwd(dy, h, rstd, w, dh, m)
        for name, v in zip(("dresidual", "dx", "dw"), cake.cake_dropout_norm_bwd(dy, h, rstd, w, p, seed, 4, dh)):
            assert ref.excess(v, *want[name]) <= 1, name


def test_an_elements_place_does_not_go_by_the_shape(cake):
    """A dense tensor's mask is that of its elements in a row, as [T, H] or as [T, n, H / n]."""
    g = torch.Generator().manual_seed(1)
    x, e = rows(g, 33, 8192), rows(g, 33, 8192)
    want = cake.cake_dropout_fwd(x, 0.3, 5, 6, e)
    for n in (2, 8, 1024):
        assert torch.equal(cake.cake_dropout_fwd(x.view(33, n, -1), 0.3, 5, 6, e.view(33, n, -1)).view(33, -1), want)
