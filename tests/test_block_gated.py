"""The gated feed-forward block against FP64 on a GB300."""
import pytest
import torch

from tests import block_reference as ref

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF16, F32 = torch.bfloat16, torch.float32
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cake():
    import __graft_entry__
    __graft_entry__.build()
    import bwd_dw_column_gb300 as cake
    yield cake
    assert cake.cake_rmsnorm_device_status() == 0


def check(name, got, want, allow):
    share = ref.excess(got, want, allow)
    assert share <= 1, f"{name}: {share:.3g} of its bound"


def matrix(g, rows, cols, pad=0, std=1.0):
    return (torch.randn(rows, cols + pad, generator=g, device=DEV) * std).to(BF16)[:, :cols]


def make(T, H, F, pad=0):
    g = torch.Generator(device=DEV).manual_seed(T + H + F)
    return matrix(g, T, H, pad), matrix(g, F, H, 0, H ** -0.5), matrix(g, F, H, pad, H ** -0.5), g


# one token to several tiles; odd widths; sums over k of part of a block, of one block, and of more than the ring holds
SHAPES = [(1, 8, 8), (1, 64, 128), (1, 2048, 640), (3, 1000, 264), (16, 128, 128), (17, 520, 1032), (48, 256, 384),
          (64, 1024, 2000), (100, 264, 136), (128, 4096, 512), (129, 8, 8), (129, 64, 128), (200, 72, 264),
          (256, 512, 256), (257, 1000, 136), (300, 2048, 520), (513, 328, 1160), (1000, 136, 72), (2048, 1024, 2048)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,H,F", SHAPES)
def test_gated_fwd(cake, T, H, F, act):
    x, wg, wu, _ = make(T, H, F, 8)
    got = cake.cake_gated_fwd(x, wg, wu, act)
    want = ref.gated_fwd(x, wg, wu, act)
    for name, v in zip("hgu", got):
        check(name, v, *want[name])
    h, g, u = cake.cake_gated_fwd(x, wg, wu, act, save=False)
    assert g is u is None and torch.equal(h, got[0])
    # into columns of a wider buffer: what lies beside them stays
    buf = torch.full((T + 2, 3 * F + 16), 7.0, dtype=BF16, device=DEV)
    outs = [buf[1:T + 1, 8 + i * F:8 + (i + 1) * F] for i in range(3)]
    cake.cake_gated_fwd(x, wg, wu, act, h=outs[0], g=outs[1], u=outs[2])
    assert all(torch.equal(a, b) for a, b in zip(outs, got))
    for rest in (buf[0], buf[-1], buf[:, :8], buf[:, 8 + 3 * F:]):
        assert bool((rest == 7.0).all())


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,H,F", SHAPES)
def test_gated_bwd(cake, T, H, F, act):
    x, wg, wu, gen = make(T, H, F, 8)
    g, u, dh = (matrix(gen, T, F, p) for p in (0, 0, 16))
    got = cake.cake_gated_bwd(dh, x, g, u, wg, wu, act)
    want = ref.gated_bwd(dh, x, g, u, wg, wu, act)
    for name, v in zip(("dx", "dw_gate", "dw_up"), got):
        check(name, v, *want[name])
    again = cake.cake_gated_bwd(dh, x, g, u, wg, wu, act)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    # one of the two alone
    dx, none, _ = cake.cake_gated_bwd(dh, x, g, u, wg, wu, act, need_dw=False)
    assert none is None and torch.equal(dx, got[0])
    none, a, b = cake.cake_gated_bwd(dh, x, g, u, wg, wu, act, need_dx=False)
    assert none is None and torch.equal(a, got[1]) and torch.equal(b, got[2])
    # into slices: what lies beside them stays
    buf = torch.full((2 * F + 2, H + 16), 7.0, dtype=BF16, device=DEV)
    bx = torch.full((T + 2, H + 16), 7.0, dtype=BF16, device=DEV)
    dx, a, b = bx[1:T + 1, 8:8 + H], buf[1:F + 1, 8:8 + H], buf[F + 1:2 * F + 1, 8:8 + H]
    cake.cake_gated_bwd(dh, x, g, u, wg, wu, act, dx=dx, dw_gate=a, dw_up=b)
    assert torch.equal(dx, got[0]) and torch.equal(a, got[1]) and torch.equal(b, got[2])
    for rest in (buf[0], buf[-1], buf[:, :8], buf[:, 8 + H:], bx[0], bx[-1], bx[:, :8], bx[:, 8 + H:]):
        assert bool((rest == 7.0).all())


def test_large_and_special_values(cake):
    """Activations far out, where an exponential overflows or vanishes; infinities and NaN stay in their row."""
    T, H, F = 160, 64, 128
    x = torch.zeros(T, H, dtype=BF16, device=DEV)
    wg, wu = torch.zeros(F, H, dtype=BF16, device=DEV), torch.zeros(F, H, dtype=BF16, device=DEV)
    wg[:, 0] = 1
    wu[:, 1] = 1
    values = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 5.0, -5.0, 20.0, -20.0, 90.0, -90.0, 300.0, -300.0, 1e20, -1e20, 3e38])
    x[:len(values), 0] = values.to(BF16).to(DEV)
    x[:, 1] = 2
    for act in ("silu", "gelu"):
        h, g, u = cake.cake_gated_fwd(x, wg, wu, act)
        want = ref.gated_fwd(x, wg, wu, act)
        finite = want["h"][0].abs().cpu() < 3e38
        assert torch.equal(g[:, 0], x[:, 0])
        bad = ((h.double().cpu() - want["h"][0].cpu()).abs() > want["h"][1].cpu()) & finite
        assert not bool(bad.any())
        dh = torch.ones(T, F, dtype=BF16, device=DEV)
        eye = torch.zeros(F, H, dtype=BF16, device=DEV)
        eye[:H] = torch.eye(H, dtype=BF16, device=DEV)
        dx, _, _ = cake.cake_gated_bwd(dh, x, g, u, eye, torch.zeros_like(eye), act)
        _, da, _ = ref.act(g.double(), act)
        want = 2 * da[:, :H]
        assert bool(((dx.double() - want).abs() <= 2.0 ** -7 * want.abs() + 1e-5).all())
    x[5, 7], x[9, 3] = float("nan"), float("inf")
    wg[:, 3] = wu[:, 3] = 1
    for rows in (T, 32):
        h, g, u = cake.cake_gated_fwd(x[:rows], wg, wu)
        clean = [i for i in range(rows) if i not in (5, 9)]
        assert bool(torch.isnan(h[5]).all()) and bool((g[9] == float("inf")).all())
        assert bool(torch.isfinite(h[clean].float()[:12]).all())


def test_rows_do_not_depend_on_their_neighbours(cake):
    """A token's h has the same bits in batches of the same form, wherever it stands."""
    x, wg, wu, _ = make(600, 256, 384)
    h = cake.cake_gated_fwd(x, wg, wu)[0]
    assert torch.equal(cake.cake_gated_fwd(x.flip(0), wg, wu)[0].flip(0), h)
    assert torch.equal(cake.cake_gated_fwd(x[:300].contiguous(), wg, wu)[0], h[:300])
    few = cake.cake_gated_fwd(x[:40].contiguous(), wg, wu)[0]
    assert torch.equal(cake.cake_gated_fwd(x[20:40].contiguous(), wg, wu)[0], few[20:])


def test_weights_as_halves_of_one_matrix(cake):
    x, wg, wu, gen = make(333, 136, 200)
    both = torch.cat([wg, wu])
    got = cake.cake_gated_fwd(x, both[:200], both[200:])
    assert all(torch.equal(a, b) for a, b in zip(got, cake.cake_gated_fwd(x, wg.contiguous(), wu.contiguous())))
    # and side by side
    beside = torch.cat([wg, wu], 1)
    assert torch.equal(cake.cake_gated_fwd(x, beside[:, :136], beside[:, 136:])[0], got[0])


def test_autograd(cake):
    x, wg, wu, gen = make(140, 128, 192)
    x, wg, wu = (t.contiguous().requires_grad_() for t in (x, wg, wu))
    dh = matrix(gen, 140, 192)
    cake.cake_gated(x.view(4, 35, 128), wg, wu, "gelu").backward(dh.view(4, 35, 192))
    h, g, u = cake.cake_gated_fwd(x.detach(), wg.detach(), wu.detach(), "gelu")
    want = cake.cake_gated_bwd(dh, x.detach(), g, u, wg.detach(), wu.detach(), "gelu")
    assert all(torch.equal(a.grad, b) for a, b in zip((x, wg, wu), want))
    with torch.no_grad():
        assert torch.equal(cake.cake_gated(x, wg, wu, "gelu"), h)
    # the weights' gradients alone, and only the input's
    gx, = torch.autograd.grad(cake.cake_gated(x, wg.detach(), wu.detach(), "gelu"), x, dh)
    assert torch.equal(gx, want[0])
    gw, = torch.autograd.grad(cake.cake_gated(x.detach(), wg, wu.detach(), "gelu"), wg, dh)
    assert torch.equal(gw, want[1])


def test_gradients_against_differences(cake):
    """Gradients against central differences of the FP64 form: BF16 roundings of dg, du and of the result."""
    T, H, F = 5, 16, 24
    x, wg, wu, gen = make(T, H, F)
    dh = matrix(gen, T, F)
    for act in ("silu", "gelu"):
        _, g, u = cake.cake_gated_fwd(x, wg, wu, act)
        got = cake.cake_gated_bwd(dh, x, g, u, wg, wu, act)
        leaves = [t.double().cpu() for t in (x, wg, wu)]

        def terms(leaves):
            gg, uu = leaves[0] @ leaves[1].t(), leaves[0] @ leaves[2].t()
            return ref.act(gg, act)[0] * uu * dh.double().cpu()

        for n, d in enumerate(got):
            for at in ((0, 0), (d.shape[0] - 1, 3), (2, d.shape[1] - 1)):
                e = torch.zeros_like(leaves[n])
                e[at] = 1e-4
                up, down = (terms([t + s * e if i == n else t for i, t in enumerate(leaves)]) for s in (1, -1))
                diff = (up - down) / 2e-4
                # every term carries the roundings of g, u (saved) and of dg, du
                assert abs(float(d[at]) - float(diff.sum())) <= 4 * 2.0 ** -8 * float(diff.abs().sum()) + 0.02


def test_offsets_past_31_bits(cake):
    """Outputs of more than 2^31 elements: the last rows, and columns of the weights' gradients."""
    T, H, F = 270000, 64, 8192
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    x, wg, wu, gen = make(T, H, F)
    h, g, u = cake.cake_gated_fwd(x, wg, wu)
    for s in (slice(0, 40), slice(262140, 262150), slice(T - 40, T)):
        want = ref.gated_fwd(x[s], wg, wu, "silu")
        for name, v in (("h", h), ("g", g), ("u", u)):
            check(name, v[s], *want[name])
    del h
    dh = torch.empty_like(g).normal_(generator=gen)
    dx, dwg, dwu = cake.cake_gated_bwd(dh, x, g, u, wg, wu)
    for s in (slice(0, 40), slice(T - 40, T)):
        check("dx", dx[s], *ref.gated_bwd(dh[s], x[s], g[s], u[s], wg, wu, "silu", False)["dx"])
    for s in (slice(0, 8), slice(F - 8, F)):
        want = ref.gated_bwd(dh[:, s], x, g[:, s], u[:, s], wg[s], wu[s], "silu")
        check("dw_gate", dwg[s], *want["dw_gate"])
        check("dw_up", dwu[s], *want["dw_up"])


def test_few_tokens_lose_nothing_to_a_rounding_of_the_gradients(cake):
    """One token: a weight's gradient is a single product, which is rounded once (and off by FP32 roundings)."""
    for T in (1, 2):
        x, wg, wu, gen = make(T, 64, 1024)
        g, u, dh = (matrix(gen, T, 1024) for _ in range(3))
        dx, dwg, dwu = cake.cake_gated_bwd(dh, x, g, u, wg, wu)
        a, da, _ = ref.act(g.double(), "silu")
        for got, d in ((dwg, dh.double() * u.double() * da), (dwu, dh.double() * a)):
            want = d.t() @ x.double()
            terms = d.abs().t() @ x.double().abs()
            # half a BF16 step of the result, 2^-16 of each term for the rest's rounding, FP32's of act' and the sum
            assert bool(((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -15 * terms + 1e-30).all())


def test_infinite_gradients_of_few_tokens(cake):
    """An infinite or NaN gradient stays what it is: no rest is taken of it."""
    x, wg, wu, gen = make(3, 64, 128)
    g, u, dh = (matrix(gen, 3, 128).contiguous() for _ in range(3))
    dh[1, 5], dh[2, 7] = float("inf"), float("nan")
    u[1, 5] = g[1, 5] = 1
    x[1, 0] = 2
    x[0] = x[2] = 0
    _, dwg, dwu = cake.cake_gated_bwd(dh, x, g, u, wg, wu)
    assert dwg[5, 0] == float("inf") and dwu[5, 0] == float("inf")
    assert bool(torch.isnan(dwg[7]).all()) and bool(torch.isfinite(dwg[8:].float()).all())
