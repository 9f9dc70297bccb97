"""Gradients as autograd hands them to the package's functions: slices of longer ones,
on any boundary, and in other storage orders."""
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


def rows(*size, seed=1):
    return torch.randn(*size, generator=torch.Generator().manual_seed(seed)).to(BF16).to(DEV)


@pytest.mark.parametrize("T", [1, 6])
def test_gradients_that_lie_anywhere(cake, T):
    """A concatenation's gradients are slices of one: contiguous, but on any boundary, and a single row's stride is
    whatever the buffer's is.  They give what copies of them give."""
    H, F, D = 64, 136, 32
    x, res, wg, wu, w = rows(T, H, seed=2), rows(T, H, seed=3), rows(F, H, seed=4), rows(F, H, seed=5), rows(H, seed=6)
    q, k, wd = rows(T, 4, D, seed=7), rows(T, 2, D, seed=8), rows(D, seed=9)
    ids, table = torch.arange(T, device=DEV), rows(16, H, seed=10)
    turns, _ = cake.cake_rotary_table((16,), device=DEV)
    pos = torch.arange(T, device=DEV)
    calls = [
        (lambda a, b, c: (cake.cake_gated(a, b, c),), (x, wg, wu)),
        (lambda a, b, c, d: cake.cake_rotary(a, b, pos, turns, None, c, d), (q, k, wd, wd)),
        (lambda a, b: cake.cake_rotary(a, b, pos, turns), (q, k)),
        (lambda a, b: (cake.cake_dropout(a, 0.3, 5, residual=b),), (x, res)),
        (lambda a, b, c: cake.cake_dropout_norm(a, b, c, 0.3, 5), (x, res, w)),
        (lambda a, b, c, d: cake.cake_sandwich_norm(a, b, c, d), (x, res, w, w)),
        (lambda a, b: cake.cake_rmsnorm(a, b, residual=res), (x, w)),
        (lambda a: (cake.cake_embedding(ids, a),), (table,)),
    ]
    for i, (call, ins) in enumerate(calls):
        leaves = [t.clone().requires_grad_() for t in ins]
        outs = call(*leaves)
        shapes = [o.shape for o in outs]
        n = sum(o.numel() for o in outs)
        flat = rows(3 + n, seed=20 + i)
        parts = [p.view(s) for p, s in zip(flat[3:].split([s.numel() for s in shapes]), shapes)]
        want = torch.autograd.grad(outs, leaves, [p.clone() for p in parts])
        # behind three other elements of a vector
        outs = call(*leaves)
        got = torch.autograd.grad(torch.cat([rows(3), *(o.reshape(-1) for o in outs)]), leaves, flat)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
        # beside three other columns
        outs = call(*leaves)
        wide = [torch.cat([o, o.detach()[..., :3]], -1) for o in outs]
        got = torch.autograd.grad(wide, leaves, [torch.cat([p, p[..., :3]], -1) for p in parts])
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_heads_major_gradients(cake):
    """The rotary backward of gradients in [heads, T, D] storage, as an attention over such heads hands them back."""
    T, D = 70, 64
    q, k, w = rows(T, 5, D, seed=2), rows(T, 2, D, seed=3), rows(D, seed=4)
    turns, _ = cake.cake_rotary_table((32,), device=DEV)
    pos = torch.arange(T, device=DEV)
    dq, dk = rows(5, T, D, seed=5).transpose(0, 1), rows(2, T, D, seed=6).transpose(0, 1)
    _, _, rq, rk = cake.cake_rotary_fwd(q, k, pos, turns, None, w, w)
    norm = (q, k, rq, rk, w, w)
    for rest in (norm, ()):
        want = cake.cake_rotary_bwd(dq.contiguous(), dk.contiguous(), pos, turns, None, *rest)
        got = cake.cake_rotary_bwd(dq, dk, pos, turns, None, *rest)
        assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, want))
        a, b = dq.clone(), dk.clone()  # in place (a copy keeps the strides)
        assert a.stride() == dq.stride()
        cake.cake_rotary_bwd(a, b, pos, turns, None, *rest, dq_out=a, dk_out=b)
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
