"""The embedding and its gradient by sorted tokens against FP64: id types and
distributions, runs of one id around the kernels' window sizes, ids without a
token, padding and ids outside the table, both table types, strided rows,
added and overwritten gradients."""
import pytest
import torch

from tests import step_reference as ref

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def cake():
    import __graft_entry__
    __graft_entry__.build()
    import bwd_dw_column_gb300 as cake
    cake.cake_rmsnorm_device_status(clear=True) if torch.cuda.is_available() else None
    yield cake
    if torch.cuda.is_available():
        assert cake.cake_rmsnorm_device_status() == 0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def make_ids(kind, T, V, seed=0):
    g = gen(seed + 17 * T + V)
    if kind == "one":
        return torch.full((T,), V - 1)
    if kind == "all":
        return torch.arange(T) % V
    if kind == "log":
        return (torch.rand(T, generator=g, dtype=torch.float64) * torch.tensor(V + 1.0).log()).exp().long().sub(1).clamp(0, V - 1)
    if kind == "uniform":
        return torch.randint(0, V, (T,), generator=g)
    # runs whose lengths lie around the windows' and the overrun's
    lengths = [1, 2, 31, 32, 33, 34, 63, 64, 65, 66, 95, 96, 97, 127, 128, 129, 159, 160, 161, 300, 1]
    order = torch.randperm(len(lengths), generator=g).tolist()
    ids, k = [], 0
    while len(ids) < T:
        ids += [k % V] * lengths[order[k % len(order)]]
        k += 1
    return torch.tensor(ids[:T])[torch.randperm(T, generator=g)]


def check_bwd(cake, dy, ids, V, scale=1.0, pad=None, out=None, accumulate=False, dtype=F32):
    base = out.clone() if accumulate else None
    got = cake.cake_embedding_bwd(dy, ids, V, scale, pad, out, accumulate, dtype)
    torch.cuda.synchronize()
    want, mags, counts = ref.embedding_bwd(dy, ids, V, scale, pad, base)
    # as many additions as tokens, the scale, the addition to the base, the output's rounding
    err = (counts[:, None] + 4) * ref.U * mags + 2 * ref.U * want.abs()
    allow = ref.rounded(want, err) if got.dtype == BF16 else err + 2.0 ** -149
    assert ref.excess(got, want, allow) <= 1
    untouched = counts == 0
    rows = got.cpu()[untouched]
    assert torch.equal(rows, base.cpu()[untouched]) if accumulate else not rows.any()
    return got


# ---------------------------------------------------------------------- forward

@pytest.mark.gpu
@pytest.mark.parametrize("T,H,V", [(1, 8, 1), (3, 64, 10), (64, 2048, 1000), (777, 1032, 50), (5, 8192, 7), (4099, 256, 3)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
def test_forward(cake, T, H, V, dtype, idt):
    table = torch.randn(V, H, generator=gen(T)).to(dtype).to(DEV)
    ids = make_ids("uniform", T, V).to(idt).to(DEV)
    y = cake.cake_embedding_fwd(ids, table, 1.7)
    # the product in FP32 of the FP32 scale, rounded once
    want = (table.float()[ids.long()] * 1.7).to(BF16)
    assert torch.equal(y, want)


@pytest.mark.gpu
def test_forward_shapes_strides_and_missing_tokens(cake):
    V, H = 40, 264
    buf = torch.randn(V, 300, generator=gen(1)).to(DEV)
    table = buf[:, 4:4 + H]  # rows of a wider buffer
    ids = make_ids("uniform", 60, V).view(3, 4, 5).to(DEV)
    ids[1, 2, 3], ids[0, 0, 0] = -1, -100
    want = (table[ids.clamp(min=0)]).to(BF16)
    want[1, 2, 3], want[0, 0, 0] = 0, 0
    y = cake.cake_embedding_fwd(ids, table)
    assert y.shape == (3, 4, 5, H) and torch.equal(y, want)
    assert cake.cake_rmsnorm_device_status() == 0  # no token is no mistake
    out = torch.full((60, 280), 5.0, dtype=BF16, device=DEV)
    cake.cake_embedding_fwd(ids.view(60), table, y=out[:, 8:8 + H])
    assert torch.equal(out[:, 8:8 + H], want.view(60, H))
    assert bool((out[:, :8] == 5).all()) and bool((out[:, 8 + H:] == 5).all())
    nc = ids.view(12, 5).t()  # ids in another order
    assert torch.equal(cake.cake_embedding_fwd(nc, table), want.view(12, 5, H).transpose(0, 1))
    assert cake.cake_embedding_fwd(ids.view(60)[:0], table).shape == (0, H)


@pytest.mark.gpu
def test_ids_outside_the_table_are_reported(cake):
    table = torch.randn(10, 64, generator=gen(2)).to(BF16).to(DEV)
    ids = torch.tensor([3, 10, -1, 2 ** 40, 9], device=DEV)
    y = cake.cake_embedding_fwd(ids, table)
    assert cake.cake_rmsnorm_device_status(clear=True) == 1
    assert not y[1:4].any() and torch.equal(y[[0, 4]], table[[3, 9]])
    dy = torch.ones(5, 64, dtype=BF16, device=DEV)
    got = cake.cake_embedding_bwd(dy, ids, 10)
    assert cake.cake_rmsnorm_device_status(clear=True) == 1
    want = torch.zeros(10, 64, device=DEV)
    want[[3, 9]] = 1
    assert torch.equal(got, want)
    cake.cake_embedding_bwd(dy, torch.tensor([3, -1, -1, -7, 9], device=DEV), 10)
    assert cake.cake_rmsnorm_device_status() == 0


# --------------------------------------------------------------------- gradient

@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["one", "all", "log", "uniform", "runs"])
@pytest.mark.parametrize("T,H,V", [(1, 8, 1), (2, 64, 300), (31, 72, 33), (128, 1024, 100), (129, 1032, 7),
                                   (2049, 256, 70000), (5000, 128, 1000), (20_011, 64, 257)])
def test_gradient(cake, kind, T, H, V):
    dy = torch.randn(T, H, generator=gen(T + H)).to(BF16).to(DEV)
    ids = make_ids(kind, T, V).to(DEV)
    check_bwd(cake, dy, ids if T % 2 else ids.int(), V, 0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(6))
def test_runs_across_windows(cake, seed):
    # enough tokens and columns for the longer windows (shapes choose 8 to 128)
    T, H = [(3000, 64), (40_000, 64), (90_000, 64), (160_000, 64), (50_000, 1032), (30_000, 2056)][seed]
    dy = torch.randn(T, H, generator=gen(seed)).to(BF16).to(DEV)
    ids = make_ids("runs", T, 100_000, seed)
    check_bwd(cake, dy, ids.to(DEV), 100_000, 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(300, 64), (3000, 520), (9000, 1544), (25_000, 64), (25_000, 264), (6000, 4104)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_short_runs_across_short_windows(cake, T, H, accumulate):
    # windows of 8 and 16 (of 32 with the widest rows), runs that end at, before and after their ends and overruns
    lengths = [1, 2, 7, 8, 9, 10, 15, 16, 17, 18, 23, 24, 25, 31, 32, 33, 34, 40, 64, 65, 100]
    g = gen(T + H)
    order = torch.randperm(len(lengths), generator=g).tolist()
    ids, k = [], 0
    while len(ids) < T:
        ids += [k] * lengths[order[k % len(order)]]
        k += 1
    ids = torch.tensor(ids[:T])[torch.randperm(T, generator=g)].to(DEV)
    dy = torch.randn(T, H, generator=g).to(BF16).to(DEV)
    base = torch.randn(k, H, generator=g).to(DEV) if accumulate else None
    check_bwd(cake, dy, ids, k, 0.5, None, base, accumulate)
    ids[ids == 3] = -1
    check_bwd(cake, dy, ids, k, 0.5, k // 2, base, accumulate)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(70_000, 64), (300_000, 8)])
def test_one_id_has_most_tokens(cake, T, H):
    # a cut run of thousands of pieces, more than a CTA looks at in one step
    ids = make_ids("log", T, 500, 3)
    ids[torch.rand(T, generator=gen(T)) < 0.9] = 250
    dy = torch.randn(T, H, generator=gen(H)).to(BF16).to(DEV)
    check_bwd(cake, dy, ids.to(DEV), 500, 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1024, 1025, 16_384, 16_385, 32_769, 65_537, 131_072, 131_073, 200_000])
def test_both_sorts(cake, T):
    # one cluster of 1 to 16 CTAs with 1 to 8 keys a thread up to 131072 tokens, a launch per pass beyond
    dy = torch.randn(T, 8, generator=gen(T)).to(BF16).to(DEV)
    ids = make_ids("log", T, 3000, 1)
    ids[::13] = -1
    check_bwd(cake, dy, ids.to(DEV), 3000, 0.5)
    check_bwd(cake, dy, ids.int().to(DEV), 3000, 0.5, 17, torch.randn(3000, 8, generator=gen(1)).to(DEV), True)
    ids[3] = 1 << 30
    check_bwd(cake, dy, ids.to(DEV), 3000)
    assert cake.cake_rmsnorm_device_status(clear=True) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 255, 256, 65_535, 65_536, 300_001, 5_000_000])
def test_table_sizes(cake, V):
    # digits of a pass, and bitmaps zeroed by the sort or before it
    dy = torch.randn(700, 16, generator=gen(V)).to(BF16).to(DEV)
    check_bwd(cake, dy, make_ids("uniform", 700, V).to(DEV), V)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("accumulate", [False, True])
def test_padding_types_and_adding(cake, dtype, accumulate):
    T, H, V = 3001, 320, 500
    dy = torch.randn(T, H, generator=gen(5)).to(BF16).to(DEV)
    ids = make_ids("log", T, V).to(DEV)
    ids[::7] = 123
    ids[5::11] = -1
    buf = torch.randn(V, 400, generator=gen(6)).to(dtype).to(DEV)
    before = buf.clone()
    out = buf[:, 16:16 + H]
    check_bwd(cake, dy, ids, V, 0.3, 123, out, accumulate, dtype)
    assert torch.equal(buf[:, :16], before[:, :16]) and torch.equal(buf[:, 16 + H:], before[:, 16 + H:])
    if not accumulate:
        assert torch.equal(cake.cake_embedding_bwd(dy, ids, V, 0.3, 123, dtype=dtype), out)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_of_tokens_that_do_not_count(cake, bad):
    # what stands in the rows of padding and of missing tokens is not looked at
    T, H, V = 900, 136, 40
    dy = torch.randn(T, H, generator=gen(11)).to(BF16).to(DEV)
    ids = make_ids("log", T, V).to(DEV)
    ids[::5], ids[1::7] = 9, -3
    out = (ids == 9) | (ids < 0)
    want = cake.cake_embedding_bwd(dy, ids, V, padding_idx=9)
    dy[out] = bad
    got = cake.cake_embedding_bwd(dy, ids, V, padding_idx=9)
    assert torch.equal(got, want) and bool(torch.isfinite(got).all())
    # and where they count, they stay in their row
    hit = int(ids[~out][0])
    dy[out] = 0
    dy[(ids == hit).nonzero()[0], 5] = bad
    got = cake.cake_embedding_bwd(dy, ids, V, padding_idx=9)
    assert not bool(torch.isfinite(got[hit, 5])) and int((~torch.isfinite(got)).sum()) == 1


@pytest.mark.gpu
def test_all_tokens_are_padding(cake):
    dy = torch.randn(700, 64, generator=gen(7)).to(BF16).to(DEV)
    for ids in (torch.full((700,), 4), torch.full((700,), -1)):
        check_bwd(cake, dy, ids.to(DEV), 9, pad=4)
        check_bwd(cake, dy, ids.to(DEV), 9, pad=4, out=torch.randn(9, 64, device=DEV), accumulate=True)


@pytest.mark.gpu
def test_no_tokens(cake):
    dy, ids = torch.empty(0, 64, dtype=BF16, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV)
    buf = torch.ones(5, 72, device=DEV)
    cake.cake_embedding_bwd(dy, ids, 5, out=buf[:, :64])
    assert not buf[:, :64].any() and bool((buf[:, 64:] == 1).all())
    keep = torch.ones(5, 64, device=DEV)
    cake.cake_embedding_bwd(dy, ids, 5, out=keep, accumulate=True)
    assert bool((keep == 1).all())


@pytest.mark.gpu
def test_strided_rows_and_shapes(cake):
    T, H, V = 210, 256, 30
    wide = torch.randn(T, 320, generator=gen(8)).to(BF16).to(DEV)
    ids = make_ids("log", T, V).to(DEV)
    a = check_bwd(cake, wide[:, 64:], ids, V)
    b = check_bwd(cake, wide[:, 64:].contiguous().view(7, 30, H), ids.view(7, 30), V)
    assert torch.equal(a, b)


@pytest.mark.gpu
def test_the_same_bits_every_time_and_in_graphs(cake):
    T, H, V = 9000, 512, 4000
    dys = [torch.randn(T, H, generator=gen(s)).to(BF16).to(DEV) for s in (1, 2)]
    ids = [make_ids("log", T, V, s).to(DEV) for s in (1, 2)]
    want = [cake.cake_embedding_bwd(d, i, V, 0.5).clone() for d, i in zip(dys, ids)]
    outs, graphs = [], []
    for d, i in zip(dys, ids):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(cake.cake_embedding_bwd(d, i, V, 0.5))
        graphs.append(g)
    for _ in range(4):
        streams = [torch.cuda.Stream() for _ in graphs]
        for o in outs:
            o.fill_(9)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,V", [(1, 64, 3000), (700, 256, 20_000), (1024, 1024, 8000), (3000, 128, 50_000),
                                   (140_000, 8, 9000)])
def test_a_workspace_holds_nothing_between_calls(cake, T, H, V):
    """Calls one after another in one workspace, whose flags, bitmap and lists are those of other ids' calls."""
    sets = [(make_ids("uniform", T, V, s).to(DEV), torch.randn(T, H, generator=gen(s)).to(BF16).to(DEV))
            for s in range(3)]
    want = [cake.cake_embedding_bwd(dy, ids, V) for ids, dy in sets]
    base = torch.randn(V, H, generator=gen(9)).to(DEV)
    added = [cake.cake_embedding_bwd(dy, ids, V, out=base.clone(), accumulate=True) for ids, dy in sets]
    ws = torch.full((cake.cake_embedding_bwd_workspace_size(T, V, H),), 0xff, dtype=torch.uint8, device=DEV)
    outs = [torch.empty(V, H, device=DEV) for _ in range(6)]
    for _ in range(20):
        for k, o in enumerate(outs):  # nothing waits between the calls
            ids, dy = sets[k % 3]
            cake.cake_embedding_bwd(dy, ids, V, out=o.copy_(base) if k == 4 else o.fill_(5), accumulate=k == 4,
                                    workspace=ws)
        torch.cuda.synchronize()
        for k, o in enumerate(outs):
            assert torch.equal(o, added[k % 3] if k == 4 else want[k % 3]), k


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_autograd(cake, dtype):
    V, H = 300, 192
    table = torch.randn(V, H, generator=gen(9)).to(dtype).to(DEV).requires_grad_()
    ids = make_ids("log", 400, V).view(4, 100).to(DEV)
    y = cake.cake_embedding(ids, table, 2.0, padding_idx=3)
    dy = torch.randn(4, 100, H, generator=gen(10)).to(BF16).to(DEV)
    y.backward(dy)
    assert torch.equal(y, cake.cake_embedding_fwd(ids, table.detach(), 2.0))
    assert table.grad.dtype == dtype
    assert torch.equal(table.grad, cake.cake_embedding_bwd(dy, ids, V, 2.0, 3, dtype=dtype))


@pytest.mark.gpu
def test_python_refusals(cake):
    table = torch.zeros(10, 64, device=DEV)
    ids = torch.zeros(4, dtype=torch.int64, device=DEV)
    dy = torch.zeros(4, 64, dtype=BF16, device=DEV)
    for call, error in ((lambda: cake.cake_embedding_fwd(ids.float(), table), TypeError),
                        (lambda: cake.cake_embedding_fwd(ids, table.half()), TypeError),
                        (lambda: cake.cake_embedding_fwd(ids, table[0]), ValueError),
                        (lambda: cake.cake_embedding_fwd(ids, table.t()), ValueError),
                        (lambda: cake.cake_embedding_fwd(ids.cpu(), table), ValueError),
                        (lambda: cake.cake_embedding_fwd(ids, table, y=dy[:3]), ValueError),
                        (lambda: cake.cake_embedding_bwd(dy[:3], ids, 10), ValueError),
                        (lambda: cake.cake_embedding_bwd(dy.float(), ids, 10), TypeError),
                        (lambda: cake.cake_embedding_bwd(dy, ids, 10, accumulate=True), ValueError),
                        (lambda: cake.cake_embedding_bwd(dy, ids, 11, out=table), ValueError),
                        (lambda: cake.cake_embedding_bwd(dy, ids, 10, padding_idx=10), ValueError),
                        (lambda: cake.cake_embedding_bwd(dy, ids, 10, padding_idx=-1), ValueError),
                        (lambda: cake.cake_embedding_bwd(dy[:, :60], ids, 10), cake.CakeError)):
        with pytest.raises(error):
            call()


@pytest.mark.gpu
def test_a_table_beyond_2_to_31_values(cake):
    V, H = 300_000, 8192  # 2.46e9 values
    table = torch.zeros(V, H, dtype=BF16, device=DEV)
    ids = torch.tensor([V - 1, 5, V - 1, 290_000], device=DEV)
    table[V - 1], table[290_000] = 3.0, 2.0
    y = cake.cake_embedding_fwd(ids, table)
    assert [float(y[i, -1]) for i in range(4)] == [3.0, 0.0, 3.0, 2.0]
    got = cake.cake_embedding_bwd(y, ids, V, out=table.fill_(7))
    assert got.data_ptr() == table.data_ptr()
    assert [float(got[i, -1]) for i in (V - 1, 290_000, 5, 0, V - 2)] == [6.0, 2.0, 0.0, 0.0, 0.0]
