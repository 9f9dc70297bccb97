"""The training-step operators used together, as a training loop uses them:
embedding -> two blocks, each followed by a sandwich norm -> gradients ->
clipping.  Every operator is held to FP64 in its own test; here the autograd
functions' run must give the bits of the same run written out with the entry
points, eagerly and replayed from a CUDA graph, and a few optimizer steps have
to run."""
import pytest
import torch

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF16 = torch.bfloat16
pytestmark = pytest.mark.gpu
V, H, T = 500, 640, 300
PAD = 7


@pytest.fixture(scope="module")
def cake():
    import __graft_entry__
    __graft_entry__.build()
    import bwd_dw_column_gb300 as cake
    yield cake
    assert cake.cake_rmsnorm_device_status() == 0


def make():
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    params = {"table": r(V, H).mul(0.1), "w1": r(H, H).div(H ** 0.5).to(BF16), "w2": r(H, H).div(H ** 0.5).to(BF16),
              "post1": 1 + 0.1 * r(H), "pre1": (1 + 0.1 * r(H)).to(BF16), "post2": (1 + 0.1 * r(H)).to(BF16),
              "pre2": 1 + 0.1 * r(H), "gate": torch.sigmoid(r(T))}
    ids = torch.randint(0, V, (T,), generator=g)
    ids[::9], ids[5] = PAD, -1
    return {k: v.to(DEV).requires_grad_() for k, v in params.items()}, ids.to(DEV), r(T, H).to(BF16).to(DEV)


def forward(cake, p, ids):
    x0 = cake.cake_embedding(ids, p["table"], 2.0, padding_idx=PAD)
    z1 = x0 @ p["w1"]
    y1, h1 = cake.cake_sandwich_norm(z1, x0, p["post1"], p["pre1"], 1e-6, p["gate"], 0.5)
    z2 = y1 @ p["w2"]
    return cake.cake_sandwich_norm(z2, h1, p["post2"], p["pre2"])


def written_out(cake, p, ids, dy):
    p = {k: v.detach() for k, v in p.items()}
    x0 = cake.cake_embedding_fwd(ids, p["table"], 2.0)
    z1 = x0 @ p["w1"]
    y1, h1, a1, b1 = cake.cake_sandwich_fwd(z1, x0, p["post1"], p["pre1"], 1e-6, p["gate"], 0.5)
    z2 = y1 @ p["w2"]
    y2, h2, a2, b2 = cake.cake_sandwich_fwd(z2, h1, p["post2"], p["pre2"])
    dh1, dz2, dpost2, dpre2, _ = cake.cake_sandwich_bwd(dy, h2, z2, a2, b2, p["post2"], p["pre2"])
    dy1 = dz2 @ p["w2"].t()
    dx0, dz1, dpost1, dpre1, dgate = cake.cake_sandwich_bwd(dy1, h1, z1, a1, b1, p["post1"], p["pre1"], dh1, p["gate"],
                                                            0.5)
    dx0 = dx0 + dz1 @ p["w1"].t()
    return y2, {"table": cake.cake_embedding_bwd(dx0, ids, V, 2.0, PAD), "w1": x0.t() @ dz1, "w2": y1.t() @ dz2,
                "post1": dpost1, "pre1": dpre1.to(BF16), "post2": dpost2.to(BF16), "pre2": dpre2, "gate": dgate}


def test_autograd_run_gives_the_written_out_bits(cake):
    p, ids, dy = make()
    y, _ = forward(cake, p, ids)
    y.backward(dy)
    y2, want = written_out(cake, p, ids, dy)
    torch.cuda.synchronize()
    assert torch.equal(y, y2)
    for k, v in p.items():
        assert v.grad.dtype == v.dtype and torch.equal(v.grad, want[k]), k
    assert not p["table"].grad[PAD].any()
    # clipping the run's gradients, in place and into FP32 buffers
    grads = [v.grad for v in p.values()]
    into = [torch.empty(g.shape, dtype=torch.float32, device=DEV) for g in grads]
    norm = float(cake.cake_grad_norm(grads))
    assert norm > 0
    n1 = cake.cake_clip_grad_norm(grads, norm / 2, out=into)
    n2 = cake.cake_clip_grad_norm(grads, norm / 2)
    assert float(n1) == float(n2) == norm
    for g, o in zip(grads, into):
        assert torch.equal(g, o.to(g.dtype))


def test_step_in_a_graph(cake):
    p, ids, dy = make()
    opt = torch.optim.SGD(list(p.values()), lr=0.05)

    def step():
        opt.zero_grad(set_to_none=True)
        y, _ = forward(cake, p, ids)
        y.backward(dy)
        norm = cake.cake_clip_grad_norm([v.grad for v in p.values()], 1.0)
        opt.step()
        return norm

    start = {k: v.detach().clone() for k, v in p.items()}
    eager = [float(step()) for _ in range(4)]
    after = {k: v.detach().clone() for k, v in p.items()}
    assert all(n > 0 for n in eager)

    def reset():
        with torch.no_grad():
            for k, v in p.items():
                v.copy_(start[k])

    # no eager graph of these leaves is alive any more, and the warm-up runs on the capturing side
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = step()
    reset()
    replayed = []
    for _ in range(4):
        graph.replay()
        replayed.append(float(norm))
    torch.cuda.synchronize()
    assert replayed == eager
    for k, v in p.items():
        assert torch.equal(v, after[k]), k


def test_given_streams_and_host_threads(cake):
    """Calls of several host threads, each on a stream of its own, give what each gives alone."""
    import threading

    def work(seed, stream):
        g = torch.Generator().manual_seed(seed)
        with torch.cuda.stream(stream):
            ids = torch.randint(0, V, (2000 + seed,), generator=g).to(DEV)
            rows = [torch.randn(2000 + seed, H, generator=g).to(BF16).to(DEV) for _ in range(3)]
            w = torch.ones(H, device=DEV)
        stream.synchronize()
        got = []
        for _ in range(6):
            _, h, a, b = cake.cake_sandwich_fwd(rows[0], rows[1], w, w, stream=stream)
            _, dz, dwo, _, _ = cake.cake_sandwich_bwd(rows[2], h, rows[0], a, b, w, w, stream=stream)
            table = cake.cake_embedding_bwd(dz, ids, V, stream=stream)
            norm = cake.cake_grad_norm([table, dwo, dz], stream=stream)
            y = cake.cake_embedding_fwd(ids, table, stream=stream)
            with torch.cuda.stream(stream):
                got.append([t.clone() for t in (dz, dwo, table, y)] + [norm])
                cake.cake_clip_grad_norm([table, dwo], 1e-3, stream=stream)
                got[-1] += [table, dwo]
        stream.synchronize()
        return got

    alone = [work(s, torch.cuda.Stream()) for s in range(3)]
    streams, out = [torch.cuda.Stream() for _ in range(3)], [None] * 3

    def run(s):
        out[s] = work(s, streams[s])

    threads = [threading.Thread(target=run, args=(s,)) for s in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for a, b in zip(alone, out):
        for i in range(6):
            for x, y in zip(a[0], b[i]):
                assert torch.equal(x, y)


def _calls(cake, seed):
    """Inputs, and a call of every operator that reads them and returns what it wrote."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(BF16).to(DEV)  # noqa: E731
    big, table_rows, n = 5_000_000, 700, 3000
    ins = {"z": r(n, H), "x": r(n, H), "dy": r(n, H), "table": r(table_rows, H).float(),
           "ids": torch.randint(0, table_rows, (n,), generator=g).to(DEV),
           "far": torch.randint(0, big, (n,), generator=g).to(DEV)}
    w = torch.ones(H, device=DEV)
    small = torch.full((n, 8), 0.5, dtype=BF16, device=DEV)
    _, h, a, b = cake.cake_sandwich_fwd(ins["z"], ins["x"], w, w)

    def clip(t):
        out = torch.empty(t.shape, dtype=torch.float32, device=DEV)
        return cake.cake_clip_grad_norm([t], 1.0, out=[out]), out

    return ins, {
        "fwd": ("z", lambda i: cake.cake_sandwich_fwd(i["z"], i["x"], w, w)),
        "bwd": ("dy", lambda i: cake.cake_sandwich_bwd(i["dy"], h, i["z"], a, b, w, w)[:4]),
        "norm": ("x", lambda i: (cake.cake_grad_norm([i["x"], i["z"]]),)),
        "short": ("table", lambda i: (cake.cake_grad_norm([i["table"][:9]]),)),
        "clip": ("x", lambda i: clip(i["x"])),
        "clip short": ("z", lambda i: clip(i["z"][:20])),
        "lookup": ("ids", lambda i: (cake.cake_embedding_fwd(i["ids"], i["table"]),)),
        "gradient": ("dy", lambda i: (cake.cake_embedding_bwd(i["dy"], i["ids"], table_rows),)),
        "gradient, many rows": ("far", lambda i: (cake.cake_embedding_bwd(small, i["far"], big),)),
    }


@pytest.mark.parametrize("name", ["fwd", "bwd", "norm", "short", "clip", "clip short", "lookup", "gradient",
                                  "gradient, many rows"])
def test_waits_for_the_work_before(cake, name):
    """A call right behind the kernel, copy or fill that writes its input reads what that has written, eagerly and in
    a graph, and its outputs are whole for the work behind it."""
    ins, calls = _calls(cake, 11)
    key, call = calls[name]
    other = _calls(cake, 12)[0][key]
    zero, slow = torch.zeros_like(other), torch.randn(4096, 4096, device=DEV)
    want = {}
    for k, src in (("a", ins[key].clone()), ("b", other), ("zero", zero)):
        ins[key].copy_(src)
        torch.cuda.synchronize()
        want[k] = src, [t.clone() for t in call(ins)]
        torch.cuda.synchronize()

    def run():
        got = []
        for k in ("a", "b", "zero", "b", "a"):
            slow @ slow  # work that the writer of the input waits behind
            if k == "zero":
                ins[key].zero_()
            else:
                ins[key].copy_(want[k][0])
            got.append((k, [t.clone() for t in call(ins)]))
            ins[key].copy_(want["a"][0])  # and one behind the call, over what it has read
        return got

    def check(got):
        torch.cuda.synchronize()
        for k, ts in got:
            for t, w in zip(ts, want[k][1]):
                assert torch.equal(t, w) or (torch.equal(t.isnan(), w.isnan()) and torch.equal(t.nan_to_num(), w.nan_to_num()))

    for _ in range(3):
        check(run())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(2):
        graph.replay()
        check(got)


@pytest.mark.parametrize("name", ["fwd", "bwd", "norm", "short", "clip", "clip short", "lookup", "gradient",
                                  "gradient, many rows"])
def test_waits_for_another_stream(cake, name):
    """A call behind a wait for another stream, which writes its input late, reads what that has written; work of
    the other stream behind the call does not reach it."""
    ins, calls = _calls(cake, 21)
    key, call = calls[name]
    other = _calls(cake, 22)[0][key]
    slow, side = torch.randn(4096, 4096, device=DEV), torch.cuda.Stream()
    want = {}
    for k, src in (("a", ins[key].clone()), ("b", other)):
        ins[key].copy_(src)
        torch.cuda.synchronize()
        want[k] = src, [t.clone() for t in call(ins)]
        torch.cuda.synchronize()
    spot = torch.zeros(8, device=DEV)

    def run():
        main, got, made = torch.cuda.current_stream(), [], []
        for k in ("a", "b", "a"):
            side.wait_stream(main)
            with torch.cuda.stream(side):
                made.append(slow @ slow)
                ins[key].copy_(want[k][0])
            spot.add_(1)  # a short kernel of this stream before the wait
            main.wait_stream(side)
            got.append((k, call(ins)))
            side.wait_stream(main)
            with torch.cuda.stream(side):
                ins[key].copy_(want["b" if k == "a" else "a"][0])
        main.wait_stream(side)
        return got, made

    def check(got):
        torch.cuda.synchronize()
        for k, ts in got:
            for t, w in zip(ts, want[k][1]):
                assert torch.equal(t, w)

    for _ in range(3):
        check(run()[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, made = run()
    for _ in range(2):
        graph.replay()
        check(got)


@pytest.mark.parametrize("rows", [300, 40_000])
def test_behind_the_norms_own_kernels(cake, rows):
    """The norm's backward, whose gradients the step's operators take up at once."""
    g = torch.Generator().manual_seed(rows)
    x, dy, z = (torch.randn(rows, H, generator=g).to(BF16).to(DEV) for _ in range(3))
    w = (1 + 0.1 * torch.randn(H, generator=g)).to(DEV)
    ids = torch.randint(0, 900, (rows,), generator=g).to(DEV)
    _, h, a, b = cake.cake_sandwich_fwd(z, x, w, w)

    def run(wait):
        pause = torch.cuda.synchronize if wait else lambda: None
        _, rstd = cake.cake_rmsnorm_fwd(x, w, 1e-6)
        dx, dw = cake.cake_rmsnorm_bwd(dy, x, rstd, w, deterministic=True)[:2]
        pause()
        norm = cake.cake_grad_norm([dw, dx])
        pause()
        dx2, dz, *_ = cake.cake_sandwich_bwd(dx, h, z, a, b, w, w)
        pause()
        table = cake.cake_embedding_bwd(dx2, ids, 900)
        pause()
        _, rstd2 = cake.cake_rmsnorm_fwd(dz, w, 1e-6)
        torch.cuda.synchronize()
        return dx, dw, norm, dx2, dz, table, rstd2

    want = run(True)
    for _ in range(5):
        for got, w_ in zip(run(False), want):
            assert torch.equal(got, w_)


def test_tensors_that_a_call_writes_count_as_changed(cake):
    """A backward pass that has saved what a call overwrites raises, as after torch's own in-place operations."""
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g).to(BF16).to(DEV)  # noqa: E731
    n, w = 40, torch.ones(H, device=DEV)
    f32 = lambda *s: torch.zeros(*s, device=DEV)  # noqa: E731
    z, x, dy, gate = r(n, H), r(n, H), r(n, H), torch.ones(n, device=DEV)
    ids = torch.randint(0, V, (n,), generator=g).to(DEV)
    table, base = r(V, H), r(V, H)
    _, h, a, b = cake.cake_sandwich_fwd(z, x, w, w)
    calls = [
        (lambda o: cake.cake_sandwich_fwd(z, x, w, w, **o), {"y": r(n, H), "h_new": r(n, H), "rstd_post": f32(n),
                                                            "rstd_pre": f32(n)}),
        (lambda o: cake.cake_sandwich_bwd(dy, h, z, a, b, w, w, None, gate, **o),
         {"dx": r(n, H), "dz": r(n, H), "dw_post": f32(H), "dw_pre": f32(H), "dgate": f32(n)}),
        (lambda o: cake.cake_grad_norm([z, x], **o), {"norm": f32(1)}),
        (lambda o: cake.cake_clip_grad_norm([z, x], 1.0, out=list(o.values())[1:], norm=o["norm"]),
         {"norm": f32(1), "a": f32(n, H), "b": f32(n, H)}),
        (lambda o: cake.cake_clip_grad_norm([None, *o.values()], 1.0), {"a": r(n, H), "b": f32(7)}),
        (lambda o: cake.cake_clip_grad_norm(o["a"], 1e9), {"a": r(3)}),
        (lambda o: cake.cake_embedding_fwd(ids, table, **o), {"y": r(n, H)}),
        (lambda o: cake.cake_embedding_bwd(dy, ids, V, **o), {"out": r(V, H)}),
        (lambda o: cake.cake_embedding_bwd(dy, ids, V, accumulate=True, **o), {"out": base}),
    ]
    read = (z, x, dy, gate, ids, table, h, a, b, w)
    before = [t._version for t in read]
    for call, outs in calls:
        was = {k: t._version for k, t in outs.items()}
        call(outs)
        assert all(t._version > was[k] for k, t in outs.items()), outs.keys()
    assert [t._version for t in read] == before

    leaf = r(n, H).requires_grad_()
    stream = leaf * 2
    kept = stream.sin()  # saves the stream for its gradient
    cake.cake_sandwich_fwd(z, stream.detach(), w, w, h_new=stream.detach())
    with pytest.raises(RuntimeError, match="inplace"):
        kept.sum().backward()
    leaf = r(n, H).requires_grad_()
    grad = leaf * 2
    kept = grad.sin()
    cake.cake_clip_grad_norm([grad.detach()], 1e-3)
    with pytest.raises(RuntimeError, match="inplace"):
        kept.sum().backward()

    with torch.inference_mode():  # such tensors have no count, in or out of the mode
        t = torch.ones(9, device=DEV)
        cake.cake_clip_grad_norm([t], 0.5)
    assert abs(float(cake.cake_clip_grad_norm([t], 0.25)) - 0.5) < 1e-5
