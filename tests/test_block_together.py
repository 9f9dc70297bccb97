"""A block's operators used together with the norm's and the step's, as a
training loop uses them: norm -> queries and keys, normed and rotated -> a plain
attention -> dropout, residual and norm -> gated block -> projection -> dropout
and residual -> gradients -> clipping.  Every operator is held to FP64 in its own
test; here the autograd functions' run must give the bits of the run written out
with the entry points, eagerly and replayed from a CUDA graph, on several streams
and behind other work."""
import threading

import pytest
import torch

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF16 = torch.bfloat16
pytestmark = pytest.mark.gpu
T, H, NQ, NK, D, F = 150, 256, 4, 2, 64, 392
P, SECTIONS = 0.1, (8, 12, 12)


@pytest.fixture(scope="module")
def cake():
    import __graft_entry__
    __graft_entry__.build()
    import bwd_dw_column_gb300 as cake
    yield cake
    assert cake.cake_rmsnorm_device_status() == 0


def make(cake, seed=5):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    m = lambda *s: r(*s).div(s[-1] ** 0.5).to(BF16)  # noqa: E731
    params = {"w0": 1 + 0.1 * r(H), "qkv": m((NQ + 2 * NK) * D, H), "wq": 1 + 0.1 * r(D), "wk": (1 + 0.1 * r(D)).to(BF16),
              "o": m(H, NQ * D), "w1": (1 + 0.1 * r(H)).to(BF16), "gate": m(F, H), "up": m(F, H), "down": m(H, F)}
    rest = {"x": r(T, H).to(BF16).to(DEV), "dy": r(T, H).to(BF16).to(DEV),
            "pos": torch.randint(0, 200, (3, T), generator=g).to(DEV),
            "rng": torch.tensor([seed, 0], dtype=torch.int64, device=DEV)}
    rest["turns"], rest["axes"] = cake.cake_rotary_table(SECTIONS, device=DEV)
    return {k: v.to(DEV).requires_grad_() for k, v in params.items()}, rest


def attention(q, k, v):
    k, v = (t.repeat_interleave(NQ // NK, 1).transpose(0, 1) for t in (k, v))
    s = (q.transpose(0, 1) @ k.transpose(1, 2)).float() * D ** -0.5
    return (torch.softmax(s, -1).to(BF16) @ v).transpose(0, 1).reshape(T, NQ * D)


def forward(cake, p, a):
    y = cake.cake_rmsnorm(a["x"], p["w0"], eps=1e-6)
    qkv = y @ p["qkv"].t()
    q, k, v = (t.view(T, -1, D) for t in qkv.split((NQ * D, NK * D, NK * D), 1))
    q, k = cake.cake_rotary(q, k, a["pos"], a["turns"], a["axes"], p["wq"], p["wk"])
    z = attention(q, k, v) @ p["o"].t()
    y, h = cake.cake_dropout_norm(z, a["x"], p["w1"], P, a["rng"], 1)
    f = cake.cake_gated(y, p["gate"], p["up"], "gelu")
    return cake.cake_dropout(f @ p["down"].t(), P, a["rng"], 2, residual=h)


def written_out(cake, p, a):
    p = {k: v.detach() for k, v in p.items()}
    x, dy = a["x"], a["dy"]
    y0, r0 = cake.cake_rmsnorm_fwd(x, p["w0"], 1e-6)
    qkv = y0 @ p["qkv"].t()
    q0, k0, v = (t.view(T, -1, D) for t in qkv.split((NQ * D, NK * D, NK * D), 1))
    rot = (a["pos"], a["turns"], a["axes"])
    q, k, rq, rk = cake.cake_rotary_fwd(q0, k0, *rot, p["wq"], p["wk"])
    with torch.enable_grad():
        leaves = [t.detach().requires_grad_() for t in (q, k, v)]
        att = attention(*leaves)
    z = att.detach() @ p["o"].t()
    y1, h, r1 = cake.cake_dropout_norm_fwd(z, x, p["w1"], P, a["rng"], 1)
    f, g, u = cake.cake_gated_fwd(y1, p["gate"], p["up"], "gelu")
    out = cake.cake_dropout_fwd(f @ p["down"].t(), P, a["rng"], 2, h)
    dd = cake.cake_dropout_bwd(dy, P, a["rng"], 2)
    dy1, dgate, dup = cake.cake_gated_bwd(dd @ p["down"], y1, g, u, p["gate"], p["up"], "gelu")
    _, dz, dw1 = cake.cake_dropout_norm_bwd(dy1, h, r1, p["w1"], P, a["rng"], 1, dy)
    dq, dk, dv = torch.autograd.grad(att, leaves, dz @ p["o"])
    dq, dk, dwq, dwk = cake.cake_rotary_bwd(dq.contiguous(), dk.contiguous(), *rot, q0, k0, rq, rk, p["wq"], p["wk"])
    dqkv = torch.cat([t.reshape(T, -1) for t in (dq, dk, dv)], 1)
    _, dw0 = cake.cake_rmsnorm_bwd(dqkv @ p["qkv"], x, r0, p["w0"], deterministic=True)
    return out, {"w0": dw0, "qkv": dqkv.t() @ y0, "wq": dwq, "wk": dwk.to(BF16), "o": dz.t() @ att.detach(),
                 "w1": dw1.to(BF16), "gate": dgate, "up": dup, "down": dd.t() @ f}


def test_autograd_run_gives_the_written_out_bits(cake):
    p, a = make(cake)
    y = forward(cake, p, a)
    y.backward(a["dy"])
    y2, want = written_out(cake, p, a)
    torch.cuda.synchronize()
    assert torch.equal(y.detach(), y2)
    for k, v in p.items():
        assert v.grad.dtype == v.dtype
        if k in ("qkv", "o", "down"):  # products of the library, whose operands' layouts differ
            assert torch.allclose(v.grad.float(), want[k].float(), rtol=2.0 ** -6, atol=float(want[k].abs().max()) * 2.0 ** -7), k
        else:
            assert torch.equal(v.grad, want[k]), k


def test_step_in_a_graph(cake):
    p, a = make(cake)
    opt = torch.optim.SGD(list(p.values()), lr=0.05)

    def step():
        opt.zero_grad(set_to_none=True)
        a["rng"][1] += 100  # another mask every step
        forward(cake, p, a).backward(a["dy"])
        norm = cake.cake_clip_grad_norm([v.grad for v in p.values()], 1.0)
        opt.step()
        return norm

    start = {k: v.detach().clone() for k, v in p.items()}
    eager = [float(step()) for _ in range(4)]
    after = {k: v.detach().clone() for k, v in p.items()}
    assert all(n > 0 for n in eager) and len(set(eager)) == 4

    def reset():
        with torch.no_grad():
            a["rng"][1] = 0
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


def test_a_mask_that_changed_before_the_backward_raises(cake):
    p, a = make(cake)
    y = forward(cake, p, a)
    a["rng"][1] += 1
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward(a["dy"])


def _calls(cake, seed, big=False):
    """Inputs, and a call of every operator that reads them and returns what it wrote."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(BF16).to(DEV)  # noqa: E731
    n, h, f = (3000, 640, 1160) if big else (100, 640, 1160)
    ins = {"x": r(n, h), "e": r(n, h), "dy": r(n, h), "wg": r(f, h) * 0.04, "wu": r(f, h) * 0.04, "dh": r(n, f),
           "q": r(n, 10, 64), "k": r(n, 2, 64), "pos": torch.randint(0, 9999, (n,), generator=g).to(DEV)}
    w, wd = torch.ones(h, device=DEV), torch.ones(64, device=DEV)
    turns, _ = cake.cake_rotary_table((32,), device=DEV)
    _, gg, uu = cake.cake_gated_fwd(ins["x"], ins["wg"], ins["wu"])
    _, hn, rstd = cake.cake_dropout_norm_fwd(ins["x"], ins["e"], w, 0.2, 1)
    _, _, rq, rk = cake.cake_rotary_fwd(ins["q"], ins["k"], ins["pos"], turns, None, wd, wd)
    return ins, {
        "gated fwd": ("x", lambda i: cake.cake_gated_fwd(i["x"], i["wg"], i["wu"])),
        "gated fwd, weights": ("wg", lambda i: cake.cake_gated_fwd(i["x"], i["wg"], i["wu"])),
        "gated bwd": ("dh", lambda i: cake.cake_gated_bwd(i["dh"], i["x"], gg, uu, i["wg"], i["wu"])),
        "gated bwd, weights": ("wu", lambda i: cake.cake_gated_bwd(i["dh"], i["x"], gg, uu, i["wg"], i["wu"])),
        "rotary fwd": ("q", lambda i: cake.cake_rotary_fwd(i["q"], i["k"], i["pos"], turns, None, wd, wd)),
        "rotary positions": ("pos", lambda i: cake.cake_rotary_fwd(i["q"], i["k"], i["pos"], turns)[:2]),
        "rotary bwd": ("k", lambda i: cake.cake_rotary_bwd(i["q"], i["k"], i["pos"], turns, None, i["q"].flip(0),
                                                           i["k"].flip(0), rq, rk, wd, wd)),
        "dropout": ("x", lambda i: (cake.cake_dropout_fwd(i["x"], 0.3, 5, 6, i["e"]),)),
        "norm fwd": ("e", lambda i: cake.cake_dropout_norm_fwd(i["x"], i["e"], w, 0.2, 1)),
        "norm bwd": ("dy", lambda i: cake.cake_dropout_norm_bwd(i["dy"], hn, rstd, w, 0.2, 1, dh=i["e"])),
    }


NAMES = ["gated fwd", "gated fwd, weights", "gated bwd", "gated bwd, weights", "rotary fwd", "rotary positions",
         "rotary bwd", "dropout", "norm fwd", "norm bwd"]


@pytest.mark.parametrize("big", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_waits_for_the_work_before(cake, name, big):
    """A call right behind the copy, fill or call that writes its input reads what that has written, eagerly and in a
    graph, and its outputs are whole for the work behind it."""
    ins, calls = _calls(cake, 11, big)
    key, call = calls[name]
    other = _calls(cake, 12, big)[0][key]
    slow = torch.randn(4096, 4096, device=DEV)
    want = {}
    for k, src in (("a", ins[key].clone()), ("b", other), ("zero", torch.zeros_like(other))):
        ins[key].copy_(src)
        torch.cuda.synchronize()
        want[k] = src, [t.clone() for t in call(ins)]
        torch.cuda.synchronize()

    def write(k):
        if k == "zero":
            ins[key].zero_()
        elif ins[key].dtype is BF16:  # by one of the library's own kernels
            rows = want[k][0].view(-1, want[k][0].shape[-1])
            cake.cake_dropout_fwd(rows, 0.0, 1, y=ins[key].view(rows.shape))
        else:
            ins[key].copy_(want[k][0])

    def run():
        got = []
        for k in ("a", "b", "zero", "b", "a"):
            slow @ slow  # work that the writer of the input waits behind
            write(k)
            got.append((k, [t.clone() for t in call(ins)]))
            write("a")  # and one behind the call, over what it has read
        return got

    def check(got):
        torch.cuda.synchronize()
        for k, ts in got:
            for t, w in zip(ts, want[k][1]):
                assert torch.equal(t, w)

    for _ in range(3):
        check(run())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(2):
        graph.replay()
        check(got)


@pytest.mark.parametrize("name", NAMES)
def test_given_streams_and_host_threads(cake, name):
    """Calls of several host threads, each on a stream of its own, give what each gives alone."""
    def work(seed, stream):
        with torch.cuda.stream(stream):
            ins, calls = _calls(cake, seed, seed % 2 == 1)
            got = [[t.clone() for t in calls[name][1](ins)] for _ in range(6)]
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


def test_the_stream_argument(cake):
    ins, _ = _calls(cake, 3)
    w, wd = torch.ones(640, device=DEV), torch.ones(64, device=DEV)
    turns, _ = cake.cake_rotary_table((32,), device=DEV)
    calls = [lambda **k: cake.cake_gated_fwd(ins["x"], ins["wg"], ins["wu"], **k),
             lambda **k: cake.cake_gated_bwd(ins["dh"], ins["x"], ins["dh"] * 2, ins["dh"] * 3, ins["wg"], ins["wu"], **k),
             lambda **k: cake.cake_rotary_fwd(ins["q"], ins["k"], ins["pos"], turns, None, wd, wd, **k),
             lambda **k: cake.cake_dropout_norm_fwd(ins["x"], ins["e"], w, 0.1, 3, **k),
             lambda **k: (cake.cake_dropout_fwd(ins["x"], 0.1, 3, **k), cake.cake_dropout_bwd(ins["x"], 0.1, 3, **k))]
    side = torch.cuda.Stream()
    for call in calls:
        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        got = call(stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_workspaces_may_be_shared_in_order_and_are_checked(cake):
    """One dirty workspace for calls that follow one another, and one that is too small."""
    ins, _ = _calls(cake, 4)
    w, wd = torch.ones(640, device=DEV), torch.ones(64, device=DEV)
    turns, _ = cake.cake_rotary_table((32,), device=DEV)
    _, g, u = cake.cake_gated_fwd(ins["x"], ins["wg"], ins["wu"])
    _, h, rstd = cake.cake_dropout_norm_fwd(ins["x"], ins["e"], w, 0.2, 1)
    _, _, rq, rk = cake.cake_rotary_fwd(ins["q"], ins["k"], ins["pos"], turns, None, wd, wd)
    calls = [lambda **k: cake.cake_gated_bwd(ins["dh"], ins["x"], g, u, ins["wg"], ins["wu"], **k),
             lambda **k: cake.cake_rotary_bwd(ins["q"], ins["k"], ins["pos"], turns, None, ins["q"], ins["k"], rq, rk, wd,
                                              wd, **k),
             lambda **k: cake.cake_dropout_norm_bwd(ins["dy"], h, rstd, w, 0.2, 1, **k)]
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device=DEV)  # NaN as BF16 and as FP32
    want = [[t.clone() for t in c()] for c in calls]
    for _ in range(2):
        for c, v in zip(calls, want):
            assert all(torch.equal(a, b) for a, b in zip(c(workspace=ws), v))
    for c in calls:
        with pytest.raises(cake.CakeError):
            c(workspace=ws[:256])


def test_tensors_that_a_call_writes_count_as_changed(cake):
    ins, _ = _calls(cake, 6)
    n, h, f = 100, 640, 1160
    e = lambda *s: torch.empty(*s, dtype=BF16, device=DEV)  # noqa: E731
    f32 = lambda *s: torch.empty(*s, device=DEV)  # noqa: E731
    w, wd = torch.ones(h, device=DEV), torch.ones(64, device=DEV)
    turns, _ = cake.cake_rotary_table((32,), device=DEV)
    _, g, u = cake.cake_gated_fwd(ins["x"], ins["wg"], ins["wu"])
    _, hn, rstd = cake.cake_dropout_norm_fwd(ins["x"], ins["e"], w, 0.2, 1)
    _, _, rq, rk = cake.cake_rotary_fwd(ins["q"], ins["k"], ins["pos"], turns, None, wd, wd)
    calls = [
        (lambda o: cake.cake_gated_fwd(ins["x"], ins["wg"], ins["wu"], **o), {"h": e(n, f), "g": e(n, f), "u": e(n, f)}),
        (lambda o: cake.cake_gated_bwd(ins["dh"], ins["x"], g, u, ins["wg"], ins["wu"], **o),
         {"dx": e(n, h), "dw_gate": e(f, h), "dw_up": e(f, h)}),
        (lambda o: cake.cake_rotary_fwd(ins["q"], ins["k"], ins["pos"], turns, None, wd, wd, **o),
         {"q_out": e(n, 10, 64), "k_out": e(n, 2, 64), "rstd_q": f32(n * 10), "rstd_k": f32(n * 2)}),
        (lambda o: cake.cake_rotary_bwd(ins["q"], ins["k"], ins["pos"], turns, None, ins["q"], ins["k"], rq, rk, wd, wd,
                                        **o),
         {"dq_out": e(n, 10, 64), "dk_out": e(n, 2, 64), "dw_q": f32(64), "dw_k": f32(64)}),
        (lambda o: cake.cake_dropout_fwd(ins["x"], 0.1, 1, **o), {"y": e(n, h)}),
        (lambda o: cake.cake_dropout_bwd(ins["x"], 0.1, 1, **o), {"dx": e(n, h)}),
        (lambda o: cake.cake_dropout_norm_fwd(ins["x"], ins["e"], w, 0.1, 1, **o),
         {"y": e(n, h), "h_new": e(n, h), "rstd": f32(n)}),
        (lambda o: cake.cake_dropout_norm_bwd(ins["dy"], hn, rstd, w, 0.1, 1, **o),
         {"dx": e(n, h), "dresidual": e(n, h), "dw": f32(h)}),
    ]
    read = [*ins.values(), g, u, hn, rstd, rq, rk, w, wd, turns]
    before = [t._version for t in read]
    for call, outs in calls:
        was = {k: t._version for k, t in outs.items()}
        got = call(outs)
        assert all(t._version > was[k] for k, t in outs.items()), outs.keys()
        got = got if isinstance(got, tuple) else (got,)
        assert {t.data_ptr() for t in outs.values()} == {t.data_ptr() for t in got}
    assert [t._version for t in read] == before


def test_python_refusals(cake):
    """Shapes, types and arguments that do not fit raise before anything is launched."""
    ins, _ = _calls(cake, 7)
    x, wg, wu, q, k, pos = (ins[n] for n in ("x", "wg", "wu", "q", "k", "pos"))
    w, wd = torch.ones(640, device=DEV), torch.ones(64, device=DEV)
    turns, axes = cake.cake_rotary_table((16, 16), device=DEV)
    bad = [
        (ValueError, lambda: cake.cake_gated(x, wg, wu, "relu")), (TypeError, lambda: cake.cake_gated_fwd(x.float(), wg, wu)),
        (ValueError, lambda: cake.cake_gated_fwd(x, wg, wu[:8])), (ValueError, lambda: cake.cake_gated_fwd(x[:, :632], wg, wu)),
        (ValueError, lambda: cake.cake_gated_fwd(x.t().contiguous().t(), wg, wu)),
        (ValueError, lambda: cake.cake_gated_fwd(x, wg, wu, save=False, g=torch.empty_like(ins["dh"]))),
        (cake.CakeError, lambda: cake.cake_gated_fwd(x[:, 4:636], wg[:, 4:636], wu[:, 4:636])),  # not aligned
        (ValueError, lambda: cake.cake_gated_bwd(ins["dh"], x, ins["dh"], ins["dh"], wg, wu, need_dx=False,
                                                 dx=torch.empty_like(x))),
        (ValueError, lambda: cake.cake_rotary_fwd(q, k, pos[:5], turns)), (TypeError, lambda: cake.cake_rotary_fwd(q, k, pos.float(), turns)),
        (ValueError, lambda: cake.cake_rotary_fwd(q, k, pos.expand(2, -1), turns)),  # axes are missing
        (ValueError, lambda: cake.cake_rotary_fwd(q, k, pos, turns, axes[:3])), (TypeError, lambda: cake.cake_rotary_fwd(q, k, pos, turns.float())),
        (ValueError, lambda: cake.cake_rotary_fwd(q, k, pos, turns, style="both")),
        (ValueError, lambda: cake.cake_rotary_fwd(q, k, pos, turns, None, wd)),  # keys without a weight
        (ValueError, lambda: cake.cake_rotary_fwd(q, None, pos, turns, k_out=k)),
        (ValueError, lambda: cake.cake_rotary_fwd(q, k, pos, turns, rstd_q=torch.empty(1000, device=DEV))),
        (ValueError, lambda: cake.cake_rotary_bwd(q, k, pos, turns, None, None, None, None, None, wd, wd)),
        (ValueError, lambda: cake.cake_rotary_fwd(q[0], k, pos, turns)), (ValueError, lambda: cake.cake_rotary_fwd(q, k[:4], pos, turns)),
        (cake.CakeError, lambda: cake.cake_rotary_fwd(q, k, pos, turns[:20])),  # pairs are not a multiple of 8
        (cake.CakeError, lambda: cake.cake_dropout(x, 1.5, 1)), (ValueError, lambda: cake.cake_dropout(x, 0.1, 1, residual=x[:5])),
        (ValueError, lambda: cake.cake_dropout(x, 0.1, torch.zeros(3, dtype=torch.int64, device=DEV))),
        (ValueError, lambda: cake.cake_dropout(x, 0.1, torch.zeros(2, dtype=torch.int64))),  # a seed on the host
        (ValueError, lambda: cake.cake_dropout_norm(x, ins["e"], wd, 0.1, 1)),
        (ValueError, lambda: cake.cake_dropout_norm_bwd(x, x, torch.ones(5, device=DEV), w, 0.1, 1)),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()


def test_no_tokens(cake):
    """Empty batches: nothing to write but zero weight gradients."""
    x, w = torch.empty(0, 64, dtype=BF16, device=DEV), torch.ones(64, device=DEV)
    wg = torch.ones(128, 64, dtype=BF16, device=DEV)
    h, g, u = cake.cake_gated_fwd(x, wg, wg)
    assert h.shape == (0, 128)
    dx, a, b = cake.cake_gated_bwd(h, x, g, u, wg, wg)
    assert dx.shape == (0, 64) and not bool(a.any()) and not bool(b.any())
    q, pos = torch.empty(0, 2, 64, dtype=BF16, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV)
    turns, _ = cake.cake_rotary_table((32,), device=DEV)
    y, z, rq, rk = cake.cake_rotary_fwd(q, q, pos, turns, None, w, w)
    _, _, dwq, dwk = cake.cake_rotary_bwd(y, z, pos, turns, None, q, q, rq, rk, w, w)
    assert y.shape == q.shape and not bool(dwq.any()) and not bool(dwk.any())
    y, h, rstd = cake.cake_dropout_norm_fwd(x, x, w, 0.1, 1)
    dres, dx, dw = cake.cake_dropout_norm_bwd(y, h, rstd, w, 0.1, 1)
    assert dx.shape == x.shape and not bool(dw.any()) and cake.cake_dropout_fwd(x, 0.1, 1).shape == x.shape
