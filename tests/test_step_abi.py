"""The C ABI and the Python names of the training-step operators without a
GPU: the library exports what the header declares, sizes are what a caller can
count on, and arguments outside the documented ranges are refused before any
launch.  No call here reaches a kernel."""
import ctypes
import os
import random
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
A = 1 << 20  # an aligned address that is never followed
MB = 1 << 20


@pytest.fixture(scope="module")
def cake():
    from bwd_dw_column_gb300 import _build
    _build.build()
    import bwd_dw_column_gb300 as cake
    cake.load_library()
    return cake


def _declared():
    text = open(os.path.join(ROOT, "include", "cake_step.h")).read()
    return sorted(set(re.findall(r"\b(cake_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S))))


def test_library_exports_every_declared_symbol(cake):
    names = _declared()
    assert len(names) == 9
    for n in names:
        assert hasattr(cake.load_library(), n), n


def test_python_names(cake):
    from bwd_dw_column_gb300 import step
    for n in step.__all__:
        assert n in cake.__all__ and callable(getattr(cake, n))


def S(T, nh=1, H=64):
    from bwd_dw_column_gb300 import _Shape
    return ctypes.byref(_Shape(T, nh, H))


def V(at, st=64, sh=0):
    from bwd_dw_column_gb300 import _Tensor
    return ctypes.byref(_Tensor(at, st, sh))


def fwd(cake, shape=None, z=None, x=None, w1=A, d1=0, w2=A, d2=0, grow=None, gate=None, scale=1.0, eps=1e-6, y=None,
        h=None, r1=A, r2=A + MB):
    return cake.load_library().cake_sandwich_fwd(shape or S(4), z or V(A), x or V(A + MB), w1, d1, w2, d2, grow, gate,
                                                 scale, eps, y or V(A + 2 * MB), h or V(A + 3 * MB), r1, r2, None)


def test_sandwich_fwd_refusals(cake):
    nan = float("nan")
    assert fwd(cake, S(-1)) == INVALID and fwd(cake, S(4, 0)) == INVALID
    assert fwd(cake, S(4, 1, 60)) == UNSUPPORTED and fwd(cake, S(4, 1, 8200)) == UNSUPPORTED
    assert fwd(cake, S(1 << 31)) == UNSUPPORTED
    assert fwd(cake, eps=-1.0) == INVALID and fwd(cake, eps=nan) == INVALID and fwd(cake, scale=nan) == INVALID
    assert fwd(cake, w1=None) == INVALID and fwd(cake, w1=A + 8) == UNSUPPORTED
    assert fwd(cake, d1=2) == INVALID and fwd(cake, d2=-1) == INVALID
    assert fwd(cake, z=V(0)) == INVALID and fwd(cake, z=V(A + 2)) == UNSUPPORTED
    assert fwd(cake, x=V(A + MB, 60)) == UNSUPPORTED and fwd(cake, x=V(A + MB, 0)) == UNSUPPORTED
    assert fwd(cake, r1=None) == INVALID and fwd(cake, r2=A + 2) == UNSUPPORTED
    assert fwd(cake, grow=A, gate=V(A + 5 * MB)) == INVALID
    assert fwd(cake, grow=A + 2) == UNSUPPORTED and fwd(cake, gate=V(A + 5 * MB + 8)) == UNSUPPORTED
    assert fwd(cake, r2=A) == INVALID and fwd(cake, r2=A + 8) == INVALID  # rstd_pre reaches into rstd_post
    assert fwd(cake, y=V(A + 3 * MB)) == INVALID            # y and h_new are one
    assert fwd(cake, h=V(A + MB + 128)) == INVALID          # h_new straddles x's rows
    assert fwd(cake, S(4, 2), z=V(A, 128, 64), x=V(A + MB, 128, 64), y=V(A + 2 * MB, 64, 64)) == INVALID  # rows overlap
    assert fwd(cake, S(0), z=V(0), w1=None) == 0            # no rows: nothing to do


def bwd(cake, shape=None, dy=None, dh=None, h=None, z=None, r1=A, r2=A, w1=A, w2=A, grow=None, gate=None, dx=None,
        dz=None, dwo=A, dwr=A + 4096, dgr=None, dg=None, ws=A, n=1 << 30, scale=1.0):
    return cake.load_library().cake_sandwich_bwd(
        shape or S(4), dy or V(A), dh, h or V(A + MB), z or V(A + 2 * MB), r1, r2, w1, 0, w2, 1, grow, gate, scale,
        dx or V(A + 3 * MB), dz or V(A + 4 * MB), dwo, dwr, dgr, dg, ws, n, None)


def test_sandwich_bwd_refusals(cake):
    assert bwd(cake, S(4, 1, 12)) == UNSUPPORTED
    assert bwd(cake, dwo=None) == INVALID and bwd(cake, dwr=A) == INVALID and bwd(cake, dwo=A + 4) == UNSUPPORTED
    assert bwd(cake, dwr=A + 128) == INVALID                # dw_pre reaches into dw_post
    assert bwd(cake, dgr=A) == INVALID and bwd(cake, dg=V(A + 5 * MB)) == INVALID   # a gradient of no gate
    assert bwd(cake, grow=A, dgr=A + 2) == UNSUPPORTED
    assert bwd(cake, dx=V(A)) == INVALID and bwd(cake, dz=V(A + 2 * MB)) == INVALID  # in place
    assert bwd(cake, dz=V(A + 3 * MB)) == INVALID
    assert bwd(cake, gate=V(A + 5 * MB), dg=V(A + 5 * MB)) == INVALID
    assert bwd(cake, dh=V(A + 3 * MB)) == INVALID
    assert bwd(cake, r1=None) == INVALID and bwd(cake, z=V(0)) == INVALID
    assert bwd(cake, ws=None) == WORKSPACE and bwd(cake, n=16) == WORKSPACE and bwd(cake, ws=A + 16) == UNSUPPORTED
    assert cake.cake_sandwich_bwd_workspace_size((0, 1, 64)) == 0
    assert cake.cake_sandwich_bwd_workspace_size((4, 1, 60)) == 0
    assert cake.cake_sandwich_bwd_workspace_size((4, 1, 64)) > 0


def test_every_width_has_a_backward_plan(cake):
    for H in range(8, 8193, 8):
        for T in (1, 151, 100_000):
            assert cake.cake_sandwich_bwd_workspace_size((T, 1, H)) >= 16 * H, (T, H)


def plan(cake, T, H, tensors):
    got = (ctypes.c_int * 9)()
    assert cake.load_library().cake_sandwich_bwd_plan(S(T, 1, H), tensors, got) == 0
    return tuple(got)


def test_every_build_of_the_backward_is_reached(cake):
    """The library holds the kernels that some width takes, for each gate, and no others."""
    names = subprocess.run(["nm", "-C", cake.LIB_PATH], capture_output=True, text=True, check=True).stdout
    held = set(re.findall(r"cake::sandwich_bwd_kernel<(\d+), (\d+), (\w+), (\d+), (\w+), (\w+)>", names))
    flag = ("false", "true")
    taken = set()
    for gate in (0, 1, 2):
        for H in range(8, 8193, 8):
            for dh in (0, 1):
                vpt, cl, rw, many, half = plan(cake, 100_000, H, 3 + (gate == 2) + dh)[:5]
                taken.add((str(vpt), str(gate), flag[cl], str(rw), flag[many], flag[half]))
    assert held and held == taken, (sorted(held - taken), sorted(taken - held))


@pytest.mark.parametrize("tensors", [4, 5])
def test_the_tested_cluster_shapes_come_round_several_times(cake, tensors):
    for H in (4104, 5120, 6144, 7168, 8192):  # (3080 columns stay on one CTA)
        cluster, _, stages, tiles = plan(cake, 2999, H, tensors)[5:]
        assert cluster > 1 and tiles >= 9 and tiles >= 2 * stages, H


def test_plan_refusals(cake):
    got, call = (ctypes.c_int * 9)(), cake.load_library().cake_sandwich_bwd_plan
    assert call(S(4), 2, got) == INVALID and call(S(4), 6, got) == INVALID and call(S(0), 3, got) == INVALID
    assert call(S(4), 3, None) == INVALID and call(S(4, 1, 60), 3, got) == UNSUPPORTED


def grads(cake, ptrs, counts, types, outs=None, otypes=None, max_norm=1.0, eps=1e-6, norm=A // 2, ws=A, n_ws=1 << 30,
          clip=True):
    n = len(ptrs)
    arr = lambda t, v: (t * max(n, 1))(*v)  # noqa: E731
    p, c, d = arr(ctypes.c_void_p, ptrs), arr(ctypes.c_int64, counts), arr(ctypes.c_int32, types)
    lib = cake.load_library()
    if not clip:
        return lib.cake_grad_norm(p, c, d, n, norm, ws, n_ws, None)
    return lib.cake_grad_clip(p, c, d, arr(ctypes.c_void_p, outs) if outs else None,
                              arr(ctypes.c_int32, otypes) if otypes else None, n, max_norm, eps, norm, ws, n_ws, None)


def test_grad_refusals(cake):
    B, C = A + MB, A + 2 * MB
    assert grads(cake, [A], [-1], [0]) == INVALID and grads(cake, [0], [4], [0]) == INVALID
    assert grads(cake, [A], [4], [2]) == INVALID
    assert grads(cake, [A + 2], [4], [1]) == UNSUPPORTED and grads(cake, [A + 1], [4], [0]) == UNSUPPORTED
    for bad in (-1.0, float("nan")):
        assert grads(cake, [A], [4], [0], max_norm=bad) == INVALID
        assert grads(cake, [A], [4], [0], eps=bad) == INVALID
    assert grads(cake, [A, A], [4, 4], [0, 0]) == INVALID                 # one tensor twice
    assert grads(cake, [A, A + 6], [4, 4], [0, 0]) == INVALID             # they overlap
    assert grads(cake, [B, A], [4, (1 << 19) + 1], [0, 0]) == INVALID
    assert grads(cake, [A], [4], [0], outs=[B]) == INVALID                # outputs without types
    assert grads(cake, [A], [4], [0], outs=[0], otypes=[0]) == INVALID
    assert grads(cake, [A], [4], [0], outs=[B + 2], otypes=[1]) == UNSUPPORTED
    assert grads(cake, [A], [8], [0], outs=[A], otypes=[1]) == INVALID    # its own input, but wider
    assert grads(cake, [A], [8], [0], outs=[A + 2], otypes=[0]) == INVALID
    assert grads(cake, [A, B], [8, 8], [0, 0], outs=[C, C + 14], otypes=[0, 0]) == INVALID
    assert grads(cake, [A, B], [8, 8], [0, 0], outs=[B, A], otypes=[0, 0]) == INVALID
    assert grads(cake, [A], [4], [0], norm=None) == INVALID
    assert grads(cake, [A], [4], [0], ws=None) == WORKSPACE and grads(cake, [A], [4], [0], n_ws=8) == WORKSPACE
    assert grads(cake, [A], [4], [0], ws=A + 8) == UNSUPPORTED
    assert grads(cake, [A], [4], [0], norm=None, clip=False) == INVALID
    assert grads(cake, [A], [1 << 46], [0], clip=False) == UNSUPPORTED
    assert grads(cake, [A] * 4000, [1 << 34] * 4000, [0] * 4000, clip=False) == UNSUPPORTED  # 2^32 chunks and more
    for at in (B, B + 8, B + 12):  # the norm lies in an output
        assert grads(cake, [A], [8], [0], outs=[B], otypes=[0], norm=at) == INVALID
    assert grads(cake, [A], [8], [0], norm=A + 4) == INVALID
    lib = cake.load_library()
    assert lib.cake_grad_norm(A, A, A, 1 << 60, A, A, 1 << 30, None) == UNSUPPORTED  # nothing of the lists is read
    assert lib.cake_grad_norm_workspace_size(1 << 60) == 0
    assert cake.cake_grad_norm_workspace_size(0) == 0
    assert cake.cake_grad_norm_workspace_size(5000) > cake.cake_grad_norm_workspace_size(1) > 0


def efwd(cake, ids=A, i64=1, T=4, table=A + MB, dt=0, vocab=10, H=64, stride=64, scale=1.0, y=None):
    return cake.load_library().cake_embedding_fwd(ids, i64, T, table, dt, vocab, H, stride, scale,
                                                  y or V(A + 2 * MB), None)


def ebwd(cake, dy=None, ids=A, i64=1, T=4, vocab=10, H=64, scale=1.0, pad=-1, out=A + MB, dt=1, stride=64, acc=0, ws=A,
         n=1 << 30):
    return cake.load_library().cake_embedding_bwd(dy or V(A + 2 * MB), ids, i64, T, vocab, H, scale, pad, out, dt,
                                                  stride, acc, ws, n, None)


@pytest.mark.parametrize("call", [efwd, ebwd])
def test_embedding_refusals(cake, call):
    assert call(cake, ids=None) == INVALID and call(cake, T=-1) == INVALID and call(cake, vocab=0) == INVALID
    assert call(cake, i64=2) == INVALID and call(cake, dt=3) == INVALID and call(cake, scale=float("nan")) == INVALID
    assert call(cake, H=60) == UNSUPPORTED and call(cake, H=8200) == UNSUPPORTED
    assert call(cake, T=1 << 31) == UNSUPPORTED and call(cake, vocab=1 << 31) == UNSUPPORTED
    assert call(cake, stride=56) == UNSUPPORTED and call(cake, stride=66, dt=0) == UNSUPPORTED
    assert call(cake, ids=A + 4) == UNSUPPORTED and call(cake, ids=A + 2, i64=0) == UNSUPPORTED
    rows = "y" if call is efwd else "dy"
    assert call(cake, **{rows: V(0)}) == INVALID and call(cake, **{rows: V(A + 2 * MB + 8)}) == UNSUPPORTED
    assert call(cake, **{rows: V(A + MB + 256)}) == INVALID  # the rows lie in the table


def test_embedding_bwd_refusals(cake):
    assert ebwd(cake, pad=-2) == INVALID and ebwd(cake, pad=10) == INVALID
    assert ebwd(cake, ws=None) == WORKSPACE and ebwd(cake, n=64) == WORKSPACE and ebwd(cake, ws=A + 8) == UNSUPPORTED
    assert ebwd(cake, out=None) == INVALID and ebwd(cake, out=A + MB + 8) == UNSUPPORTED
    assert cake.cake_embedding_bwd_workspace_size(0, 10, 64) == 0
    small, large = (cake.cake_embedding_bwd_workspace_size(T, 1000, 64) for T in (1, 100000))
    assert 0 < small < large


@pytest.mark.parametrize("shift", [0, 16, -16])
def test_written_memory_is_shared_with_nothing(cake, shift):
    """Every pair of a written tensor and another one that meet is refused (but forward rows in place)."""
    far = [(20 + k) * MB for k in range(16)]
    # 4 rows of 64 values: 512 bytes a tensor, 16 bytes a list of rows, 128 or 256 a weight
    at = dict(zip(("z", "x", "gate", "y", "h", "w1", "w2", "r1", "r2", "dy", "dh", "dgr", "dwo", "dwr", "grow", "ws"), far))

    def forward(row_gate, **moved):
        a = {**at, **moved}
        gate = {"grow": a["grow"]} if row_gate else {"gate": V(a["gate"])}
        return fwd(cake, z=V(a["z"]), x=V(a["x"]), y=V(a["y"]), h=V(a["h"]), w1=a["w1"], w2=a["w2"], r1=a["r1"],
                   r2=a["r2"], **gate)

    def meets(place):  # where a tensor of more than 16 bytes starts that reaches into the one at `place`
        return place + min(shift, 0)

    for out in ("r1", "r2"):
        for other in ("z", "x", "y", "h", "w1", "w2"):
            assert forward(True, **{out: at[other] + max(shift, 0)}) == INVALID, (out, other)
        assert forward(True, **{out: at["grow"] + (4 if shift else 0)}) == INVALID
        assert forward(False, **{out: at["gate"] + max(shift, 0)}) == INVALID
    for out in ("y", "h"):
        for other in ("w1", "w2", "grow"):
            assert forward(True, **{out: meets(at[other])}) == INVALID, (out, other)

    names = ("dx", "dz", "dwo", "dwr", "dgr")

    def backward(**moved):
        a = {**at, "dx": 40 * MB, "dz": 41 * MB, **moved}
        return bwd(cake, dy=V(a["dy"]), dh=V(a["dh"]), h=V(a["h"]), z=V(a["z"]), r1=a["r1"], r2=a["r2"], w1=a["w1"],
                   w2=a["w2"], grow=a["grow"], dx=V(a["dx"]), dz=V(a["dz"]), dwo=a["dwo"], dwr=a["dwr"], dgr=a["dgr"],
                   ws=a["ws"])

    places = {**at, "dx": 40 * MB, "dz": 41 * MB}
    for out in names:
        for other in ("dy", "dh", "h", "z", "r1", "r2", "w1", "w2", "grow", "dx", "dz", "dwo", "dwr", "dgr", "ws"):
            if out != other:
                to = places[other] if out == "dgr" else meets(places[other])
                assert backward(**{out: to}) == INVALID, (out, other)
    for other in ("dy", "dh", "h", "z", "r1", "r2", "w1", "w2", "grow"):
        assert backward(ws=places[other]) == INVALID, other


def test_columns_of_one_buffer_share_nothing(cake):
    """Rows that interleave: taken to meet exactly where bytes of them do."""
    T, H, B = 4, 64, 64 * MB
    rng, seen = random.Random(0), set()

    def meet(a, b, nh=1):
        return bool(cake.load_library().cake_step_rows_meet(S(T, nh, H), V(*a), V(*b)))

    def rows(at, st, sh, nh):
        return [at + 2 * (t * st + k * sh) for t in range(T) for k in range(nh)]

    for _ in range(4000):
        nh, sh = rng.choice([1, 2, 3]), 8 * rng.randint(8, 28)
        a = (B, nh * sh, sh)
        b = (B + 16 * rng.randint(-300, 300), nh * sh, sh)
        want = any(abs(p - q) < 2 * H for p in rows(*a, nh) for q in rows(*b, nh))
        got = meet(a, b, nh)
        inner = 0 < abs(b[0] - a[0]) < 2 * T * nh * sh - 4 * H  # (past the ends, extents alone decide)
        assert got == want or (got and not inner), (a, b, nh)
        seen.add((nh > 1, got))
    assert len(seen) == 4
    # rows of unlike strides, and heads that are not equally spaced, are taken as all that they span
    assert meet((B, 128, 0), (B + 128, 256, 0)) and not meet((B, 128, 0), (B + 1024, 256, 0))
    assert meet((B, 512, 128), (B + 128, 512, 128), 2)


def test_scratch_and_ids_are_shared_with_nothing(cake):
    B, C = A + MB, A + 2 * MB
    for n in (100, 1 << 18):
        assert grads(cake, [B], [n], [1], ws=B + 256) == INVALID
        assert grads(cake, [B], [n], [1], ws=B, clip=False) == INVALID
    assert grads(cake, [A], [4], [0], outs=[B], otypes=[1], ws=B) == INVALID
    assert grads(cake, [A], [4], [0], norm=C + 64, ws=C) == INVALID
    assert efwd(cake, ids=A + 2 * MB + 8) == INVALID and efwd(cake, ids=A + 2 * MB - 8) == INVALID
    assert ebwd(cake, ids=A + MB + 8, ws=32 * MB) == INVALID and ebwd(cake, ids=A + MB - 8, ws=32 * MB) == INVALID
    for place in (A, A + MB, A + 2 * MB):  # ids, dtable, dy
        assert ebwd(cake, ws=place) == INVALID


@pytest.mark.parametrize("clip", [False, True])
@pytest.mark.parametrize("count,dtype", [(8, 0), (8, 1), (1 << 18, 0), (1, 1)])
def test_the_norm_lies_in_no_gradient(cake, count, dtype, clip):
    """A norm inside a tensor that the call reads would overwrite some of its values."""
    B = A + MB
    size = 4 if dtype else 2
    for at in sorted({B, B + max(0, (count * size // 2) // 4 * 4), B + max(0, count * size - 4)}):
        assert grads(cake, [A + 2 * MB, B], [4, count], [0, dtype], norm=at, ws=16 * MB, clip=clip) == INVALID, at


def test_python_refusals_without_a_gpu(cake):
    z = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64)
    for call in (lambda: cake.cake_sandwich_norm(z, z, w, w), lambda: cake.cake_grad_norm([z]),
                 lambda: cake.cake_clip_grad_norm([z], 1.0),
                 lambda: cake.cake_embedding(torch.zeros(3, dtype=torch.int64), z),
                 lambda: cake.cake_embedding_bwd(z, torch.zeros(4, dtype=torch.int64), 10)):
        with pytest.raises(ValueError):  # no CPU path
            call()
