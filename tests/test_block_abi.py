"""The C ABI and the Python names of a block's operators without a GPU: the
library exports what the header declares, and arguments outside the documented
ranges are refused before any launch.  No call here reaches a kernel."""
import ctypes
import os
import re
import struct

import pytest
import torch

from bwd_dw_column_gb300.step import _three

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
MB = 1 << 20
NAN = float("nan")
_rotation = struct.Struct("=qqQQQixxxxqqixxxx").pack  # cake_rotary


@pytest.fixture(scope="module")
def cake():
    from bwd_dw_column_gb300 import _build
    _build.build()
    import bwd_dw_column_gb300 as cake
    cake.load_library()
    return cake


def test_library_exports_every_declared_symbol(cake):
    names = set()
    for header in ("cake_block.h", "cake_block_test.h"):
        text = open(os.path.join(ROOT, "include", header)).read()
        names |= set(re.findall(r"\b(cake_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert len(names) == 12
    for n in names:
        assert hasattr(cake.load_library(), n), n


def test_python_names(cake):
    from bwd_dw_column_gb300 import block
    for n in block.__all__:
        assert n in cake.__all__ and callable(getattr(cake, n))


def V(at, st=64, sh=0):
    return _three(at, st, sh)


# ------------------------------------------------------------------------ gated

AT = dict(zip(("x", "wg", "wu", "h", "g", "u", "dh", "dx", "dwg", "dwu"), range(MB, 11 * MB, MB)))


def gfwd(cake, T=4, H=64, F=128, act=0, save=True, **at):
    a = {**AT, **at}
    v = lambda n, st: V(*a[n]) if isinstance(a[n], tuple) else V(a[n], st)  # noqa: E731
    return cake.load_library().cake_gated_fwd(T, H, F, v("x", H), v("wg", H), v("wu", H), act, v("h", F),
                                              v("g", F) if save else None, v("u", F) if save else None, None)


def gbwd(cake, T=4, H=64, F=128, act=0, ws=64 * MB, n=1 << 40, with_dx=True, with_dw=True, **at):
    a = {**AT, **at}
    v = lambda n, st: V(*a[n]) if isinstance(a[n], tuple) else V(a[n], st)  # noqa: E731
    return cake.load_library().cake_gated_bwd(T, H, F, v("dh", F), v("x", H), v("g", F), v("u", F), v("wg", H),
                                              v("wu", H), act, v("dx", H) if with_dx else None,
                                              v("dwg", H) if with_dw else None, v("dwu", H) if with_dw else None, ws, n, None)


@pytest.mark.parametrize("call", [gfwd, gbwd])
def test_gated_refusals(cake, call):
    assert call(cake, T=-1) == INVALID and call(cake, H=0) == INVALID and call(cake, F=0) == INVALID
    assert call(cake, act=2) == INVALID and call(cake, act=-1) == INVALID
    assert call(cake, H=60) == UNSUPPORTED and call(cake, F=100) == UNSUPPORTED
    assert call(cake, H=131080) == UNSUPPORTED and call(cake, F=131080) == UNSUPPORTED
    assert call(cake, T=1 << 28) == UNSUPPORTED
    for n in ("x", "wg", "wu"):
        assert call(cake, **{n: 0}) == INVALID and call(cake, **{n: AT[n] + 8}) == UNSUPPORTED
        assert call(cake, **{n: (AT[n], 56)}) == UNSUPPORTED and call(cake, **{n: (AT[n], 68)}) == UNSUPPORTED
        assert call(cake, **{n: (AT[n], -64)}) == UNSUPPORTED and call(cake, **{n: (AT[n], 1 << 36)}) == UNSUPPORTED


def test_gated_outputs_share_memory_with_nothing(cake):
    for shift in (0, 64, -64):
        for out in ("h", "g", "u"):
            for other in ("x", "wg", "wu", "h", "g", "u"):
                if out != other:
                    assert gfwd(cake, **{out: AT[other] + shift}) == INVALID, (out, other)
        for out in ("dx", "dwg", "dwu"):
            for other in ("dh", "x", "g", "u", "wg", "wu", "dx", "dwg", "dwu"):
                if out != other:
                    assert gbwd(cake, **{out: AT[other] + shift}) == INVALID, (out, other)
    for other in ("dh", "x", "g", "u", "wg", "wu", "dx", "dwg", "dwu"):
        assert gbwd(cake, ws=AT[other]) == INVALID, other
    lib = cake.load_library()
    assert lib.cake_gated_fwd(4, 64, 128, V(MB), V(2 * MB), V(3 * MB), 0, V(4 * MB, 128), V(5 * MB, 128), None,
                              None) == INVALID  # g without u
    assert gbwd(cake, ws=None) == WORKSPACE and gbwd(cake, n=100) == WORKSPACE and gbwd(cake, ws=64 * MB + 8) == UNSUPPORTED
    assert gfwd(cake, T=0, x=0, h=0) == 0 and gbwd(cake, T=0, with_dw=False) == 0 and gbwd(cake, with_dx=False, with_dw=False) == 0
    assert cake.cake_gated_bwd_workspace_size(0, 64, 64) == cake.cake_gated_bwd_workspace_size(4, 60, 64) == 0
    assert cake.cake_gated_bwd_workspace_size(4, 64, 64) >= 2 * 4 * 64 * 2


# ----------------------------------------------------------------------- rotary

RAT = dict(zip(("q", "k", "qo", "ko", "wq", "wk", "rq", "rk", "turns", "axis", "pos", "dq", "dk", "dwq", "dwk"),
               range(MB, 16 * MB, MB)))
T, NQ, NK, D = 4, 6, 2, 64


def rotation(a, pairs=32, axes=2, i64=1, ast=T, tst=1, style=0):
    return _rotation(pairs, axes, a["turns"], a["axis"], a["pos"], i64, ast, tst, style)


def rfwd(cake, tokens=T, nq=NQ, nk=NK, hidden=D, eps=1e-6, dq=0, dk=1, rot=None, **at):
    a = {**RAT, **at}
    v = lambda n, heads: V(*a[n]) if isinstance(a[n], tuple) else V(a[n], heads * D, D) if a[n] is not None else None  # noqa: E731
    return cake.load_library().cake_rotary_fwd(tokens, nq, nk, hidden, v("q", NQ), v("k", NK), rotation(a, **(rot or {})),
                                               a["wq"], dq, a["wk"], dk, eps, v("qo", NQ), v("ko", NK), a["rq"],
                                               a["rk"], None)


def rbwd(cake, tokens=T, nq=NQ, nk=NK, hidden=D, ws=64 * MB, n=1 << 30, rot=None, **at):
    a = {**RAT, **at}
    v = lambda n, heads: V(*a[n]) if isinstance(a[n], tuple) else V(a[n], heads * D, D) if a[n] is not None else None  # noqa: E731
    return cake.load_library().cake_rotary_bwd(tokens, nq, nk, hidden, v("dq", NQ), v("dk", NK), rotation(a, **(rot or {})),
                                               v("q", NQ), v("k", NK), a["rq"], a["rk"], a["wq"], 0, a["wk"], 1,
                                               v("qo", NQ), v("ko", NK), a["dwq"], a["dwk"], ws, n, None)


@pytest.mark.parametrize("call", [rfwd, rbwd])
def test_rotary_refusals(cake, call):
    assert call(cake, tokens=-1) == INVALID and call(cake, nq=0) == INVALID and call(cake, nk=-1) == INVALID
    assert call(cake, hidden=0) == INVALID and call(cake, hidden=72) == UNSUPPORTED and call(cake, hidden=528) == UNSUPPORTED
    assert call(cake, tokens=1 << 31) == UNSUPPORTED
    for bad in ({"pairs": -8}, {"axes": 0}, {"style": 2}, {"style": -1}, {"ast": -1}, {"tst": -1}, {"i64": 2}):
        assert call(cake, rot=bad) == INVALID, bad
    for bad in ({"pairs": 12}, {"pairs": 40}, {"axes": 17}):
        assert call(cake, rot=bad) == UNSUPPORTED, bad
    assert call(cake, turns=0) == INVALID and call(cake, pos=0) == INVALID and call(cake, axis=0) == INVALID
    assert call(cake, turns=RAT["turns"] + 4) == UNSUPPORTED and call(cake, axis=RAT["axis"] + 2) == UNSUPPORTED
    assert call(cake, pos=RAT["pos"] + 4) == UNSUPPORTED
    assert call(cake, wk=None) == INVALID and call(cake, wq=RAT["wq"] + 8) == UNSUPPORTED
    assert call(cake, rq=None) == INVALID and call(cake, rk=RAT["rk"] + 2) == UNSUPPORTED
    for n in ("q", "k", "qo", "ko"):
        assert call(cake, **{n: (0, 384, 64)}) == INVALID
        assert call(cake, **{n: (RAT[n] + 8, 384, 64)}) == UNSUPPORTED and call(cake, **{n: (RAT[n], 384, 60)}) == UNSUPPORTED
    assert call(cake, qo=(RAT["qo"], 64, 64)) == INVALID  # its heads overlap


def test_rotary_outputs_share_memory_with_nothing(cake):
    assert rfwd(cake, eps=-1.0) == INVALID and rfwd(cake, eps=NAN) == INVALID and rfwd(cake, dq=2) == INVALID
    for out, own in (("qo", "q"), ("ko", "k")):
        for other in ("q", "k", "qo", "ko", "wq", "wk", "rq", "rk", "turns", "axis", "pos"):
            if other not in (out, own):
                assert rfwd(cake, **{out: RAT[other]}) == INVALID, (out, other)
        assert rfwd(cake, **{out: RAT[own] + 128}) == INVALID  # not exactly its own input
    for out in ("rq", "rk"):
        for other in ("q", "k", "qo", "ko", "wq", "wk", "turns", "axis", "pos"):
            assert rfwd(cake, **{out: RAT[other]}) == INVALID, (out, other)
    assert rfwd(cake, rq=RAT["rk"]) == INVALID
    for out, own in (("qo", "dq"), ("ko", "dk")):
        for other in ("q", "k", "qo", "ko", "wq", "wk", "rq", "rk", "turns", "axis", "pos", "dq", "dk", "dwq", "dwk"):
            if other not in (out, own):
                assert rbwd(cake, **{out: RAT[other]}) == INVALID, (out, other)
    for out in ("dwq", "dwk"):
        for other in ("q", "k", "qo", "ko", "wq", "wk", "rq", "rk", "turns", "axis", "pos", "dq", "dk"):
            assert rbwd(cake, **{out: RAT[other]}) == INVALID, (out, other)
    assert rbwd(cake, dwq=RAT["dwk"]) == INVALID and rbwd(cake, dwq=None) == INVALID
    assert rbwd(cake, dwq=RAT["dwq"] + 8) == UNSUPPORTED
    for other in RAT:
        assert rbwd(cake, ws=RAT[other]) == INVALID, other
    assert rbwd(cake, ws=None) == WORKSPACE and rbwd(cake, n=64) == WORKSPACE and rbwd(cake, ws=64 * MB + 16) == UNSUPPORTED


def test_heads_of_one_fused_product(cake):
    """Queries, keys and values side by side in one row: outputs over other columns of it are not refused for their
    memory (a bad workspace or weight is found after that check or before it), those that meet are."""
    wide = (NQ + 2 * NK) * D
    at = 20 * MB
    q, k = (at, wide, D), (at + 2 * NQ * D, wide, D)
    # (every other argument is right, so only a null weight's refusal shows that memory passed)
    assert rbwd(cake, dq=q, dk=k, qo=q, ko=k, ws=None) == WORKSPACE
    assert rfwd(cake, q=q, k=k, qo=q, ko=(at + 2 * (NQ - 1) * D, wide, D)) == INVALID  # reaches into a head of q
    assert rfwd(cake, q=q, k=k, qo=k, ko=q) == INVALID
    assert rfwd(cake, q=q, k=k, qo=(at + 2 * NK * D, wide, D), ko=(at + 2 * wide * T * 4, wide, D)) == INVALID


def test_rotary_sizes(cake):
    size = cake.cake_rotary_bwd_workspace_size
    assert size(0, 4, 2, 64) == size(4, 0, 2, 64) == size(4, 4, 2, 60) == 0
    for t in (1, 77, 100000):
        for n, m in ((1, 0), (24, 4), (4, 24)):
            for d in (16, 48, 512):
                assert size(t, n, m, d) >= (2 if m else 1) * d * 8


def test_a_share_for_every_warp(cake):
    """The plan's CTAs are no more than what runs at a time, and no list with rows is left out."""
    for t in (1, 3, 1000, 1 << 20):
        for n, m in ((1, 1), (64, 1), (1, 64), (24, 4)):
            ctas = cake.cake_rotary_bwd_workspace_size(t, n, m, 128) // (128 * 8)
            assert 2 <= ctas <= 305, (t, n, m, ctas)


# ---------------------------------------------------------------------- dropout

DAT = dict(zip(("x", "e", "y", "h", "w", "rstd", "rng", "dy", "dh", "dx", "dres", "dw"), range(MB, 13 * MB, MB)))
S = _three(4, 1, 64)


def plain(cake, shape=S, p=0.1, rng=None, **at):
    a = {**DAT, **at}
    v = lambda n: V(*a[n]) if isinstance(a[n], tuple) else V(a[n])  # noqa: E731
    return cake.load_library().cake_dropout(shape, v("x"), v("e"), p, 1, 2, rng, v("y"), None)


def nfwd(cake, shape=S, p=0.1, rng=None, eps=1e-6, dt=0, **at):
    a = {**DAT, **at}
    v = lambda n: V(*a[n]) if isinstance(a[n], tuple) else V(a[n])  # noqa: E731
    return cake.load_library().cake_dropout_norm_fwd(shape, v("x"), v("e"), a["w"], dt, p, 1, 2, rng, eps, v("y"),
                                                     v("h"), a["rstd"], None)


def nbwd(cake, shape=S, p=0.1, rng=None, dt=0, ws=64 * MB, n=1 << 30, **at):
    a = {**DAT, **at}
    v = lambda n: V(*a[n]) if isinstance(a[n], tuple) else V(a[n]) if a[n] else None  # noqa: E731
    return cake.load_library().cake_dropout_norm_bwd(shape, v("dy"), v("dh"), v("h"), a["rstd"], a["w"], dt, p, 1, 2,
                                                     rng, v("dx"), v("dres"), a["dw"], ws, n, None)


@pytest.mark.parametrize("call", [plain, nfwd, nbwd])
def test_dropout_refusals(cake, call):
    assert call(cake, _three(-1, 1, 64)) == INVALID and call(cake, _three(4, 0, 64)) == INVALID
    assert call(cake, _three(4, 1, 60)) == UNSUPPORTED and call(cake, _three(4, 1, 8200)) == UNSUPPORTED
    assert call(cake, _three(1 << 31, 1, 64)) == UNSUPPORTED
    for bad in (-0.1, 1.1, NAN):
        assert call(cake, p=bad) == INVALID
    assert call(cake, rng=DAT["rng"] + 4) == UNSUPPORTED
    ins = {plain: ("x", "e"), nfwd: ("x", "e"), nbwd: ("dy", "dh", "h")}[call]
    outs = {plain: ("y",), nfwd: ("y", "h"), nbwd: ("dx", "dres")}[call]
    for n in ins + outs:
        assert call(cake, **{n: (DAT[n] + 8,)}) == UNSUPPORTED and call(cake, **{n: (DAT[n], 56)}) == UNSUPPORTED
    for n in outs:
        assert call(cake, **{n: (0,)}) == INVALID
        for other in ins:  # rows of an output straddle an input's
            assert call(cake, **{n: DAT[other] + 64}) == INVALID, (n, other)
        assert call(cake, rng=DAT[n]) == INVALID
        if call is not plain:
            assert call(cake, **{n: DAT["w"]}) == INVALID and call(cake, **{n: DAT["rstd"]}) == INVALID
    if call is not plain:
        assert call(cake, dt=2) == INVALID and call(cake, w=None) == INVALID and call(cake, w=DAT["w"] + 8) == UNSUPPORTED
        assert call(cake, rstd=None) == INVALID and call(cake, rstd=DAT["rstd"] + 2) == UNSUPPORTED


def test_dropout_norm_refusals(cake):
    assert nfwd(cake, eps=-1.0) == INVALID and nfwd(cake, eps=NAN) == INVALID
    assert nfwd(cake, y=DAT["h"]) == INVALID and nfwd(cake, rstd=DAT["x"]) == INVALID and nfwd(cake, rstd=DAT["w"]) == INVALID
    assert nbwd(cake, dx=DAT["dres"]) == INVALID and nbwd(cake, dx=DAT["dy"]) == INVALID  # in place
    assert nbwd(cake, dw=None) == INVALID and nbwd(cake, dw=DAT["dw"] + 4) == UNSUPPORTED
    for n in ("dy", "dh", "h", "rstd", "w", "dx", "dres"):
        assert nbwd(cake, dw=DAT[n]) == INVALID and nbwd(cake, ws=DAT[n]) == INVALID, n
    assert nbwd(cake, ws=None) == WORKSPACE and nbwd(cake, n=8) == WORKSPACE and nbwd(cake, ws=64 * MB + 8) == UNSUPPORTED
    assert cake.cake_dropout_norm_bwd_workspace_size((0, 1, 64)) == cake.cake_dropout_norm_bwd_workspace_size((4, 1, 60)) == 0
    assert cake.cake_dropout_norm_bwd_workspace_size((4, 1, 64)) >= 64 * 8
    assert plain(cake, _three(0, 1, 64), x=(0,), y=(0,)) == 0
    got = (ctypes.c_int64 * 9)()
    lib = cake.load_library()
    assert lib.cake_dropout_norm_plan(S, 1, 0, got) == INVALID and lib.cake_dropout_norm_plan(S, 4, 1, got) == INVALID
    assert lib.cake_dropout_norm_plan(S, 2, 0, None) == INVALID


# ----------------------------------------------------------------------- Python

def test_python_refusals_without_a_gpu(cake):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    w, pos = torch.ones(64), torch.zeros(4, dtype=torch.int64)
    turns, axes = cake.cake_rotary_table((8, 8), device="cpu")
    for call in (lambda: cake.cake_gated(x, x, x), lambda: cake.cake_gated_bwd(x, x, x, x, x, x),
                 lambda: cake.cake_rotary(q, q, pos, turns), lambda: cake.cake_dropout(x, 0.1, 1),
                 lambda: cake.cake_dropout_norm(x, x, w, 0.1, 1),
                 lambda: cake.cake_dropout_norm_bwd(x, x, w, w, 0.1, 1)):
        with pytest.raises(ValueError, match="CUDA device"):  # no CPU path
            call()
