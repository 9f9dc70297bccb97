"""A training block's operators between the norms: Python binding and autograd.

Three groups of operators that run between the RMSNorm and the sandwich norm,
each in hand-written kernels behind the C ABI of ``include/cake_block.h``
(formulas and conventions there).  They have no counterpart in the pages; they
are additions of this library.

* Gated feed-forward block -- both projections, the activation and the product
  in one tensor-core kernel, and its gradients: ``cake_gated_fwd``,
  ``cake_gated_bwd`` and the differentiable ``cake_gated``;
* per-head norm of queries and keys with rotary positions of several axes:
  ``cake_rotary_table``, ``cake_rotary_fwd``, ``cake_rotary_bwd`` and the
  differentiable ``cake_rotary``;
* dropout from a counter-based generator, whose mask is never stored, alone and
  with the residual addition and the norm after it: ``cake_dropout_fwd``,
  ``cake_dropout_bwd``, ``cake_dropout_norm_fwd``, ``cake_dropout_norm_bwd`` and
  the differentiable ``cake_dropout`` and ``cake_dropout_norm``.

Devices, streams, workspaces, given outputs and errors are as in the module
``step``: a call runs on the tensors' device, on its current stream or on
``stream``; without a workspace from the caller it takes one from torch's
allocator; tensors that a caller gives to be written count as changed in place.
Every result is bitwise reproducible for equal inputs and shapes.

The entry points check their tensors, allocate and call the ABI in the compiled
module ``_cake_block`` (``csrc_block/cake_block_python.cpp``): small calls are
the host's.
"""
from __future__ import annotations

import ctypes
import decimal
import functools
import importlib
import math

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import CakeError, load_library
from .step import _check, _gradient, _on, _rows, _three

__all__ = [
    "cake_gated_fwd", "cake_gated_bwd", "cake_gated_bwd_workspace_size", "cake_gated", "CakeGatedFunction",
    "cake_rotary_table", "cake_rotary_fwd", "cake_rotary_bwd", "cake_rotary_bwd_workspace_size", "cake_rotary",
    "CakeRotaryFunction", "cake_dropout_fwd", "cake_dropout_bwd", "cake_dropout", "CakeDropoutFunction",
    "cake_dropout_norm_fwd", "cake_dropout_norm_bwd", "cake_dropout_norm_bwd_workspace_size", "cake_dropout_norm",
    "CakeDropoutNormFunction", "cake_block_wait_test",
]

_vp, _i64, _u64, _int, _size = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64, ctypes.c_int, ctypes.c_size_t
_f32, _f64 = ctypes.c_float, ctypes.c_double


def _bind(lib):
    """Declare the operators' C signatures on the library handle."""
    T = S = R = _vp  # shapes, tensors and rotations are passed as packed bytes
    for name, res, args in (
        ("cake_gated_fwd", _int, [_i64, _i64, _i64, T, T, T, _int, T, T, T, _vp]),
        ("cake_gated_bwd_workspace_size", _size, [_i64, _i64, _i64]),
        ("cake_gated_bwd", _int, [_i64, _i64, _i64, T, T, T, T, T, T, _int, T, T, T, _vp, _size, _vp]),
        ("cake_rotary_fwd", _int, [_i64, _i64, _i64, _i64, T, T, R, _vp, _int, _vp, _int, _f32, T, T, _vp, _vp, _vp]),
        ("cake_rotary_bwd_workspace_size", _size, [_i64, _i64, _i64, _i64]),
        ("cake_rotary_bwd", _int, [_i64, _i64, _i64, _i64, T, T, R, T, T, _vp, _vp, _vp, _int, _vp, _int, T, T, _vp,
                                   _vp, _vp, _size, _vp]),
        ("cake_dropout", _int, [S, T, T, _f64, _u64, _u64, _vp, T, _vp]),
        ("cake_dropout_norm_fwd", _int, [S, T, T, _vp, _int, _f64, _u64, _u64, _vp, _f32, T, T, _vp, _vp]),
        ("cake_dropout_norm_bwd_workspace_size", _size, [S]),
        ("cake_dropout_norm_bwd", _int, [S, T, T, T, _vp, _vp, _int, _f64, _u64, _u64, _vp, T, T, _vp, _vp, _size,
                                         _vp]),
        ("cake_block_wait_test", _int, [ctypes.c_uint32, _int]),
        ("cake_dropout_norm_plan", _int, [S, _int, _int, ctypes.POINTER(_i64)]),
    ):
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args


def cake_block_wait_test(wait_limit_us: int = 0, withhold: int = 0):
    """Tests of the kernels' bounded waits: the limit of the waits of the calls that this host thread makes from now
    on, and whether a part of the first copies never comes (see ``include/cake_block_test.h``); no arguments: the
    ordinary limit again."""
    _check(load_library().cake_block_wait_test(wait_limit_us, withhold), "cake_block_wait_test")


_module = None


def _native():
    """The compiled entry points (loaded once)."""
    global _module
    if _module is None:
        load_library()
        try:
            module = importlib.import_module("._cake_block", __package__)
        except ImportError as e:
            raise RuntimeError("_cake_block.so is missing or does not load: build it first "
                               "(python -c 'import __graft_entry__ as g; g.build()')") from e
        module.set_error(CakeError)
        _module = module
    return _module


# ------------------------------------------------------------------------ gated

def cake_gated_fwd(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, act: str = "silu", *, save: bool = True,
                   h: torch.Tensor | None = None, g: torch.Tensor | None = None, u: torch.Tensor | None = None,
                   stream=None):
    """Forward: (h, g, u) with g = x w_gate^T, u = x w_up^T and h = act(g) * u.

    x: BF16 [T, H]; w_gate, w_up: BF16 [F, H] (the two may be halves of one
    matrix); H and F multiples of 8.  act: "silu" or "gelu" (the tanh form).
    With ``save`` false g and u, which only the backward needs, are not written
    and come back as None.
    """
    if stream is not None:
        with _on(stream, x):
            return _native().gated_fwd(x, w_gate, w_up, act, save, h, g, u)
    return _native().gated_fwd(x, w_gate, w_up, act, save, h, g, u)


@functools.lru_cache(maxsize=256)
def cake_gated_bwd_workspace_size(tokens: int, hidden: int, ffn: int) -> int:
    """Workspace bytes of the gated block's backward."""
    return int(load_library().cake_gated_bwd_workspace_size(int(tokens), int(hidden), int(ffn)))


def cake_gated_bwd(dh: torch.Tensor, x: torch.Tensor, g: torch.Tensor, u: torch.Tensor, w_gate: torch.Tensor,
                   w_up: torch.Tensor, act: str = "silu", *, need_dx: bool = True, need_dw: bool = True,
                   workspace: torch.Tensor | None = None, dx: torch.Tensor | None = None,
                   dw_gate: torch.Tensor | None = None, dw_up: torch.Tensor | None = None, stream=None):
    """Backward: (dx, dw_gate, dw_up), BF16; None for what is not needed.

    dh: gradient of h, BF16 [T, F]; g and u as the forward gave them.  With more
    than 64 tokens the gradients of g and u are rounded to BF16 once between the
    two products (see ``include/cake_block.h``).
    """
    if stream is not None:
        with _on(stream, x):
            return _native().gated_bwd(dh, x, g, u, w_gate, w_up, act, need_dx, need_dw, workspace, dx, dw_gate, dw_up)
    return _native().gated_bwd(dh, x, g, u, w_gate, w_up, act, need_dx, need_dw, workspace, dx, dw_gate, dw_up)


class CakeGatedFunction(torch.autograd.Function):
    """The gated block with the library's forward and backward: ``apply(x, w_gate, w_up, act)``."""

    @staticmethod
    def forward(ctx, x, w_gate, w_up, act="silu"):
        rows = x.reshape(-1, x.shape[-1])
        h, g, u = cake_gated_fwd(rows, w_gate, w_up, act)
        ctx.save_for_backward(rows, g, u, w_gate, w_up)
        ctx.act, ctx.size = act, x.shape
        return h.view(*x.shape[:-1], h.shape[-1])

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        x, g, u, w_gate, w_up = ctx.saved_tensors
        dh = _gradient(dh.reshape(g.shape))
        dx, dwg, dwu = cake_gated_bwd(dh, x, g, u, w_gate, w_up, ctx.act, need_dx=ctx.needs_input_grad[0],
                                      need_dw=ctx.needs_input_grad[1] or ctx.needs_input_grad[2])
        return None if dx is None else dx.view(ctx.size), dwg, dwu, None


def cake_gated(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, act: str = "silu") -> torch.Tensor:
    """Differentiable gated block: act(x w_gate^T) * (x w_up^T) of x [..., H], reverse mode; see ``cake_gated_fwd``."""
    if torch.is_grad_enabled() and (x.requires_grad or w_gate.requires_grad or w_up.requires_grad) or \
            forward_ad._current_level >= 0 and any(forward_ad.unpack_dual(t).tangent is not None for t in (x, w_gate, w_up)):
        # (of a tangent the function raises: there is no forward mode)
        return CakeGatedFunction.apply(x, w_gate, w_up, act)
    h, _, _ = cake_gated_fwd(x.reshape(-1, x.shape[-1]), w_gate, w_up, act, save=False)
    return h.view(*x.shape[:-1], h.shape[-1])


# ----------------------------------------------------------------------- rotary

def _digits(n: int):
    """Decimal arithmetic of n digits, whatever context the caller has set."""
    return decimal.localcontext(decimal.Context(prec=n, rounding=decimal.ROUND_HALF_EVEN))


@functools.lru_cache(maxsize=8)
def _two_pi(digits: int) -> decimal.Decimal:
    """2 pi by the arithmetic-geometric mean (Brent and Salamin, 1976), which doubles its digits with every step."""
    with _digits(digits + 10):
        a, b, t, p = decimal.Decimal(1), 1 / decimal.Decimal(2).sqrt(), decimal.Decimal("0.25"), 1
        while abs(a - b) > decimal.Decimal(10) ** -(digits // 2 + 2):
            m = (a + b) / 2
            t -= p * (a - m) ** 2
            a, b, p = m, (a * b).sqrt(), 2 * p
        return (a + b) ** 2 / (2 * t)


def _ladder(base: float, n: int) -> list:
    """base^(-i / n) for i < n."""
    if n <= 1:
        return [decimal.Decimal(1)] * n
    if not base > 0:
        raise ValueError(f"the base of a ladder of frequencies is positive, got {base}")
    step, out = (-decimal.Decimal(base).ln() / n).exp(), [decimal.Decimal(1)]
    while len(out) < n:
        out.append(out[-1] * step)
    return out


def cake_rotary_table(sections, base: float = 10000.0, *, shared: bool = False, freqs=None, device="cuda"):
    """(turns, axes) of a rotation: each pair's frequency and the axis whose position turns it.

    sections: the number of pairs of each axis.  The i-th of an axis' n pairs
    has the frequency base^(-i / n) radians a position, or with ``shared`` pair
    j of all of them base^(-j / pairs); ``freqs`` gives every pair's frequency
    instead.  turns: int64, the frequency's share of a turn in units of 2^-64
    (modulo 2^64), rounded to the nearest one: an angle is off by the position
    times 2^-65 of a turn at most, besides the kernels' own rounding.
    """
    sections = [int(n) for n in sections]
    pairs = sum(sections)
    if freqs is None:
        base = float(base)
        largest = 1 / base if 0 < base < 1 else 1.0
    else:
        freqs = [float(f) for f in freqs]
        if len(freqs) != pairs:
            raise ValueError(f"{len(freqs)} frequencies for {pairs} pairs")
        for f in freqs:
            if not math.isfinite(f):
                raise ValueError(f"a frequency is {f}")
        largest = max(map(abs, freqs), default=0.0)
    # 64 bits of a turn, and the whole turns that drop out, are more than a double has
    digits = 50 + max(0, math.frexp(min(largest, 1e308))[1] // 3)
    turns = []
    with _digits(digits):
        if freqs is not None:
            freqs = [decimal.Decimal(f) for f in freqs]
        elif shared:
            freqs = _ladder(base, pairs)
        else:
            freqs = [f for n in sections for f in _ladder(base, n)]
        unit = 2 ** 64 / _two_pi(digits)
        for f in freqs:
            t = int((f * unit).to_integral_value()) % 2 ** 64
            turns.append(t - 2 ** 64 if t >= 2 ** 63 else t)
    axes = [a for a, n in enumerate(sections) for _ in range(n)]
    return (torch.tensor(turns, dtype=torch.int64, device=device),
            torch.tensor(axes, dtype=torch.int32, device=device))


def cake_rotary_fwd(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, turns: torch.Tensor,
                    axes: torch.Tensor | None = None, w_q: torch.Tensor | None = None,
                    w_k: torch.Tensor | None = None, eps: float = 1e-6, *, style: str = "half",
                    q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                    rstd_q: torch.Tensor | None = None, rstd_k: torch.Tensor | None = None, stream=None):
    """Forward: (q_out, k_out, rstd_q, rstd_k): each head normed (with w_q, w_k), then rotated by its position.

    q: BF16 [T, heads, D], k: BF16 [T, k_heads, D] or None, views with a
    contiguous D (a multiple of 16, at most 512); positions: int32 or int64 [T]
    or [axes, T]; turns, axes: see ``cake_rotary_table``.  The first 2 * pairs
    columns are rotated, pair i being columns (i, pairs + i) in style "half"
    and (2 i, 2 i + 1) in style "adjacent".  w_q, w_k: [D] BF16 or FP32; without
    them there is no norm and rstd_q and rstd_k are None, else they are FP32
    [T * heads].  q_out may be q itself and k_out k itself.
    """
    if stream is not None:
        with _on(stream, q):
            return _native().rotary_fwd(q, k, positions, turns, axes, w_q, w_k, eps, style, q_out, k_out, rstd_q, rstd_k)
    return _native().rotary_fwd(q, k, positions, turns, axes, w_q, w_k, eps, style, q_out, k_out, rstd_q, rstd_k)


@functools.lru_cache(maxsize=256)
def cake_rotary_bwd_workspace_size(tokens: int, q_heads: int, k_heads: int, hidden: int) -> int:
    """Workspace bytes of the rotary backward with a norm (k_heads 0: no keys)."""
    return int(load_library().cake_rotary_bwd_workspace_size(int(tokens), int(q_heads), int(k_heads), int(hidden)))


def cake_rotary_bwd(dq: torch.Tensor, dk: torch.Tensor | None, positions: torch.Tensor, turns: torch.Tensor,
                    axes: torch.Tensor | None = None, q: torch.Tensor | None = None, k: torch.Tensor | None = None,
                    rstd_q: torch.Tensor | None = None, rstd_k: torch.Tensor | None = None,
                    w_q: torch.Tensor | None = None, w_k: torch.Tensor | None = None, *, style: str = "half",
                    workspace: torch.Tensor | None = None, dq_out: torch.Tensor | None = None,
                    dk_out: torch.Tensor | None = None, dw_q: torch.Tensor | None = None,
                    dw_k: torch.Tensor | None = None, stream=None):
    """Backward: (dq_out, dk_out, dw_q, dw_k); dw_q and dw_k are FP32 [D], None without a norm.

    dq, dk: gradients of the forward's q_out and k_out; q, k, rstd_q, rstd_k:
    the forward's inputs and what it gave (with a norm only).  dq_out may be dq
    itself and dk_out dk itself.
    """
    if stream is not None:
        with _on(stream, dq):
            return _native().rotary_bwd(dq, dk, positions, turns, axes, q, k, rstd_q, rstd_k, w_q, w_k, style, workspace,
                                    dq_out, dk_out, dw_q, dw_k)
    return _native().rotary_bwd(dq, dk, positions, turns, axes, q, k, rstd_q, rstd_k, w_q, w_k, style, workspace,
                                    dq_out, dk_out, dw_q, dw_k)


class CakeRotaryFunction(torch.autograd.Function):
    """Normed and rotated queries and keys with the library's forward and backward:
    ``apply(q, k, positions, turns, axes, w_q, w_k, eps, style)``."""

    @staticmethod
    def forward(ctx, q, k, positions, turns, axes=None, w_q=None, w_k=None, eps=1e-6, style="half"):
        y, z, rq, rk = cake_rotary_fwd(q, k, positions, turns, axes, w_q, w_k, eps, style=style)
        norm = w_q is not None
        ctx.save_for_backward(positions, turns, axes, w_q, w_k, rq, rk, q if norm else None, k if norm else None)
        ctx.style, ctx.sizes = style, (q.shape, None if k is None else k.shape)
        ctx.set_materialize_grads(False)
        return y, z

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        if dq is None and dk is None:
            return (None,) * 9
        positions, turns, axes, w_q, w_k, rq, rk, q, k = ctx.saved_tensors
        grads = []
        for d, size in zip((dq, dk), ctx.sizes):
            if size is not None and d is None:
                d = torch.zeros(size, dtype=torch.bfloat16, device=positions.device)
            grads.append(None if size is None else _gradient(d))
        dq, dk, dwq, dwk = cake_rotary_bwd(*grads, positions, turns, axes, q, k, rq, rk, w_q, w_k, style=ctx.style)
        return (dq, dk, None, None, None, None if w_q is None else dwq.to(w_q.dtype),
                None if w_k is None or dwk is None else dwk.to(w_k.dtype), None, None)


def cake_rotary(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, turns: torch.Tensor,
                axes: torch.Tensor | None = None, w_q: torch.Tensor | None = None, w_k: torch.Tensor | None = None,
                eps: float = 1e-6, style: str = "half"):
    """Differentiable per-head norm and rotary positions: (q_out, k_out); see ``cake_rotary_fwd``."""
    return CakeRotaryFunction.apply(q, k, positions, turns, axes, w_q, w_k, eps, style)


# ---------------------------------------------------------------------- dropout

def _on_device(seed):
    return seed if isinstance(seed, torch.Tensor) else None


def cake_dropout_fwd(x: torch.Tensor, p: float, seed, offset: int = 0, residual: torch.Tensor | None = None, *,
                     y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y = bf16(m * x [+ residual]), m 0 with probability p and else 1 over the share that is kept.

    x, residual: BF16 [T, H] or [T, nh, H] views, H a multiple of 8, at most
    8192 as for the norm (a wider dense tensor goes as [T, n, H / n]: an
    element's place is the same).  The mask goes by seed,
    offset and an element's place alone and is never stored: calls with the
    same ones drop the same elements, so give every use of a step an offset of
    its own.  p counts in steps of 2^-16.  seed: a number, or an int64 tensor
    of two on the device, the seed and a number that is added to offset, which
    a captured graph reads anew at each replay.  y may be x or residual.
    """
    if stream is not None:
        with _on(stream, x):
            return _native().dropout(x, p, seed, offset, residual, y)
    return _native().dropout(x, p, seed, offset, residual, y)


def cake_dropout_bwd(dy: torch.Tensor, p: float, seed, offset: int = 0, *, dx: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """dx = bf16(m * dy): the gradient of ``cake_dropout_fwd``'s x (that of its residual is dy)."""
    return cake_dropout_fwd(dy, p, seed, offset, y=dx, stream=stream)


class CakeDropoutFunction(torch.autograd.Function):
    """Dropout with an optional residual addition: ``apply(x, residual, p, seed, offset)``."""

    @staticmethod
    def forward(ctx, x, residual, p, seed, offset=0):
        ctx.save_for_backward(_on_device(seed))
        ctx.p, ctx.seed, ctx.offset = p, None if isinstance(seed, torch.Tensor) else seed, offset
        return cake_dropout_fwd(x, p, seed, offset, residual)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        seed, = ctx.saved_tensors
        dy = _gradient(dy)
        dx = cake_dropout_bwd(dy, ctx.p, ctx.seed if seed is None else seed, ctx.offset) \
            if ctx.needs_input_grad[0] else None
        return dx, dy if ctx.needs_input_grad[1] else None, None, None, None


def cake_dropout(x: torch.Tensor, p: float, seed, offset: int = 0,
                 residual: torch.Tensor | None = None) -> torch.Tensor:
    """Differentiable dropout, with an optional residual addition; see ``cake_dropout_fwd``."""
    return CakeDropoutFunction.apply(x, residual, p, seed, offset)


def cake_dropout_norm_fwd(x: torch.Tensor, residual: torch.Tensor, w: torch.Tensor, p: float, seed, offset: int = 0,
                          eps: float = 1e-6, *, y: torch.Tensor | None = None, h_new: torch.Tensor | None = None,
                          rstd: torch.Tensor | None = None, stream=None):
    """Forward: (y, h_new, rstd): h_new = bf16(residual + m * x), y = norm(h_new) * w.

    x: a block's output, residual: the residual stream, BF16 [T, H] or
    [T, nh, H]; w: [H] BF16 or FP32; p, seed, offset: see ``cake_dropout_fwd``.
    y and h_new may be x or residual themselves.
    """
    if stream is not None:
        with _on(stream, x):
            return _native().dropout_norm_fwd(x, residual, w, p, seed, offset, eps, y, h_new, rstd)
    return _native().dropout_norm_fwd(x, residual, w, p, seed, offset, eps, y, h_new, rstd)


@functools.lru_cache(maxsize=256)
def _dropout_norm_bwd_bytes(T, nh, H):
    return int(load_library().cake_dropout_norm_bwd_workspace_size(_three(T, nh, H)))


def cake_dropout_norm_bwd_workspace_size(x_or_shape) -> int:
    """Workspace bytes the backward needs for this row set ([T, H] / [T, nh, H] tensor or (T, nh, H))."""
    return _dropout_norm_bwd_bytes(*(_rows(x_or_shape) if isinstance(x_or_shape, torch.Tensor) else x_or_shape))


def cake_dropout_norm_bwd(dy: torch.Tensor, h_new: torch.Tensor, rstd: torch.Tensor, w: torch.Tensor, p: float, seed,
                          offset: int = 0, dh: torch.Tensor | None = None, *, workspace: torch.Tensor | None = None,
                          dx: torch.Tensor | None = None, dresidual: torch.Tensor | None = None,
                          dw: torch.Tensor | None = None, stream=None):
    """Backward: (dresidual, dx, dw); dw is FP32 [H].

    dy: gradient of y; dh: that reaching h_new directly, or None; h_new and rstd
    as the forward gave them, p, seed and offset as it took them.
    """
    if stream is not None:
        with _on(stream, dy):
            return _native().dropout_norm_bwd(dy, h_new, rstd, w, p, seed, offset, dh, workspace, dx, dresidual, dw)
    return _native().dropout_norm_bwd(dy, h_new, rstd, w, p, seed, offset, dh, workspace, dx, dresidual, dw)


class CakeDropoutNormFunction(torch.autograd.Function):
    """(y, h_new) of dropout, residual addition and norm:
    ``apply(x, residual, w, p, seed, offset, eps)``."""

    @staticmethod
    def forward(ctx, x, residual, w, p, seed, offset=0, eps=1e-6):
        y, h, rstd = cake_dropout_norm_fwd(x, residual, w, p, seed, offset, eps)
        ctx.save_for_backward(h, rstd, w, _on_device(seed))
        ctx.p, ctx.seed, ctx.offset = p, None if isinstance(seed, torch.Tensor) else seed, offset
        ctx.set_materialize_grads(False)
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        if dy is None and dh is None:
            return (None,) * 7
        h, rstd, w, seed = ctx.saved_tensors
        dy = torch.zeros_like(h) if dy is None else _gradient(dy)
        dh = None if dh is None else _gradient(dh)
        dres, dx, dw = cake_dropout_norm_bwd(dy, h, rstd, w, ctx.p, ctx.seed if seed is None else seed, ctx.offset, dh)
        return dx, dres, dw.to(w.dtype), None, None, None, None


def cake_dropout_norm(x: torch.Tensor, residual: torch.Tensor, w: torch.Tensor, p: float, seed, offset: int = 0,
                      eps: float = 1e-6):
    """Differentiable dropout, residual addition and norm: (y, h_new); see ``cake_dropout_norm_fwd``."""
    return CakeDropoutNormFunction.apply(x, residual, w, p, seed, offset, eps)
