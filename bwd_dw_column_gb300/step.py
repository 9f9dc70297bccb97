"""Training-step operators around the RMSNorm: Python binding and autograd.

Three groups of operators that a training step needs next to the norm, each in
hand-written kernels behind the C ABI of ``include/cake_step.h`` (formulas and
conventions there).  They have no counterpart in the pages; they are additions
of this library.

* Sandwich norm -- the norm after a block, a gate, the residual scale and
  addition, and the norm before the next block in one pass:
  ``cake_sandwich_fwd``, ``cake_sandwich_bwd`` and the differentiable
  ``cake_sandwich_norm``;
* gradient norm and clipping over many tensors: ``cake_grad_norm`` and
  ``cake_clip_grad_norm``;
* embedding lookup with a scale, and its gradient by sorted tokens:
  ``cake_embedding_fwd``, ``cake_embedding_bwd`` and the differentiable
  ``cake_embedding``.

Every result is bitwise reproducible for equal inputs and shapes.  Workspaces
hold nothing between calls; without one from the caller a call takes it from
torch's allocator, so calls on several streams and in several captured graphs
never share one.  A call runs on the tensors' device, on its current stream or
on ``stream``, where its outputs and workspace are allocated too.  Tensors that a caller gives
to be written count as changed in place for autograd, as with torch's own
in-place operations: a backward pass that has saved one raises.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from array import array
from operator import attrgetter, is_not

import torch
from torch.autograd.function import once_differentiable
from torch.autograd.graph import increment_version

from . import CAKE_BF16, CAKE_FP32, CAKE_OK, CakeError, load_library

__all__ = [
    "cake_sandwich_fwd", "cake_sandwich_bwd", "cake_sandwich_bwd_workspace_size", "cake_sandwich_norm",
    "CakeSandwichFunction", "cake_grad_norm", "cake_clip_grad_norm", "cake_grad_norm_workspace_size",
    "cake_embedding_fwd", "cake_embedding_bwd", "cake_embedding_bwd_workspace_size", "cake_embedding",
    "CakeEmbeddingFunction", "cake_step_wait_test",
]

_vp, _i64, _f32, _int, _size = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int, ctypes.c_size_t


def _bind(lib):
    """Declare the operators' C signatures on the library handle."""
    T = S = _vp  # shapes and tensors are passed as packed bytes (see _three)
    for name, res, args in (
        ("cake_sandwich_fwd", _int, [S, T, T, _vp, _int, _vp, _int, _vp, T, _f32, _f32, T, T, _vp, _vp, _vp]),
        ("cake_sandwich_bwd_workspace_size", _size, [S]),
        ("cake_sandwich_bwd", _int, [S, T, T, T, T, _vp, _vp, _vp, _int, _vp, _int, _vp, T, _f32, T, T, _vp, _vp, _vp,
                                     T, _vp, _size, _vp]),
        ("cake_grad_norm_workspace_size", _size, [_i64]),
        ("cake_grad_norm", _int, [_vp, _vp, _vp, _i64, _vp, _vp, _size, _vp]),
        ("cake_grad_clip", _int, [_vp, _vp, _vp, _vp, _vp, _i64, _f32, _f32, _vp, _vp, _size, _vp]),
        ("cake_embedding_fwd", _int, [_vp, _int, _i64, _vp, _int, _i64, _i64, _i64, _f32, T, _vp]),
        ("cake_embedding_bwd_workspace_size", _size, [_i64, _i64, _i64]),
        ("cake_embedding_bwd", _int, [T, _vp, _int, _i64, _i64, _i64, _f32, _i64, _vp, _int, _i64, _int, _vp, _size,
                                      _vp]),
        ("cake_step_wait_test", _int, [ctypes.c_uint32, _int]),
        ("cake_sandwich_bwd_plan", _int, [S, _int, ctypes.POINTER(_int)]),
        ("cake_step_rows_meet", _int, [S, T, T]),
    ):
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args


# ------------------------------------------------------------- devices, streams

class _Here:
    """No change of device or stream."""

    def __enter__(self):
        return None

    def __exit__(self, *a):
        return None


_here = _Here()


class _On:
    """The tensors' device, and the given stream of it."""

    def __init__(self, device, stream):
        self.contexts = [torch.cuda.device(device)] + ([torch.cuda.stream(stream)] if stream is not None else [])

    def __enter__(self):
        for c in self.contexts:
            c.__enter__()

    def __exit__(self, *a):
        for c in reversed(self.contexts):
            c.__exit__(*a)


def _on(stream, *tensors):
    """Context of a call: every tensor (None: left out) on one CUDA device, which becomes
    the current one, with `stream` (None: its current stream) the current stream."""
    return _on_devices(stream, {t.get_device() for t in tensors if t is not None})


def _on_devices(stream, devices):
    if -1 in devices:
        raise ValueError("every tensor must be on a CUDA device (no CPU path)")
    if len(devices) != 1:
        raise ValueError("every tensor must be on the same device")
    dev, = devices
    if stream is None:
        if torch.cuda.current_device() == dev:
            return _here
    elif stream.device.index != dev:
        raise ValueError("the stream belongs to another device than the tensors")
    return _On(dev, stream)


def _current() -> int:
    """The current device's current stream."""
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def cake_step_wait_test(wait_limit_us: int = 0, withhold: int = 0):
    """Tests of the kernels' bounded waits: the limit of the waits of the calls that this host thread makes from now
    on, and what never comes to them (see ``include/cake_step_test.h``); no arguments: the ordinary limit again."""
    _check(load_library().cake_step_wait_test(wait_limit_us, withhold), "cake_step_wait_test")


# ------------------------------------------------------------------- marshalling

# cake_shape and cake_tensor are three int64 each.  Packed bytes cost a third
# of a ctypes structure, which counts where a call takes microseconds.
_three = struct.Struct("=qqq").pack


def _check(status: int, what: str):
    if status != CAKE_OK:
        raise CakeError(status, what)


def _given(*tensors):
    """The tensors among a call's outputs that the caller has given."""
    return [t for t in tensors if t is not None]


def _rows(t):
    """(T, nh, H) of a [T, H] or [T, nh, H] tensor."""
    if t.dim() == 2:
        T, H = t.shape
        return T, 1, H
    if t.dim() == 3:
        return tuple(t.shape)
    raise ValueError(f"expected a [T, H] or [T, nh, H] tensor, got shape {tuple(t.shape)}")


def _ref(t, shape, what):
    """A BF16 activation of the given shape as a packed cake_tensor (None: NULL)."""
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"activations are BF16, got {t.dtype}")
    st = t.stride()
    if st[-1] != 1 and t.numel():
        raise ValueError("the hidden dimension must be contiguous")
    return _three(t.data_ptr(), st[0], st[1] if len(st) == 3 else 0)


def _dtype(w):
    if w.dtype is torch.bfloat16:
        return CAKE_BF16
    if w.dtype is torch.float32:
        return CAKE_FP32
    raise TypeError(f"weight is BF16 or FP32, got {w.dtype}")


def _weight(w, H, what):
    if w.dim() != 1 or w.shape[0] != H:
        raise ValueError(f"{what} has shape {tuple(w.shape)}, expected ({H},)")
    return w if w.is_contiguous() else w.contiguous()


def _rows_f32(t, rows, what):
    if t.dtype is not torch.float32 or t.numel() != rows or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous FP32 tensor of T*nh elements")
    return t.data_ptr()


def _like(z):
    return torch.empty_like(z) if z.is_contiguous() else torch.empty(z.shape, dtype=z.dtype, device=z.device)


def _workspace(workspace, size, device):
    """(tensor that keeps it alive, address, bytes)"""
    if workspace is None:
        workspace = torch.empty(size or 256, dtype=torch.uint8, device=device)
        return workspace, workspace.data_ptr(), size
    if not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


# ---------------------------------------------------------------- sandwich norm

def _gate(gate, z):
    """(row gate or None, element gate or None)."""
    if gate is None:
        return None, None
    if gate.shape == z.shape:
        return None, gate
    if gate.shape == z.shape[:-1]:
        if gate.dtype != torch.float32:
            raise TypeError(f"a gate of one value per row is FP32, got {gate.dtype}")
        return (gate if gate.is_contiguous() else gate.contiguous()), None
    raise ValueError(f"gate has shape {tuple(gate.shape)}, expected {tuple(z.shape[:-1])} (rows) or {tuple(z.shape)}")


def cake_sandwich_fwd(z: torch.Tensor, x: torch.Tensor, w_post: torch.Tensor, w_pre: torch.Tensor,
                      eps: float = 1e-6, gate: torch.Tensor | None = None, scale: float = 1.0, *,
                      y: torch.Tensor | None = None, h_new: torch.Tensor | None = None,
                      rstd_post: torch.Tensor | None = None, rstd_pre: torch.Tensor | None = None, stream=None):
    """Forward: (y, h_new, rstd_post, rstd_pre).

    z: a block's output, x: the residual stream, BF16 [T, H] or [T, nh, H]
    views (hidden dim contiguous); w_post, w_pre: [H] BF16 or FP32 each;
    gate: None, FP32 of z's leading shape (a value per row) or BF16 of z's
    shape.  h_new = bf16(x + scale * gate * norm(z) * w_post) is the new
    residual stream and y = norm(h_new) * w_pre the next block's input.
    h_new may be x itself and y z itself (in place).
    """
    lib = load_library()
    with _on(stream, z, x, w_post, w_pre, gate, y, h_new, rstd_post, rstd_pre):
        T, nh, H = _rows(z)
        size, rows = z.shape, T * nh
        w_post, w_pre = _weight(w_post, H, "w_post"), _weight(w_pre, H, "w_pre")
        g_row, g_elem = _gate(gate, z)
        given = _given(y, h_new, rstd_post, rstd_pre)
        if y is None:
            y = _like(z)
        if h_new is None:
            h_new = _like(z)
        if rstd_post is None:
            rstd_post = torch.empty(rows, dtype=torch.float32, device=z.device)
        if rstd_pre is None:
            rstd_pre = torch.empty(rows, dtype=torch.float32, device=z.device)
        st = lib.cake_sandwich_fwd(_three(T, nh, H), _ref(z, size, "z"), _ref(x, size, "x"), w_post.data_ptr(),
                                   _dtype(w_post), w_pre.data_ptr(), _dtype(w_pre),
                                   None if g_row is None else g_row.data_ptr(), _ref(g_elem, size, "gate"), scale, eps,
                                   _ref(y, size, "y"), _ref(h_new, size, "h_new"),
                                   _rows_f32(rstd_post, rows, "rstd_post"), _rows_f32(rstd_pre, rows, "rstd_pre"),
                                   _current())
        _check(st, "cake_sandwich_fwd")
        if given:
            increment_version(given)
    return y, h_new, rstd_post, rstd_pre


@functools.lru_cache(maxsize=256)
def _sandwich_bwd_bytes(T, nh, H):
    return int(load_library().cake_sandwich_bwd_workspace_size(_three(T, nh, H)))


def cake_sandwich_bwd_workspace_size(x_or_shape) -> int:
    """Workspace bytes the backward needs for this row set ([T, H] / [T, nh, H] tensor or (T, nh, H))."""
    return _sandwich_bwd_bytes(*(_rows(x_or_shape) if isinstance(x_or_shape, torch.Tensor) else x_or_shape))


def cake_sandwich_bwd(dy: torch.Tensor, h_new: torch.Tensor, z: torch.Tensor, rstd_post: torch.Tensor,
                      rstd_pre: torch.Tensor, w_post: torch.Tensor, w_pre: torch.Tensor,
                      dh: torch.Tensor | None = None, gate: torch.Tensor | None = None, scale: float = 1.0, *,
                      need_dgate: bool = True, workspace: torch.Tensor | None = None, dx: torch.Tensor | None = None,
                      dz: torch.Tensor | None = None, dw_post: torch.Tensor | None = None,
                      dw_pre: torch.Tensor | None = None, dgate: torch.Tensor | None = None, stream=None):
    """Backward: (dx, dz, dw_post, dw_pre, dgate).

    dy: gradient of y; dh: that reaching h_new directly, or None; h_new and the
    rstd as the forward gave them.  dx (of the residual stream) and dz (of the
    block's output) are BF16, dw_post and dw_pre FP32 [H].  dgate has the
    gate's shape and type, or is None without a gate or with need_dgate false.
    """
    lib = load_library()
    with _on(stream, dy, h_new, z, rstd_post, rstd_pre, w_post, w_pre, dh, gate, workspace, dx, dz, dw_post, dw_pre,
             dgate):
        T, nh, H = _rows(z)
        size, rows = z.shape, T * nh
        w_post, w_pre = _weight(w_post, H, "w_post"), _weight(w_pre, H, "w_pre")
        g_row, g_elem = _gate(gate, z)
        dev = z.device
        given = _given(dx, dz, dw_post, dw_pre, dgate)
        if dx is None:
            dx = _like(z)
        if dz is None:
            dz = _like(z)
        if dw_post is None:
            dw_post = torch.empty(H, dtype=torch.float32, device=dev)
        if dw_pre is None:
            dw_pre = torch.empty(H, dtype=torch.float32, device=dev)
        for t, what in ((dw_post, "dw_post"), (dw_pre, "dw_pre")):
            if t.dtype is not torch.float32 or t.numel() != H or not t.is_contiguous():
                raise ValueError(f"{what} must be a contiguous FP32 tensor of H elements")
        if gate is None or not need_dgate:
            if dgate is not None:
                raise ValueError("dgate is given, but no gradient of a gate is asked for")
        elif dgate is None:
            dgate = torch.empty(gate.shape, dtype=gate.dtype, device=dev)
        elif dgate.shape != gate.shape or (g_row is not None and (dgate.dtype is not torch.float32 or
                                                                  not dgate.is_contiguous())):
            raise ValueError("dgate must have the gate's shape (and be contiguous FP32 for a value per row)")
        workspace, ws, ws_bytes = _workspace(workspace, _sandwich_bwd_bytes(T, nh, H), dev)
        st = lib.cake_sandwich_bwd(_three(T, nh, H), _ref(dy, size, "dy"), _ref(dh, size, "dh"),
                                   _ref(h_new, size, "h_new"), _ref(z, size, "z"),
                                   _rows_f32(rstd_post, rows, "rstd_post"), _rows_f32(rstd_pre, rows, "rstd_pre"),
                                   w_post.data_ptr(), _dtype(w_post), w_pre.data_ptr(), _dtype(w_pre),
                                   None if g_row is None else g_row.data_ptr(), _ref(g_elem, size, "gate"), scale,
                                   _ref(dx, size, "dx"), _ref(dz, size, "dz"), dw_post.data_ptr(), dw_pre.data_ptr(),
                                   dgate.data_ptr() if g_row is not None and dgate is not None else None,
                                   _ref(dgate, size, "dgate") if g_elem is not None else None, ws, ws_bytes,
                                   _current())
        _check(st, "cake_sandwich_bwd")
        if given:
            increment_version(given)
    return dx, dz, dw_post, dw_pre, dgate


class CakeSandwichFunction(torch.autograd.Function):
    """(y, h_new) of the sandwich norm with the library's forward and backward:
    ``apply(z, x, w_post, w_pre, eps, gate, scale)``."""

    @staticmethod
    def forward(ctx, z, x, w_post, w_pre, eps=1e-6, gate=None, scale=1.0):
        y, h, r_post, r_pre = cake_sandwich_fwd(z, x, w_post, w_pre, eps, gate, scale)
        ctx.save_for_backward(h, z, r_post, r_pre, w_post, w_pre, gate)
        ctx.scale = float(scale)
        ctx.set_materialize_grads(False)
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        if dy is None and dh is None:
            return (None,) * 7
        h, z, r_post, r_pre, w_post, w_pre, gate = ctx.saved_tensors
        dy = torch.zeros_like(h) if dy is None else dy.to(torch.bfloat16).contiguous()
        dh = None if dh is None else dh.to(torch.bfloat16).contiguous()
        dx, dz, dwo, dwr, dgate = cake_sandwich_bwd(dy, h, z, r_post, r_pre, w_post, w_pre, dh, gate, ctx.scale,
                                                    need_dgate=ctx.needs_input_grad[5])
        return dz, dx, dwo.to(w_post.dtype), dwr.to(w_pre.dtype), None, dgate, None


def cake_sandwich_norm(z: torch.Tensor, x: torch.Tensor, w_post: torch.Tensor, w_pre: torch.Tensor, eps: float = 1e-6,
                       gate: torch.Tensor | None = None, scale: float = 1.0):
    """Differentiable sandwich norm: (y, h_new); see ``cake_sandwich_fwd``."""
    return CakeSandwichFunction.apply(z, x, w_post, w_pre, eps, gate, scale)


# --------------------------------------------------- gradient norm and clipping

def _dense(t: torch.Tensor) -> bool:
    """Whether the tensor's values fill one block of memory, in any order of its dimensions."""
    want = 1
    for stride, size in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n != 1):
        if stride != want:
            return False
        want *= size
    return True


_GRAD_DTYPES = {torch.bfloat16: CAKE_BF16, torch.float32: CAKE_FP32}
_T = torch.Tensor  # its methods and attributes, mapped over lists of hundreds of tensors
_dtype_of, _is_tensor = attrgetter("dtype"), functools.partial(is_not, None)


def _tensors(grads, what):
    """The tensors as the ABI's arrays (pointers, counts, dtypes), and whether all are contiguous."""
    try:
        types = array("i", map(_GRAD_DTYPES.__getitem__, map(_dtype_of, grads)))
    except KeyError as e:
        raise TypeError(f"{what} are BF16 or FP32, got {e.args[0]}") from None
    plain = all(map(_T.is_contiguous, grads))
    if not plain:
        for t in grads:
            if not _dense(t):
                raise ValueError(
                    f"{what} must fill one block of memory each (strides {t.stride()} of {tuple(t.shape)})")
    return array("Q", map(_T.data_ptr, grads)), array("q", map(_T.numel, grads)), types, plain


def _addr(a):
    return a.buffer_info()[0] if len(a) else None


@functools.lru_cache(maxsize=64)
def cake_grad_norm_workspace_size(n: int) -> int:
    """Workspace bytes of a norm over (or clipping of) n tensors."""
    return int(load_library().cake_grad_norm_workspace_size(int(n)))


def _grad_call(grads, outs, clip, max_norm, eps, norm, workspace, stream):
    lib = load_library()
    if not grads and norm is None:
        raise ValueError("no gradients: give the norm's tensor")
    devices = set(map(_T.get_device, grads))
    devices.update(t.get_device() for t in (norm, workspace) if t is not None)
    if outs is not None:
        devices.update(map(_T.get_device, outs))
    with _on_devices(stream, devices):
        ptrs, counts, types, plain = _tensors(grads, "gradients")
        n = len(grads)
        given = _given(norm)
        if norm is None:
            norm = torch.empty((), dtype=torch.float32, device=grads[0].device)
        elif norm.dtype is not torch.float32 or norm.numel() != 1:
            raise ValueError("norm must be an FP32 tensor of one element")
        workspace, ws, ws_bytes = _workspace(workspace, cake_grad_norm_workspace_size(n), norm.device)
        if not clip:
            st = lib.cake_grad_norm(_addr(ptrs), _addr(counts), _addr(types), n, norm.data_ptr(), ws, ws_bytes,
                                    _current())
            _check(st, "cake_grad_norm")
            if given:
                increment_version(given)
            return norm
        optrs = otypes = ()
        if outs:
            optrs, ocounts, otypes, oplain = _tensors(outs, "outputs")
            if ocounts != counts or not (plain and oplain or all(
                    g.is_contiguous() and o.is_contiguous() or (g.shape == o.shape and g.stride() == o.stride())
                    for g, o in zip(grads, outs))):
                raise ValueError("an output must hold its gradient's values in the same order")
        st = lib.cake_grad_clip(_addr(ptrs), _addr(counts), _addr(types), _addr(optrs), _addr(otypes), n, max_norm,
                                eps, norm.data_ptr(), ws, ws_bytes, _current())
        _check(st, "cake_grad_clip")
        increment_version(given + (grads if outs is None else outs))
        return norm


def cake_grad_norm(grads, *, norm: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """The L2 norm of all values of all tensors together: an FP32 device scalar.

    grads: a tensor or an iterable of them (None entries are left out), BF16
    and FP32 mixed as they come, each filling one block of memory.
    """
    grads = [grads] if isinstance(grads, torch.Tensor) else [g for g in grads if g is not None]
    return _grad_call(grads, None, False, 0.0, 0.0, norm, workspace, stream)


def cake_clip_grad_norm(grads, max_norm: float, eps: float = 1e-6, out=None, *, norm: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, stream=None):
    """Scale all gradients by min(1, max_norm / (norm + eps)); returns the norm before it.

    In place, or into ``out`` (a tensor per gradient, as many values in the same
    order, BF16 or FP32: for instance the optimizer's FP32 buffers).  The host waits for nothing: a
    NaN or infinite norm is for the caller to look at, and makes the gradients
    NaN as the formula says.  No tensor may be given twice, nor share memory
    with another.
    """
    if isinstance(grads, torch.Tensor):
        grads, out = [grads], (None if out is None else [out] if isinstance(out, torch.Tensor) else list(out))
    grads = list(grads)
    if out is not None:
        out = list(out)
        if len(out) != len(grads):
            raise ValueError(f"{len(out)} outputs for {len(grads)} gradients")
    if not all(map(_is_tensor, grads)):
        if out is not None:
            out = [o for g, o in zip(grads, out) if g is not None]
        grads = [g for g in grads if g is not None]
    if out is not None and not all(map(_is_tensor, out)):
        raise ValueError("an output is missing for a gradient")
    return _grad_call(grads, out, True, max_norm, eps, norm, workspace, stream)


# -------------------------------------------------------------------- embedding

def _ids(ids):
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"ids are int32 or int64, got {ids.dtype}")
    return ids if ids.is_contiguous() else ids.contiguous()


def _table(table, what):
    if table.dim() != 2:
        raise ValueError(f"{what} has shape {tuple(table.shape)}, expected [V, H]")
    if table.numel() and table.stride(1) != 1:
        raise ValueError("the hidden dimension must be contiguous")
    return table.shape


def cake_embedding_fwd(ids: torch.Tensor, table: torch.Tensor, scale: float = 1.0, *, y: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """y = bf16(scale * table[ids]), of ids' shape and [H].

    ids: int32 or int64; a negative one means no token (a zero row), one
    outside the table gives a zero row and sets the device status.  table:
    [V, H] BF16 or FP32.
    """
    lib = load_library()
    with _on(stream, ids, table, y):
        ids = _ids(ids)
        V, H = _table(table, "table")
        T = ids.numel()
        given = _given(y)
        if y is None:
            y = torch.empty((*ids.shape, H), dtype=torch.bfloat16, device=table.device)
        elif y.shape != (*ids.shape, H):
            raise ValueError(f"y has shape {tuple(y.shape)}, expected {(*ids.shape, H)}")
        st = lib.cake_embedding_fwd(ids.data_ptr(), int(ids.dtype is torch.int64), T, table.data_ptr(),
                                    _dtype(table), V, H, table.stride(0), scale,
                                    _ref(y if y.dim() == 2 else y.view(T, H), (T, H), "y"), _current())
        _check(st, "cake_embedding_fwd")
        if given:
            increment_version(given)
    return y


@functools.lru_cache(maxsize=256)
def cake_embedding_bwd_workspace_size(tokens: int, vocab: int, hidden: int) -> int:
    """Workspace bytes of an embedding's gradient."""
    return int(load_library().cake_embedding_bwd_workspace_size(int(tokens), int(vocab), int(hidden)))


def cake_embedding_bwd(dy: torch.Tensor, ids: torch.Tensor, vocab: int, scale: float = 1.0,
                       padding_idx: int | None = None, out: torch.Tensor | None = None, accumulate: bool = False,
                       dtype: torch.dtype = torch.float32, *, workspace: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """The table's gradient [vocab, H]: scale * the sum of dy over the tokens of each id.

    dy: BF16, of ids' shape and [H].  out: a BF16 or FP32 table that is written
    whole, or with ``accumulate`` added to (where it has tokens); without one a
    new table of ``dtype``.  Tokens with id ``padding_idx``, a negative id or
    one outside the table add nothing.
    """
    lib = load_library()
    with _on(stream, dy, ids, out, workspace):
        ids = _ids(ids)
        T, H = ids.numel(), dy.shape[-1]
        if dy.shape[:-1] != ids.shape:
            raise ValueError(f"dy has shape {tuple(dy.shape)}, expected {(*ids.shape, H)}")
        rows = dy if dy.dim() == 2 else dy.reshape(T, H)
        given = _given(out)
        if out is None:
            if accumulate:
                raise ValueError("accumulate needs the table that is added to")
            out = torch.empty((vocab, H), dtype=dtype, device=dy.device)
        if _table(out, "out") != (vocab, H):
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {(vocab, H)}")
        if padding_idx is not None and not 0 <= padding_idx < vocab:
            raise ValueError(f"padding_idx {padding_idx} is outside the table")
        workspace, ws, ws_bytes = _workspace(workspace, cake_embedding_bwd_workspace_size(T, vocab, H), dy.device)
        st = lib.cake_embedding_bwd(_ref(rows, (T, H), "dy"), ids.data_ptr(), int(ids.dtype is torch.int64), T, vocab, H, scale,
                                    -1 if padding_idx is None else padding_idx, out.data_ptr(), _dtype(out),
                                    out.stride(0), int(bool(accumulate)), ws, ws_bytes, _current())
        _check(st, "cake_embedding_bwd")
        if given:
            increment_version(given)
    return out


class CakeEmbeddingFunction(torch.autograd.Function):
    """Embedding lookup with the library's forward and gradient:
    ``apply(ids, table, scale, padding_idx)``."""

    @staticmethod
    def forward(ctx, ids, table, scale=1.0, padding_idx=None):
        ctx.save_for_backward(ids)
        ctx.vocab, ctx.dtype, ctx.scale, ctx.padding_idx = table.shape[0], table.dtype, float(scale), padding_idx
        return cake_embedding_fwd(ids, table, scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        ids, = ctx.saved_tensors
        dtable = cake_embedding_bwd(dy.to(torch.bfloat16).contiguous(), ids, ctx.vocab, ctx.scale, ctx.padding_idx,
                                    dtype=ctx.dtype)
        return None, dtable, None, None


def cake_embedding(ids: torch.Tensor, table: torch.Tensor, scale: float = 1.0,
                   padding_idx: int | None = None) -> torch.Tensor:
    """Differentiable embedding lookup; the table's gradient has the table's type."""
    return CakeEmbeddingFunction.apply(ids, table, scale, padding_idx)
