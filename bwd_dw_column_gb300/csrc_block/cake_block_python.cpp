// cake_block_python.cpp -- the Python entry points of a block's operators over
// their C ABI: checks of tensors, allocation of outputs and workspaces on the
// current stream, and the call.  Small calls are the host's, and this takes
// less than half of what the same steps take in Python (GB300's host: a token's 24 +
// 4 heads normed and rotated 7 us against 23.5, a gated backward 11 against 30).
//
// Every function takes its arguments by position; block.py has their names,
// defaults and documentation.
#include <initializer_list>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <pybind11/pybind11.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/cake_block.h"

namespace {

using at::Tensor;

PyObject *g_cake_error; // bwd_dw_column_gb300.CakeError

// ---------------------------------------------------------------- arguments

Tensor tensor_or_none(PyObject *o, const char *what)
{
    if (o == Py_None)
        return Tensor();
    TORCH_CHECK_TYPE(THPVariable_Check(o), what, " is a tensor, got ", Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

Tensor tensor(PyObject *o, const char *what)
{
    TORCH_CHECK_TYPE(THPVariable_Check(o), what, " is a tensor, got ", Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

double number(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw python_error();
    return v;
}

bool truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw python_error();
    return v != 0;
}

// A whole number modulo 2^64.
uint64_t whole(PyObject *o)
{
    PyObject *i = PyNumber_Index(o);
    if (!i)
        throw python_error();
    const uint64_t v = PyLong_AsUnsignedLongLongMask(i);
    Py_DECREF(i);
    if (v == (uint64_t)-1 && PyErr_Occurred())
        throw python_error();
    return v;
}

int choice(PyObject *o, const char *what, const char *first, const char *second, const char *note)
{
    if (PyUnicode_Check(o)) {
        if (PyUnicode_CompareWithASCIIString(o, first) == 0)
            return 0;
        if (PyUnicode_CompareWithASCIIString(o, second) == 0)
            return 1;
    }
    TORCH_CHECK_VALUE(false, what, " is '", first, "' or '", second, "'", note);
}

void count(Py_ssize_t got, Py_ssize_t want)
{
    TORCH_CHECK_TYPE(got == want, "takes ", want, " arguments, got ", got);
}

// The device that every tensor (undefined: left out) is on.
int device_of(std::initializer_list<const Tensor *> tensors)
{
    int dev = -1;
    for (const Tensor *t : tensors) {
        if (!t->defined())
            continue;
        TORCH_CHECK_VALUE(t->is_cuda(), "every tensor must be on a CUDA device (no CPU path)");
        const int d = t->get_device();
        TORCH_CHECK_VALUE(dev < 0 || d == dev, "every tensor must be on the same device");
        dev = d;
    }
    return dev;
}

void bf16(const Tensor &t)
{
    TORCH_CHECK_TYPE(t.scalar_type() == at::kBFloat16, "activations are BF16, got ", t.scalar_type());
    TORCH_CHECK_VALUE(t.stride(-1) == 1 || t.numel() == 0, "the hidden dimension must be contiguous");
}

// A BF16 [rows, cols] matrix (undefined: none).
cake_tensor matrix(const Tensor &t, int64_t rows, int64_t cols, const char *what)
{
    if (!t.defined())
        return {nullptr, 0, 0};
    TORCH_CHECK_VALUE(t.dim() == 2 && t.size(0) == rows && t.size(1) == cols, what, " has shape ", t.sizes(),
                      ", expected [", rows, ", ", cols, "]");
    bf16(t);
    return {t.data_ptr(), t.stride(0), 0};
}

// (T, heads, H) of a [T, H] or [T, heads, H] tensor.
cake_shape rows_shape(const Tensor &t)
{
    TORCH_CHECK_VALUE(t.dim() == 2 || t.dim() == 3, "expected a [T, H] or [T, nh, H] tensor, got shape ", t.sizes());
    return t.dim() == 2 ? cake_shape{t.size(0), 1, t.size(1)} : cake_shape{t.size(0), t.size(1), t.size(2)};
}

// BF16 rows of `like`'s shape (undefined: none).
cake_tensor rows(const Tensor &t, const Tensor &like, const char *what)
{
    if (!t.defined())
        return {nullptr, 0, 0};
    TORCH_CHECK_VALUE(t.sizes() == like.sizes(), what, " has shape ", t.sizes(), ", expected ", like.sizes());
    bf16(t);
    return {t.data_ptr(), t.stride(0), t.dim() == 3 ? t.stride(1) : 0};
}

float *floats(const Tensor &t, int64_t n, const char *what)
{
    TORCH_CHECK_VALUE(t.scalar_type() == at::kFloat && t.numel() == n && t.is_contiguous(), what,
                      " must be a contiguous FP32 tensor of ", n, " elements");
    return t.data_ptr<float>();
}

Tensor weight(const Tensor &w, int64_t H, const char *what)
{
    TORCH_CHECK_VALUE(w.dim() == 1 && w.size(0) == H, what, " has shape ", w.sizes(), ", expected (", H, ",)");
    TORCH_CHECK_TYPE(w.scalar_type() == at::kBFloat16 || w.scalar_type() == at::kFloat, "weight is BF16 or FP32, got ",
                     w.scalar_type());
    return w.is_contiguous() ? w : w.contiguous();
}

cake_dtype dtype(const Tensor &w) { return w.defined() && w.scalar_type() == at::kFloat ? CAKE_FP32 : CAKE_BF16; }

const void *address(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

// -------------------------------------------------------------- allocation

// Straight from torch's allocator on the current stream: by way of the
// dispatcher a tensor took 1.4 us, and 0.8 like this.
Tensor fresh(at::IntArrayRef size, at::ScalarType type, int dev)
{
    return at::detail::empty_cuda(size, type, c10::Device(c10::kCUDA, (c10::DeviceIndex)dev), std::nullopt);
}

struct Scratch {
    Tensor t;
    void *at;
    size_t bytes;
};

Scratch workspace(const Tensor &given, size_t size, int dev)
{
    if (!given.defined()) {
        Tensor t = fresh({(int64_t)(size ? size : 256)}, at::kByte, dev);
        return {t, t.data_ptr(), size};
    }
    TORCH_CHECK_VALUE(given.is_contiguous(), "the workspace must be contiguous");
    return {given, given.data_ptr(), (size_t)given.numel() * given.element_size()};
}

// The tensors among a call's outputs that the caller has given count as changed in place.
void changed(std::initializer_list<const Tensor *> given)
{
    for (const Tensor *t : given)
        if (t->defined() && !t->is_inference())
            t->unsafeGetTensorImpl()->bump_version();
}

cake_stream_t stream(int dev) { return (cake_stream_t)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

// The outputs as a tuple; an error of the C call as a CakeError.
PyObject *done(cake_status st, const char *what, std::initializer_list<const Tensor *> outs)
{
    if (st != CAKE_OK) {
        PyObject *e = PyObject_CallFunction(g_cake_error, "is", (int)st, what);
        if (e) {
            PyErr_SetObject(g_cake_error, e);
            Py_DECREF(e);
        }
        return nullptr;
    }
    PyObject *t = PyTuple_New((Py_ssize_t)outs.size());
    Py_ssize_t i = 0;
    for (const Tensor *o : outs) {
        PyObject *v = Py_None;
        if (o->defined())
            v = THPVariable_Wrap(*o);
        else
            Py_INCREF(v);
        PyTuple_SET_ITEM(t, i++, v);
    }
    return t;
}

// What follows the arguments of every entry point: without the interpreter's
// lock, on the tensors' device.
#define ON_DEVICE(...)                          \
    const int dev = device_of({__VA_ARGS__});   \
    pybind11::gil_scoped_release nogil;         \
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev)

// -------------------------------------------------------------------- gated

int act(PyObject *o) { return choice(o, "act", "silu", "gelu", " (the tanh form)"); }

void gated_shapes(const Tensor &x, const Tensor &w_gate)
{
    TORCH_CHECK_VALUE(x.dim() == 2 && w_gate.dim() == 2, "expected x [T, H] and w_gate [F, H], got ", x.sizes(), " and ",
                      w_gate.sizes());
}

// x, w_gate, w_up, act, save, h, g, u
PyObject *gated_fwd(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 8);
    const Tensor x = tensor(a[0], "x"), wg = tensor(a[1], "w_gate"), wu = tensor(a[2], "w_up");
    const int kind = act(a[3]);
    const bool save = truth(a[4]);
    const Tensor gh = tensor_or_none(a[5], "h"), gg = tensor_or_none(a[6], "g"), gu = tensor_or_none(a[7], "u");
    Tensor h = gh, g = gg, u = gu;
    cake_status st;
    {
        ON_DEVICE(&x, &wg, &wu, &h, &g, &u);
        gated_shapes(x, wg);
        const int64_t T = x.size(0), H = x.size(1), F = wg.size(0);
        TORCH_CHECK_VALUE(save || (!g.defined() && !u.defined()), "g or u is given, but save is false");
        if (!h.defined())
            h = fresh({T, F}, at::kBFloat16, dev);
        if (save && !g.defined())
            g = fresh({T, F}, at::kBFloat16, dev);
        if (save && !u.defined())
            u = fresh({T, F}, at::kBFloat16, dev);
        const cake_tensor cx = matrix(x, T, H, "x"), cg = matrix(wg, F, H, "w_gate"), cu = matrix(wu, F, H, "w_up"),
                          oh = matrix(h, T, F, "h"), og = matrix(g, T, F, "g"), ou = matrix(u, T, F, "u");
        st = cake_gated_fwd(T, H, F, &cx, &cg, &cu, (cake_act)kind, &oh, save ? &og : nullptr, save ? &ou : nullptr,
                            stream(dev));
        if (st == CAKE_OK)
            changed({&gh, &gg, &gu});
    }
    return done(st, "cake_gated_fwd", {&h, &g, &u});
    END_HANDLE_TH_ERRORS
}

// dh, x, g, u, w_gate, w_up, act, need_dx, need_dw, workspace, dx, dw_gate, dw_up
PyObject *gated_bwd(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 13);
    const Tensor dh = tensor(a[0], "dh"), x = tensor(a[1], "x"), g = tensor(a[2], "g"), u = tensor(a[3], "u"),
                 wg = tensor(a[4], "w_gate"), wu = tensor(a[5], "w_up");
    const int kind = act(a[6]);
    const bool need_dx = truth(a[7]), need_dw = truth(a[8]);
    const Tensor given_ws = tensor_or_none(a[9], "workspace"), gx = tensor_or_none(a[10], "dx"),
                 gg = tensor_or_none(a[11], "dw_gate"), gu = tensor_or_none(a[12], "dw_up");
    Tensor dx = gx, dwg = gg, dwu = gu;
    cake_status st;
    {
        ON_DEVICE(&dh, &x, &g, &u, &wg, &wu, &given_ws, &dx, &dwg, &dwu);
        gated_shapes(x, wg);
        const int64_t T = x.size(0), H = x.size(1), F = wg.size(0);
        TORCH_CHECK_VALUE((need_dx || !dx.defined()) && (need_dw || (!dwg.defined() && !dwu.defined())),
                          "an output is given for a gradient that is not asked for");
        if (need_dx && !dx.defined())
            dx = fresh({T, H}, at::kBFloat16, dev);
        if (need_dw && !dwg.defined())
            dwg = fresh({F, H}, at::kBFloat16, dev);
        if (need_dw && !dwu.defined())
            dwu = fresh({F, H}, at::kBFloat16, dev);
        const cake_tensor cd = matrix(dh, T, F, "dh"), cx = matrix(x, T, H, "x"), cg = matrix(g, T, F, "g"),
                          cu = matrix(u, T, F, "u"), cwg = matrix(wg, F, H, "w_gate"), cwu = matrix(wu, F, H, "w_up"),
                          ox = matrix(dx, T, H, "dx"), og = matrix(dwg, F, H, "dw_gate"), ou = matrix(dwu, F, H, "dw_up");
        const Scratch ws = workspace(given_ws, cake_gated_bwd_workspace_size(T, H, F), dev);
        st = cake_gated_bwd(T, H, F, &cd, &cx, &cg, &cu, &cwg, &cwu, (cake_act)kind, need_dx ? &ox : nullptr,
                            need_dw ? &og : nullptr, need_dw ? &ou : nullptr, ws.at, ws.bytes, stream(dev));
        if (st == CAKE_OK)
            changed({&gx, &gg, &gu});
    }
    return done(st, "cake_gated_bwd", {&dx, &dwg, &dwu});
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------- rotary

int style(PyObject *o) { return choice(o, "style", "half", "adjacent", ""); }

void heads(const Tensor &t, const char *what)
{
    TORCH_CHECK_VALUE(!t.defined() || t.dim() == 3, what, " has shape ", t.sizes(), ", expected [T, heads, D]");
}

// [T, heads, D] views of the same tokens and D.
cake_tensor head_rows(const Tensor &t, int64_t T, int64_t nh, int64_t D, const char *what)
{
    if (!t.defined())
        return {nullptr, 0, 0};
    TORCH_CHECK_VALUE(t.dim() == 3 && t.size(0) == T && t.size(1) == nh && t.size(2) == D, what, " has shape ",
                      t.sizes(), ", expected [", T, ", ", nh, ", ", D, "]");
    bf16(t);
    return {t.data_ptr(), t.stride(0), t.stride(1)};
}

// The rotation; `turns` and `axes` become contiguous.
cake_rotary rotation(const Tensor &positions, Tensor &turns, Tensor &axes, int kind, int64_t T)
{
    const auto type = positions.scalar_type();
    TORCH_CHECK_TYPE(type == at::kInt || type == at::kLong, "positions are int32 or int64, got ", type);
    const int64_t dims = positions.dim();
    TORCH_CHECK_VALUE((dims == 1 || dims == 2) && positions.size(-1) == T, "positions have shape ", positions.sizes(),
                      ", expected [", T, "] or [axes, ", T, "]");
    TORCH_CHECK_TYPE(turns.scalar_type() == at::kLong && turns.dim() == 1,
                     "turns is an int64 tensor [pairs] (see cake_rotary_table)");
    turns = turns.contiguous();
    const int64_t n = dims == 2 ? positions.size(0) : 1;
    if (axes.defined()) {
        TORCH_CHECK_VALUE(axes.scalar_type() == at::kInt && axes.sizes() == turns.sizes(),
                          "axes is an int32 tensor of turns' shape");
        axes = axes.contiguous();
    } else {
        TORCH_CHECK_VALUE(n <= 1, "positions of several axes need each pair's axis");
    }
    cake_rotary r{};
    r.pairs = turns.numel();
    r.axes = n;
    r.turns = static_cast<const uint64_t *>(turns.data_ptr());
    r.axis = static_cast<const int32_t *>(address(axes));
    r.positions = positions.data_ptr();
    r.positions_int64 = type == at::kLong;
    r.axis_stride = dims == 2 ? positions.stride(0) : 0;
    r.token_stride = positions.stride(-1);
    r.style = kind;
    return r;
}

// Both weights, or without keys the queries', or none.
bool norm_weights(const Tensor &keys, Tensor &wq, Tensor &wk, int64_t D)
{
    TORCH_CHECK_VALUE(!keys.defined() || wq.defined() == wk.defined(),
                      "queries and keys are normed both or neither: give w_q and w_k, or none");
    if (!wq.defined() || !keys.defined())
        wk = Tensor();
    if (!wq.defined())
        return false;
    wq = weight(wq, D, "w_q");
    if (keys.defined())
        wk = weight(wk, D, "w_k");
    return true;
}

Tensor head_output(const Tensor &like, int dev) { return fresh(like.sizes(), at::kBFloat16, dev); }

// q, k, positions, turns, axes, w_q, w_k, eps, style, q_out, k_out, rstd_q, rstd_k
PyObject *rotary_fwd(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 13);
    const Tensor q = tensor(a[0], "q"), k = tensor_or_none(a[1], "k"), pos = tensor(a[2], "positions");
    Tensor turns = tensor(a[3], "turns"), axes = tensor_or_none(a[4], "axes"), wq = tensor_or_none(a[5], "w_q"),
           wk = tensor_or_none(a[6], "w_k");
    const float eps = (float)number(a[7]);
    const int kind = style(a[8]);
    const Tensor gq = tensor_or_none(a[9], "q_out"), gk = tensor_or_none(a[10], "k_out"),
                 grq = tensor_or_none(a[11], "rstd_q"), grk = tensor_or_none(a[12], "rstd_k");
    Tensor qo = gq, ko = gk, rq = grq, rk = grk;
    cake_status st;
    {
        ON_DEVICE(&q, &k, &pos, &turns, &axes, &wq, &wk, &qo, &ko, &rq, &rk);
        heads(q, "q");
        heads(k, "k");
        const int64_t T = q.size(0), nq = q.size(1), D = q.size(2), nk = k.defined() ? k.size(1) : 0;
        TORCH_CHECK_VALUE(k.defined() || (!ko.defined() && !rk.defined()), "an output for keys is given without keys");
        const bool norm = norm_weights(k, wq, wk, D);
        TORCH_CHECK_VALUE(norm || (!rq.defined() && !rk.defined()), "rstd is given, but there is no norm");
        const cake_rotary r = rotation(pos, turns, axes, kind, T);
        if (!qo.defined())
            qo = head_output(q, dev);
        if (k.defined() && !ko.defined())
            ko = head_output(k, dev);
        if (norm && !rq.defined())
            rq = fresh({T * nq}, at::kFloat, dev);
        if (norm && k.defined() && !rk.defined())
            rk = fresh({T * nk}, at::kFloat, dev);
        const cake_tensor cq = head_rows(q, T, nq, D, "q"), ck = head_rows(k, T, nk, D, "k"),
                          oq = head_rows(qo, T, nq, D, "q_out"), ok = head_rows(ko, T, nk, D, "k_out");
        st = cake_rotary_fwd(T, nq, nk, D, &cq, &ck, &r, address(wq), dtype(wq), address(wk), dtype(wk), eps, &oq, &ok,
                             rq.defined() ? floats(rq, T * nq, "rstd_q") : nullptr,
                             rk.defined() ? floats(rk, T * nk, "rstd_k") : nullptr, stream(dev));
        if (st == CAKE_OK)
            changed({&gq, &gk, &grq, &grk});
    }
    return done(st, "cake_rotary_fwd", {&qo, &ko, &rq, &rk});
    END_HANDLE_TH_ERRORS
}

// dq, dk, positions, turns, axes, q, k, rstd_q, rstd_k, w_q, w_k, style, workspace, dq_out, dk_out, dw_q, dw_k
PyObject *rotary_bwd(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 17);
    const Tensor dq = tensor(a[0], "dq"), dk = tensor_or_none(a[1], "dk"), pos = tensor(a[2], "positions");
    Tensor turns = tensor(a[3], "turns"), axes = tensor_or_none(a[4], "axes");
    Tensor q = tensor_or_none(a[5], "q"), k = tensor_or_none(a[6], "k"), rq = tensor_or_none(a[7], "rstd_q"),
           rk = tensor_or_none(a[8], "rstd_k"), wq = tensor_or_none(a[9], "w_q"), wk = tensor_or_none(a[10], "w_k");
    const int kind = style(a[11]);
    const Tensor given_ws = tensor_or_none(a[12], "workspace"), gq = tensor_or_none(a[13], "dq_out"),
                 gk = tensor_or_none(a[14], "dk_out"), gwq = tensor_or_none(a[15], "dw_q"),
                 gwk = tensor_or_none(a[16], "dw_k");
    Tensor qo = gq, ko = gk, dwq = gwq, dwk = gwk;
    cake_status st;
    {
        ON_DEVICE(&dq, &dk, &pos, &turns, &axes, &q, &k, &rq, &rk, &wq, &wk, &given_ws, &qo, &ko, &dwq, &dwk);
        heads(dq, "dq");
        heads(dk, "dk");
        const int64_t T = dq.size(0), nq = dq.size(1), D = dq.size(2), nk = dk.defined() ? dk.size(1) : 0;
        TORCH_CHECK_VALUE(dk.defined() || (!ko.defined() && !dwk.defined()), "an output for keys is given without keys");
        const bool norm = norm_weights(dk, wq, wk, D), keys = norm && dk.defined();
        TORCH_CHECK_VALUE(!norm || (q.defined() && rq.defined() && (!keys || (k.defined() && rk.defined()))),
                          "the norm's gradient needs the forward's inputs and rstd");
        TORCH_CHECK_VALUE(norm || (!dwq.defined() && !dwk.defined()),
                          "a weight's gradient is given, but there is no norm");
        if (!norm)
            q = rq = Tensor();
        if (!keys)
            k = rk = Tensor();
        const cake_rotary r = rotation(pos, turns, axes, kind, T);
        if (!qo.defined())
            qo = head_output(dq, dev);
        if (dk.defined() && !ko.defined())
            ko = head_output(dk, dev);
        if (norm && !dwq.defined())
            dwq = fresh({D}, at::kFloat, dev);
        if (keys && !dwk.defined())
            dwk = fresh({D}, at::kFloat, dev);
        const Scratch ws = norm ? workspace(given_ws, cake_rotary_bwd_workspace_size(T, nq, nk, D), dev)
                                : Scratch{Tensor(), nullptr, 0};
        const cake_tensor cq = head_rows(dq, T, nq, D, "dq"), ck = head_rows(dk, T, nk, D, "dk"),
                          vq = head_rows(q, T, nq, D, "q"), vk = head_rows(k, T, nk, D, "k"),
                          oq = head_rows(qo, T, nq, D, "dq_out"), ok = head_rows(ko, T, nk, D, "dk_out");
        st = cake_rotary_bwd(T, nq, nk, D, &cq, &ck, &r, &vq, &vk, norm ? floats(rq, T * nq, "rstd_q") : nullptr,
                             keys ? floats(rk, T * nk, "rstd_k") : nullptr, address(wq), dtype(wq), address(wk),
                             dtype(wk), &oq, &ok, norm ? floats(dwq, D, "dw_q") : nullptr,
                             keys ? floats(dwk, D, "dw_k") : nullptr, ws.at, ws.bytes, stream(dev));
        if (st == CAKE_OK)
            changed({&gq, &gk, &gwq, &gwk});
    }
    return done(st, "cake_rotary_bwd", {&qo, &ko, &dwq, &dwk});
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------ dropout

// A seed on the host, or a seed and a number added to the offset on the device.
struct Seed {
    uint64_t host;
    Tensor device;
};

Seed seed_of(PyObject *o)
{
    if (!THPVariable_Check(o))
        return {whole(o), Tensor()};
    return {0, THPVariable_Unpack(o)};
}

const uint64_t *rng(const Seed &s)
{
    if (!s.device.defined())
        return nullptr;
    TORCH_CHECK_VALUE(s.device.scalar_type() == at::kLong && s.device.numel() == 2 && s.device.is_contiguous(),
                      "a seed on the device is a contiguous int64 tensor of two: the seed, and a number added to offset");
    return static_cast<const uint64_t *>(s.device.data_ptr());
}

// x, p, seed, offset, residual, y
PyObject *dropout(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 6);
    const Tensor x = tensor(a[0], "x");
    const double p = number(a[1]);
    const Seed seed = seed_of(a[2]);
    const uint64_t offset = whole(a[3]);
    const Tensor res = tensor_or_none(a[4], "residual"), given = tensor_or_none(a[5], "y");
    Tensor y = given;
    cake_status st;
    {
        ON_DEVICE(&x, &res, &y, &seed.device);
        const cake_shape s = rows_shape(x);
        if (!y.defined())
            y = fresh(x.sizes(), at::kBFloat16, dev);
        const cake_tensor cx = rows(x, x, "x"), ce = rows(res, x, "residual"), cy = rows(y, x, "y");
        st = cake_dropout(&s, &cx, &ce, p, seed.host, offset, rng(seed), &cy, stream(dev));
        if (st == CAKE_OK)
            changed({&given});
    }
    if (st != CAKE_OK)
        return done(st, "cake_dropout", {});
    return THPVariable_Wrap(y);
    END_HANDLE_TH_ERRORS
}

// x, residual, w, p, seed, offset, eps, y, h_new, rstd
PyObject *dropout_norm_fwd(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 10);
    const Tensor x = tensor(a[0], "x"), res = tensor(a[1], "residual");
    Tensor w = tensor(a[2], "w");
    const double p = number(a[3]);
    const Seed seed = seed_of(a[4]);
    const uint64_t offset = whole(a[5]);
    const float eps = (float)number(a[6]);
    const Tensor gy = tensor_or_none(a[7], "y"), gh = tensor_or_none(a[8], "h_new"), gr = tensor_or_none(a[9], "rstd");
    Tensor y = gy, h = gh, r = gr;
    cake_status st;
    {
        ON_DEVICE(&x, &res, &w, &y, &h, &r, &seed.device);
        const cake_shape s = rows_shape(x);
        w = weight(w, s.hidden, "w");
        if (!y.defined())
            y = fresh(x.sizes(), at::kBFloat16, dev);
        if (!h.defined())
            h = fresh(x.sizes(), at::kBFloat16, dev);
        if (!r.defined())
            r = fresh({s.tokens * s.heads}, at::kFloat, dev);
        const cake_tensor cx = rows(x, x, "x"), ce = rows(res, x, "residual"), cy = rows(y, x, "y"),
                          ch = rows(h, x, "h_new");
        st = cake_dropout_norm_fwd(&s, &cx, &ce, w.data_ptr(), dtype(w), p, seed.host, offset, rng(seed), eps, &cy, &ch,
                                   floats(r, s.tokens * s.heads, "rstd"), stream(dev));
        if (st == CAKE_OK)
            changed({&gy, &gh, &gr});
    }
    return done(st, "cake_dropout_norm_fwd", {&y, &h, &r});
    END_HANDLE_TH_ERRORS
}

// dy, h_new, rstd, w, p, seed, offset, dh, workspace, dx, dresidual, dw
PyObject *dropout_norm_bwd(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 12);
    const Tensor dy = tensor(a[0], "dy"), h = tensor(a[1], "h_new"), r = tensor(a[2], "rstd");
    Tensor w = tensor(a[3], "w");
    const double p = number(a[4]);
    const Seed seed = seed_of(a[5]);
    const uint64_t offset = whole(a[6]);
    const Tensor dh = tensor_or_none(a[7], "dh"), given_ws = tensor_or_none(a[8], "workspace"),
                 gx = tensor_or_none(a[9], "dx"), ge = tensor_or_none(a[10], "dresidual"),
                 gw = tensor_or_none(a[11], "dw");
    Tensor dx = gx, de = ge, dw = gw;
    cake_status st;
    {
        ON_DEVICE(&dy, &h, &r, &w, &dh, &given_ws, &dx, &de, &dw, &seed.device);
        const cake_shape s = rows_shape(dy);
        w = weight(w, s.hidden, "w");
        if (!dx.defined())
            dx = fresh(dy.sizes(), at::kBFloat16, dev);
        if (!de.defined())
            de = fresh(dy.sizes(), at::kBFloat16, dev);
        if (!dw.defined())
            dw = fresh({s.hidden}, at::kFloat, dev);
        const Scratch ws = workspace(given_ws, cake_dropout_norm_bwd_workspace_size(&s), dev);
        const cake_tensor cy = rows(dy, dy, "dy"), ch = rows(h, dy, "h_new"), cd = rows(dh, dy, "dh"),
                          ox = rows(dx, dy, "dx"), oe = rows(de, dy, "dresidual");
        st = cake_dropout_norm_bwd(&s, &cy, &cd, &ch, floats(r, s.tokens * s.heads, "rstd"), w.data_ptr(), dtype(w), p,
                                   seed.host, offset, rng(seed), &ox, &oe, floats(dw, s.hidden, "dw"), ws.at, ws.bytes,
                                   stream(dev));
        if (st == CAKE_OK)
            changed({&gx, &ge, &gw});
    }
    return done(st, "cake_dropout_norm_bwd", {&de, &dx, &dw});
    END_HANDLE_TH_ERRORS
}

// The class of the errors that a call's status becomes.
PyObject *set_error(PyObject *, PyObject *type)
{
    Py_INCREF(type);
    Py_XDECREF(g_cake_error);
    g_cake_error = type;
    Py_RETURN_NONE;
}

#define FAST(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}

PyMethodDef methods[] = {FAST(gated_fwd),        FAST(gated_bwd),        FAST(rotary_fwd),
                         FAST(rotary_bwd),       FAST(dropout),          FAST(dropout_norm_fwd),
                         FAST(dropout_norm_bwd), {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_cake_block", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__cake_block() { return PyModule_Create(&module); }
