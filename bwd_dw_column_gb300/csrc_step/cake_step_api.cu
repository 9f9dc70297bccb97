// cake_step_api.cu -- the C ABI of the training-step operators: argument
// validation, workspace layout and dispatch to the launchers.  Host code only.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdlib>
#include <vector>

#include <cuda_runtime.h>

#include "../../include/cake_step_test.h"
#include "cake_call.h"
#include "cake_step_launch.h"

using namespace cake;

namespace {

// The limit of the kernels' waits, and what never comes (cake_step_wait_test).
struct Waits {
    uint64_t ns = kWaitLimitNs;
    int withhold = 0;
};
thread_local Waits t_waits;

// The weights and the gate of a sandwich norm.
cake_status check_sandwich(const cake_shape *shape, const void *w_post, cake_dtype post_dtype, const void *w_pre,
                           cake_dtype pre_dtype, const float *gate_rows, const cake_tensor *gate, float scale)
{
    if (!good_dtype(post_dtype) || !good_dtype(pre_dtype) || std::isnan(scale))
        return CAKE_ERR_INVALID;
    if (gate_rows && has(gate))
        return CAKE_ERR_INVALID;
    if (shape->tokens == 0)
        return CAKE_OK;
    if (!w_post || !w_pre)
        return CAKE_ERR_INVALID;
    if (!aligned16(w_post) || !aligned16(w_pre))
        return CAKE_ERR_UNSUPPORTED;
    if (gate_rows && (reinterpret_cast<uintptr_t>(gate_rows) & 3u))
        return CAKE_ERR_UNSUPPORTED;
    return has(gate) ? check_tensor(gate, shape) : CAKE_OK;
}

SandwichLayout sandwich_layout(const SandwichPlan &plan, const cake_shape *shape, uint32_t rows, int ntens)
{
    SandwichLayout L;
    L.H = (int)shape->hidden;
    L.nvec = L.H / 8;
    L.cluster = plan.cluster;
    L.cols = plan.cols;
    L.W = plan.W;
    L.groups = plan.groups;
    L.stages = plan.stages;
    L.ntens = ntens;
    L.rows = rows;
    L.nh = (uint32_t)shape->heads;
    L.rows_per_cta = plan.rows_per_cta;
    L.inv_h = 1.0f / (float)L.H;
    return L;
}

} // namespace

extern "C" cake_status cake_step_wait_test(uint32_t wait_limit_us, int withhold)
{
    if (wait_limit_us > 1000000 || withhold < 0 || withhold > 2 || (wait_limit_us == 0 && withhold))
        return CAKE_ERR_INVALID;
    t_waits.ns = wait_limit_us ? (uint64_t)wait_limit_us * 1000u : kWaitLimitNs;
    t_waits.withhold = withhold;
    return CAKE_OK;
}

extern "C" int cake_step_rows_meet(const cake_shape *shape, const cake_tensor *a, const cake_tensor *b)
{
    return meet(memory(a, shape), memory(b, shape));
}

// ------------------------------------------------------------ sandwich norm

extern "C" cake_status cake_sandwich_fwd(const cake_shape *shape, const cake_tensor *z, const cake_tensor *x,
                                         const void *w_post, cake_dtype w_post_dtype, const void *w_pre,
                                         cake_dtype w_pre_dtype, const float *gate_rows, const cake_tensor *gate,
                                         float scale, float eps, const cake_tensor *y, const cake_tensor *h_new,
                                         float *rstd_post, float *rstd_pre, cake_stream_t stream)
{
    uint32_t rows = 0;
    cake_status st = check_shape(shape, &rows);
    if (st != CAKE_OK)
        return st;
    if (!(eps >= 0.0f))
        return CAKE_ERR_INVALID;
    if ((st = check_sandwich(shape, w_post, w_post_dtype, w_pre, w_pre_dtype, gate_rows, gate, scale)) != CAKE_OK)
        return st;
    if (rows == 0)
        return CAKE_OK;
    if ((st = check_tensor(z, shape)) != CAKE_OK || (st = check_tensor(x, shape)) != CAKE_OK ||
        (st = check_out_tensor(y, shape)) != CAKE_OK || (st = check_out_tensor(h_new, shape)) != CAKE_OK ||
        (st = check_rows_f32(rstd_post)) != CAKE_OK || (st = check_rows_f32(rstd_pre)) != CAKE_OK)
        return st;
    // a row is written after it is read: y and h_new may be an input's view
    // exactly, and not straddle other rows of one; nothing else is shared
    const uint64_t rb = (uint64_t)rows * 4, wb = (uint64_t)shape->hidden;
    const Memory written[4] = {memory(rstd_post, rb), memory(rstd_pre, rb), memory(y, shape), memory(h_new, shape)};
    const Memory lists[3] = {memory(gate_rows, rb), memory(w_post, wb * (w_post_dtype == CAKE_FP32 ? 4 : 2)),
                             memory(w_pre, wb * (w_pre_dtype == CAKE_FP32 ? 4 : 2))};
    const Memory rows_in[3] = {memory(z, shape), memory(x, shape), memory(gate, shape)};
    if (any_meet(written, 4, lists, 3) || any_meet(written, 2, rows_in, 3))
        return CAKE_ERR_INVALID;
    const cake_tensor *outs[2] = {y, h_new}, *ins[3] = {z, x, has(gate) ? gate : nullptr};
    for (const cake_tensor *o : outs)
        for (const cake_tensor *i : ins)
            if (i && meet(memory(o, shape), memory(i, shape)) && !same_view(o, i, shape))
                return CAKE_ERR_INVALID;
    SandwichFwdParams p{};
    const SandwichPlan plan = sandwich_plan((int)shape->hidden, rows, has(gate) ? 3 : 2, false);
    p.L = sandwich_layout(plan, shape, rows, has(gate) ? 3 : 2);
    p.eps = eps;
    p.scale = scale;
    p.in[0] = make_view(z, shape);
    p.in[1] = make_view(x, shape);
    p.in[2] = make_view(gate, shape);
    p.y = make_view(y, shape);
    p.h_new = make_view(h_new, shape);
    p.gate_rows = gate_rows;
    p.w_post = w_post;
    p.w_pre = w_pre;
    p.post_f32 = w_post_dtype == CAKE_FP32;
    p.pre_f32 = w_pre_dtype == CAKE_FP32;
    p.rstd_post = rstd_post;
    p.rstd_pre = rstd_pre;
    p.wait_ns = t_waits.ns;
    p.withhold = t_waits.withhold;
    if (step_status_ptr(&p.status) != cudaSuccess)
        return CAKE_ERR_CUDA;
    return cuda_status(launch_sandwich_fwd(p, plan, cu(stream)));
}

extern "C" cake_status cake_sandwich_bwd_plan(const cake_shape *shape, int tensors, int plan[9])
{
    uint32_t rows = 0;
    cake_status st = check_shape(shape, &rows);
    if (st != CAKE_OK)
        return st;
    if (!plan || rows == 0 || tensors < 3 || tensors > 5)
        return CAKE_ERR_INVALID;
    const SandwichPlan p = sandwich_plan((int)shape->hidden, rows, tensors, true);
    const SandwichBuild b = sandwich_build(p);
    const int got[9] = {b.vpt,     b.cl,     b.rw,     b.many, b.half,
                        p.cluster, p.groups, p.stages, (int)((p.rows_per_cta + p.groups - 1) / p.groups)};
    std::copy(got, got + 9, plan);
    return CAKE_OK;
}

extern "C" size_t cake_sandwich_bwd_workspace_size(const cake_shape *shape)
{
    uint32_t rows = 0;
    if (check_shape(shape, &rows) != CAKE_OK || rows == 0)
        return 0;
    // the plan depends on the number of staged tensors: room for each choice
    int parts = 0;
    for (int ntens = 3; ntens <= 5; ++ntens)
        parts = std::max(parts, sandwich_plan((int)shape->hidden, rows, ntens, true).parts);
    return (size_t)2 * parts * shape->hidden * sizeof(float2);
}

extern "C" cake_status cake_sandwich_bwd(const cake_shape *shape, const cake_tensor *dy, const cake_tensor *dh,
                                         const cake_tensor *h_new, const cake_tensor *z, const float *rstd_post,
                                         const float *rstd_pre, const void *w_post, cake_dtype w_post_dtype,
                                         const void *w_pre, cake_dtype w_pre_dtype, const float *gate_rows,
                                         const cake_tensor *gate, float scale, const cake_tensor *dx,
                                         const cake_tensor *dz, float *dw_post, float *dw_pre, float *dgate_rows,
                                         const cake_tensor *dgate, void *workspace, size_t workspace_bytes,
                                         cake_stream_t stream)
{
    uint32_t rows = 0;
    cake_status st = check_shape(shape, &rows);
    if (st != CAKE_OK)
        return st;
    if ((st = check_sandwich(shape, w_post, w_post_dtype, w_pre, w_pre_dtype, gate_rows, gate, scale)) != CAKE_OK)
        return st;
    if (!dw_post || !dw_pre || std::abs(reinterpret_cast<intptr_t>(dw_post) - reinterpret_cast<intptr_t>(dw_pre)) <
                                   (intptr_t)(shape->hidden * sizeof(float)))
        return CAKE_ERR_INVALID; // missing, or one reaches into the other
    if (!aligned16(dw_post) || !aligned16(dw_pre))
        return CAKE_ERR_UNSUPPORTED;
    if ((dgate_rows && !gate_rows) || (has(dgate) && !has(gate)))
        return CAKE_ERR_INVALID;
    const int H = (int)shape->hidden;
    if (rows == 0) {
        cudaError_t e = cudaMemsetAsync(dw_post, 0, (size_t)H * sizeof(float), cu(stream));
        if (e == cudaSuccess)
            e = cudaMemsetAsync(dw_pre, 0, (size_t)H * sizeof(float), cu(stream));
        return cuda_status(e);
    }
    if ((st = check_tensor(dy, shape)) != CAKE_OK || (st = check_tensor(h_new, shape)) != CAKE_OK ||
        (st = check_tensor(z, shape)) != CAKE_OK || (has(dh) && (st = check_tensor(dh, shape)) != CAKE_OK) ||
        (st = check_out_tensor(dx, shape)) != CAKE_OK || (st = check_out_tensor(dz, shape)) != CAKE_OK ||
        (has(dgate) && (st = check_out_tensor(dgate, shape)) != CAKE_OK) ||
        (st = check_rows_f32(rstd_post)) != CAKE_OK || (st = check_rows_f32(rstd_pre)) != CAKE_OK ||
        (dgate_rows && (st = check_rows_f32(dgate_rows)) != CAKE_OK))
        return st;
    const size_t need = cake_sandwich_bwd_workspace_size(shape);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != CAKE_OK)
        return st;
    // outputs are written while later rows of the inputs are still being read
    const uint64_t rb = (uint64_t)rows * 4, wb = (uint64_t)H;
    const Memory written[7] = {memory(dx, shape),       memory(dz, shape),     memory(dgate, shape),
                               memory(dgate_rows, rb),  memory(dw_post, wb * 4), memory(dw_pre, wb * 4),
                               memory(workspace, need)};
    const Memory read[10] = {memory(dy, shape),    memory(h_new, shape),
                             memory(z, shape),     memory(dh, shape),
                             memory(gate, shape),  memory(gate_rows, rb),
                             memory(rstd_post, rb), memory(rstd_pre, rb),
                             memory(w_post, wb * (w_post_dtype == CAKE_FP32 ? 4 : 2)),
                             memory(w_pre, wb * (w_pre_dtype == CAKE_FP32 ? 4 : 2))};
    if (any_meet(written, 7, read, 10))
        return CAKE_ERR_INVALID;
    SandwichBwdParams p{};
    p.in[0] = make_view(h_new, shape);
    p.in[1] = make_view(z, shape);
    p.in[2] = make_view(dy, shape);
    int ntens = 3;
    if (has(gate))
        p.in[ntens++] = make_view(gate, shape);
    if (has(dh))
        p.in[ntens++] = make_view(dh, shape);
    const SandwichPlan plan = sandwich_plan(H, rows, ntens, true);
    p.L = sandwich_layout(plan, shape, rows, ntens);
    p.scale = scale;
    p.gate = has(gate) ? 2 : gate_rows ? 1 : 0;
    p.has_dh = has(dh);
    p.dx = make_view(dx, shape);
    p.dz = make_view(dz, shape);
    p.dgate = make_view(dgate, shape);
    p.gate_rows = gate_rows;
    p.dgate_rows = dgate_rows;
    p.rstd_post = rstd_post;
    p.rstd_pre = rstd_pre;
    p.w_post = w_post;
    p.w_pre = w_pre;
    p.post_f32 = w_post_dtype == CAKE_FP32;
    p.pre_f32 = w_pre_dtype == CAKE_FP32;
    p.partials = static_cast<float2 *>(workspace);
    p.wait_ns = t_waits.ns;
    p.withhold = t_waits.withhold;
    if (step_status_ptr(&p.status) != cudaSuccess || launch_sandwich_bwd(p, plan, cu(stream)) != cudaSuccess)
        return CAKE_ERR_CUDA;
    SandwichReduceParams rp{p.partials, plan.parts, H, {dw_post, dw_pre}};
    return cuda_status(launch_sandwich_reduce(rp, cu(stream)));
}

// ----------------------------------------------- gradient norm and clipping

namespace {

constexpr int64_t kGradMostTensors = 1000000;

struct Range {
    uintptr_t lo, hi;
    int64_t id; // tensor; an output's is -1 - tensor where it is not the input itself; the norm's is INT64_MIN
};

// The tensors of a call, checked; `clip`: outputs too.
cake_status check_grads(const void *const *data, const int64_t *counts, const int32_t *dtypes, void *const *outs,
                        const int32_t *out_dtypes, int64_t n, bool clip, const float *norm, const Memory &scratch)
{
    if (n < 0 || (n > 0 && (!data || !counts || !dtypes)) || (outs == nullptr) != (out_dtypes == nullptr))
        return CAKE_ERR_INVALID;
    if (n > kGradMostTensors)
        return CAKE_ERR_UNSUPPORTED;
    std::vector<Range> written, read;
    if (clip) {
        written.reserve((size_t)n + 1);
        written.push_back({reinterpret_cast<uintptr_t>(norm), reinterpret_cast<uintptr_t>(norm) + 4, INT64_MIN});
    }
    uint64_t chunks = 0;
    for (int64_t i = 0; i < n; ++i) {
        if (counts[i] < 0 || !good_dtype(dtypes[i]) || (outs && !good_dtype(out_dtypes[i])))
            return CAKE_ERR_INVALID;
        chunks += (uint64_t)(counts[i] / kGradChunk) + 1;
        if (chunks >= (uint64_t(1) << 31)) // a launch counts its chunks in 32 bits
            return CAKE_ERR_UNSUPPORTED;
        if (counts[i] == 0)
            continue;
        const uintptr_t size = dtypes[i] == CAKE_FP32 ? 4 : 2, a = reinterpret_cast<uintptr_t>(data[i]);
        if (!a)
            return CAKE_ERR_INVALID;
        if (a % size)
            return CAKE_ERR_UNSUPPORTED;
        if (!clip)
            continue;
        const Range in{a, a + size * (uintptr_t)counts[i], i};
        if (!outs) {
            written.push_back(in);
            continue;
        }
        const uintptr_t osize = out_dtypes[i] == CAKE_FP32 ? 4 : 2, o = reinterpret_cast<uintptr_t>(outs[i]);
        if (!o)
            return CAKE_ERR_INVALID;
        if (o % osize)
            return CAKE_ERR_UNSUPPORTED;
        written.push_back({o, o + osize * (uintptr_t)counts[i], o == a && osize == size ? i : -1 - i});
        read.push_back(in);
    }
    if (meet(scratch, memory(norm, 4)))
        return CAKE_ERR_INVALID;
    // (of clipping, the norm is among the written ranges below)
    for (int64_t i = 0; i < n; ++i) {
        const Memory in = memory(data[i], (uint64_t)counts[i] * (dtypes[i] == CAKE_FP32 ? 4 : 2));
        if (meet(scratch, in) || (!clip && meet(memory(norm, 4), in)) ||
            (outs && meet(scratch, memory(outs[i], (uint64_t)counts[i] * (out_dtypes[i] == CAKE_FP32 ? 4 : 2)))))
            return CAKE_ERR_INVALID;
    }
    // written ranges share memory with no other range but their own input
    const auto by_lo = [](const Range &x, const Range &y) { return x.lo < y.lo; };
    std::sort(written.begin(), written.end(), by_lo);
    for (size_t k = 1; k < written.size(); ++k)
        if (written[k].lo < written[k - 1].hi)
            return CAKE_ERR_INVALID;
    for (const Range &r : read) {
        // the written ranges are disjoint, so those that meet r follow one another
        auto it = std::upper_bound(written.begin(), written.end(), r, by_lo);
        if (it != written.begin())
            --it;
        for (; it != written.end() && it->lo < r.hi; ++it)
            if (it->hi > r.lo && it->id != r.id)
                return CAKE_ERR_INVALID;
    }
    return CAKE_OK;
}

int64_t grad_launches(int64_t n)
{
    return n <= 0 || n > kGradMostTensors ? 0 : (n + kGradMaxTensors - 1) / kGradMaxTensors;
}

// The launches' tensors [i0, i1) as parameters; returns the CTAs.
template <int N>
int fill_grads(GradParams<N> &p, const void *const *data, const int64_t *counts, const int32_t *dtypes,
               void *const *outs, const int32_t *out_dtypes, int64_t i0, int64_t i1, int most, int64_t chunk = kGradChunk)
{
    uint64_t chunks = 0;
    int k = 0;
    for (int64_t i = i0; i < i1; ++i) {
        if (counts[i] == 0)
            continue;
        GradDesc &d = p.t[k++];
        d.src = data[i];
        d.dst = outs ? outs[i] : const_cast<void *>(data[i]);
        d.count = counts[i];
        d.chunk0 = (uint32_t)chunks;
        const bool o32 = outs ? out_dtypes[i] == CAKE_FP32 : dtypes[i] == CAKE_FP32;
        d.flags = (dtypes[i] == CAKE_FP32 ? kGradSrcF32 : 0) | (o32 ? kGradDstF32 : 0) |
                  (aligned16(d.src) && aligned16(d.dst) ? kGradVector : 0);
        chunks += (uint64_t)((counts[i] + chunk - 1) / chunk);
    }
    p.n = k;
    p.chunks = (uint32_t)chunks;
    return (int)std::min<uint64_t>(chunks, most);
}

template <int N>
cudaError_t run_grads(const void *const *data, const int64_t *counts, const int32_t *dtypes, void *const *outs,
                      const int32_t *out_dtypes, int64_t n, bool clip, float max_norm, float eps, float *norm,
                      double *partials, cudaStream_t s)
{
    // the parameters of a launch are too large for the stack of a small thread
    static thread_local GradParams<N> p;
    if constexpr (N == kGradFewTensors) {
        int64_t pieces = 0;
        for (int64_t i = 0; i < n && pieces <= kGradOnePieces; ++i)
            pieces += (counts[i] + kGradPiece - 1) / kGradPiece;
        if (pieces > 0 && pieces <= kGradOnePieces) {
            fill_grads(p, data, counts, dtypes, outs, out_dtypes, 0, n, 1, kGradPiece);
            p.max_norm = max_norm;
            p.eps = eps;
            p.in_place = outs == nullptr;
            p.norm = norm;
            return launch_grad_one(p, clip, s);
        }
    }
    int total = 0;
    for (int64_t i0 = 0; i0 < n; i0 += N) {
        const int ctas = fill_grads(p, data, counts, dtypes, outs, out_dtypes, i0, std::min(n, i0 + N), kGradCtas);
        if (ctas == 0)
            continue;
        p.partials = partials + total;
        total += ctas;
        cudaError_t e = launch_grad_sumsq(p, ctas, s);
        if (e != cudaSuccess)
            return e;
    }
    if (total == 0)
        return cudaMemsetAsync(norm, 0, sizeof(float), s);
    if (!clip)
        return launch_grad_final(partials, total, norm, s);
    bool first = true;
    for (int64_t i0 = 0; i0 < n; i0 += N) {
        const int ctas = fill_grads(p, data, counts, dtypes, outs, out_dtypes, i0, std::min(n, i0 + N), kGradClipCtas);
        if (ctas == 0)
            continue;
        p.partials = partials;
        p.npartials = total;
        p.max_norm = max_norm;
        p.eps = eps;
        p.in_place = outs == nullptr;
        p.norm = first ? norm : nullptr;
        cudaError_t e = launch_grad_clip(p, ctas, s);
        if (e != cudaSuccess)
            return e;
        first = false;
    }
    return cudaSuccess;
}

cake_status grads(const void *const *data, const int64_t *counts, const int32_t *dtypes, void *const *outs,
                  const int32_t *out_dtypes, int64_t n, bool clip, float max_norm, float eps, float *norm,
                  void *workspace, size_t workspace_bytes, cake_stream_t stream)
{
    cake_status st = check_rows_f32(norm);
    if (st != CAKE_OK)
        return st;
    const size_t need = cake_grad_norm_workspace_size(n);
    if (n > 0 && (st = check_workspace(workspace, workspace_bytes, need)) != CAKE_OK)
        return st;
    try {
        st = check_grads(data, counts, dtypes, outs, out_dtypes, n, clip, norm, memory(workspace, need));
    } catch (...) { // no host memory for the list
        return CAKE_ERR_WORKSPACE;
    }
    if (st != CAKE_OK)
        return st;
    if (n == 0)
        return cuda_status(cudaMemsetAsync(norm, 0, sizeof(float), cu(stream)));
    double *partials = static_cast<double *>(workspace);
    // the fewer parameters a launch carries, the sooner it starts
    const auto run = n <= kGradFewTensors    ? run_grads<kGradFewTensors>
                     : n <= kGradSomeTensors ? run_grads<kGradSomeTensors>
                                             : run_grads<kGradMaxTensors>;
    return cuda_status(run(data, counts, dtypes, outs, out_dtypes, n, clip, max_norm, eps, norm, partials, cu(stream)));
}

} // namespace

extern "C" size_t cake_grad_norm_workspace_size(int64_t n)
{
    return (size_t)grad_launches(n) * kGradCtas * sizeof(double);
}

extern "C" cake_status cake_grad_norm(const void *const *data, const int64_t *counts, const int32_t *dtypes, int64_t n,
                                      float *norm, void *workspace, size_t workspace_bytes, cake_stream_t stream)
{
    return grads(data, counts, dtypes, nullptr, nullptr, n, false, 0.f, 0.f, norm, workspace, workspace_bytes, stream);
}

extern "C" cake_status cake_grad_clip(void *const *data, const int64_t *counts, const int32_t *dtypes,
                                      void *const *outs, const int32_t *out_dtypes, int64_t n, float max_norm,
                                      float eps, float *norm, void *workspace, size_t workspace_bytes,
                                      cake_stream_t stream)
{
    if (!(max_norm >= 0.0f) || !(eps >= 0.0f) || std::isinf(eps))
        return CAKE_ERR_INVALID;
    return grads(data, counts, dtypes, outs, out_dtypes, n, true, max_norm, eps, norm, workspace, workspace_bytes,
                 stream);
}

// ---------------------------------------------------------------- embedding

namespace {

Memory table_memory(const void *table, int dtype, int64_t vocab, int64_t hidden, int64_t stride)
{
    return memory(table, ((uint64_t)(vocab - 1) * (uint64_t)stride + (uint64_t)hidden) * (dtype == CAKE_FP32 ? 4 : 2));
}

cake_status check_embedding(const void *ids, int ids_int64, int64_t tokens, const void *table, int dtype,
                            int64_t vocab, int64_t hidden, int64_t stride, float scale, const cake_tensor *rows,
                            bool rows_out)
{
    if (tokens < 0 || vocab < 1 || hidden < 1 || !good_dtype(dtype) || (ids_int64 != 0 && ids_int64 != 1) ||
        std::isnan(scale) || !table || (tokens > 0 && !ids))
        return CAKE_ERR_INVALID;
    if (hidden % 8 != 0 || hidden > CAKE_MAX_HIDDEN || tokens >= (int64_t(1) << 31) || vocab >= (int64_t(1) << 31))
        return CAKE_ERR_UNSUPPORTED;
    if (!aligned16(table) || stride % (dtype == CAKE_FP32 ? 4 : 8) != 0 || (vocab > 1 && stride < hidden) ||
        stride >= (int64_t(1) << 31))
        return CAKE_ERR_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(ids) & (ids_int64 ? 7u : 3u))
        return CAKE_ERR_UNSUPPORTED;
    if (tokens == 0)
        return CAKE_OK;
    const cake_shape shape{tokens, 1, hidden};
    cake_status st = rows_out ? check_out_tensor(rows, &shape) : check_tensor(rows, &shape);
    if (st != CAKE_OK)
        return st;
    // what is written, the rows or the table, shares memory with nothing else
    const Memory r = memory(rows, &shape), t = table_memory(table, dtype, vocab, hidden, stride);
    const Memory i = memory(ids, (uint64_t)tokens * (ids_int64 ? 8 : 4));
    return meet(r, t) || meet(i, rows_out ? r : t) ? CAKE_ERR_INVALID : CAKE_OK;
}

// Sizes of a gradient call; they depend on the shape alone.
struct EmbedPlan {
    int bits, passes, tiles, window, windows, slices, threads;
    int cluster; // CTAs of the one-launch sort; 0: a launch per pass
    uint32_t tile_keys;
    size_t present_bytes, hist_bytes, pairs_bytes, part_bytes, meta_bytes, total;
};

EmbedPlan embed_plan(int64_t T, int64_t V, int64_t H)
{
    EmbedPlan e{};
    int key_bits = 1;
    while ((V >> key_bits) != 0) // keys 0 .. V
        ++key_bits;
    e.passes = (key_bits + kSortMaxBits - 1) / kSortMaxBits;
    e.bits = (key_bits + e.passes - 1) / e.passes;
    e.cluster = 0;
    if (T <= kClusterSortKeys)
        for (e.cluster = 1; e.cluster < kMaxSortCluster && (int64_t)e.cluster * kClusterThreads < T;)
            e.cluster *= 2;
    const int64_t per = ((T + kSortMaxTiles - 1) / kSortMaxTiles + kSortBlock - 1) / kSortBlock * kSortBlock;
    e.tile_keys = (uint32_t)per;
    e.tiles = (int)((T + per - 1) / per);
    const int nvec = (int)(H / 8);
    e.slices = (nvec + kSegMaxThreads - 1) / kSegMaxThreads;
    e.threads = ((nvec + e.slices - 1) / e.slices + 31) / 32 * 32;
    // long windows (T = 65536, H = 4096 added: 188 us with 128 positions, 193
    // with 64), shorter ones where that leaves SMs without work (T = 4096,
    // H = 1024 added: 32 us with at least 32 positions, 23 with at least 8)
    e.window = kSegMaxWindow;
    while (e.window > kSegMinWindow && ((T + e.window - 1) / e.window) * e.slices < 152 * 8)
        e.window /= 2;
    e.windows = (int)((T + e.window - 1) / e.window);
    e.present_bytes = 256 + align256(((size_t)V + 31) / 32 * 4); // a flag, then the bitmap
    e.hist_bytes = e.cluster ? 0 : align256((size_t)e.passes * e.tiles * ((size_t)4 << e.bits));
    e.pairs_bytes = align256((size_t)T * 8);
    e.part_bytes = align256((size_t)e.windows * 2 * H * 4);
    e.meta_bytes = align256((size_t)e.windows * 12);
    e.total = e.present_bytes + e.hist_bytes + 2 * e.pairs_bytes + e.part_bytes + e.meta_bytes;
    return e;
}

} // namespace

extern "C" cake_status cake_embedding_fwd(const void *ids, int ids_int64, int64_t tokens, const void *table,
                                          cake_dtype table_dtype, int64_t vocab, int64_t hidden, int64_t table_stride,
                                          float scale, const cake_tensor *y, cake_stream_t stream)
{
    cake_status st = check_embedding(ids, ids_int64, tokens, table, table_dtype, vocab, hidden, table_stride, scale, y,
                                     true);
    if (st != CAKE_OK || tokens == 0)
        return st;
    EmbedFwdParams p{};
    if (step_status_ptr(&p.status) != cudaSuccess)
        return CAKE_ERR_CUDA;
    p.ids = ids;
    p.ids_i64 = ids_int64;
    p.tokens = (uint32_t)tokens;
    p.nvec = (int)(hidden / 8);
    p.table = table;
    p.table_f32 = table_dtype == CAKE_FP32;
    p.vocab = vocab;
    p.table_stride = table_stride;
    p.scale = scale;
    p.y = static_cast<uint16_t *>(y->data);
    p.y_stride = y->stride_token;
    return cuda_status(launch_embed_fwd(p, cu(stream)));
}

extern "C" size_t cake_embedding_bwd_workspace_size(int64_t tokens, int64_t vocab, int64_t hidden)
{
    if (tokens <= 0 || vocab < 1 || hidden < 1 || tokens >= (int64_t(1) << 31) || vocab >= (int64_t(1) << 31) ||
        hidden > CAKE_MAX_HIDDEN)
        return 0;
    return embed_plan(tokens, vocab, hidden).total;
}

extern "C" cake_status cake_embedding_bwd(const cake_tensor *dy, const void *ids, int ids_int64, int64_t tokens,
                                          int64_t vocab, int64_t hidden, float scale, int64_t padding_idx,
                                          void *dtable, cake_dtype dtable_dtype, int64_t dtable_stride, int accumulate,
                                          void *workspace, size_t workspace_bytes, cake_stream_t stream)
{
    cake_status st = check_embedding(ids, ids_int64, tokens, dtable, dtable_dtype, vocab, hidden, dtable_stride, scale,
                                     dy, false);
    if (st != CAKE_OK)
        return st;
    if (padding_idx < -1 || padding_idx >= vocab || (vocab > 1 && dtable_stride < hidden))
        return CAKE_ERR_INVALID;
    cudaStream_t s = cu(stream);
    const size_t size = dtable_dtype == CAKE_FP32 ? 4 : 2;
    if (tokens == 0) {
        if (accumulate)
            return CAKE_OK;
        return cuda_status(cudaMemset2DAsync(dtable, (size_t)std::max(dtable_stride, hidden) * size, 0,
                                             (size_t)hidden * size, (size_t)vocab, s));
    }
    const EmbedPlan e = embed_plan(tokens, vocab, hidden);
    if ((st = check_workspace(workspace, workspace_bytes, e.total)) != CAKE_OK)
        return st;
    const cake_shape shape{tokens, 1, hidden};
    const Memory scratch = memory(workspace, e.total);
    const Memory others[3] = {memory(dy, &shape), memory(ids, (uint64_t)tokens * (ids_int64 ? 8 : 4)),
                              table_memory(dtable, dtable_dtype, vocab, hidden, dtable_stride)};
    if (any_meet(&scratch, 1, others, 3))
        return CAKE_ERR_INVALID;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    SortParams q{};
    if (step_status_ptr(&q.status) != cudaSuccess)
        return CAKE_ERR_CUDA;
    q.ids = ids;
    q.ids_i64 = ids_int64;
    q.tokens = (uint32_t)tokens;
    q.vocab = (uint32_t)vocab;
    q.padding_idx = padding_idx;
    q.tile_keys = e.tile_keys;
    q.tiles = e.tiles;
    q.passes = e.passes;
    q.bits = e.bits;
    q.ready = reinterpret_cast<uint32_t *>(ws);
    q.present = q.ready + 64;
    q.hist = reinterpret_cast<uint32_t *>(ws + e.present_bytes);
    uint8_t *at = ws + e.present_bytes + e.hist_bytes;
    q.pairs[0] = reinterpret_cast<uint64_t *>(at);
    q.pairs[1] = reinterpret_cast<uint64_t *>(at + e.pairs_bytes);
    // a small bitmap is zeroed by the sort itself
    q.zero_present = e.cluster && (accumulate || e.present_bytes <= (size_t)32768 * e.cluster);
    if (accumulate)
        q.present = nullptr; // no row is to be zeroed
    uint64_t *sorted = q.pairs[0];
    cudaError_t r = q.zero_present ? cudaSuccess : cudaMemsetAsync(ws, 0, e.present_bytes + e.hist_bytes, s);
    if (r == cudaSuccess && t_waits.withhold)
        r = cudaMemsetAsync(q.ready + 2, 0, 4, s);
    if (r == cudaSuccess)
        r = e.cluster ? launch_embed_cluster_sort(q, e.cluster, s) : launch_embed_sort(q, &sorted, s);
    if (r != cudaSuccess)
        return CAKE_ERR_CUDA;
    SegmentParams g{};
    g.pairs = sorted;
    g.tokens = q.tokens;
    g.vocab = q.vocab;
    g.window = e.window;
    g.windows = e.windows;
    g.slices = e.slices;
    g.threads = e.threads;
    g.nvec = (int)(hidden / 8);
    g.dy = static_cast<const uint16_t *>(dy->data);
    g.dy_stride = dy->stride_token;
    g.scale = scale;
    g.dtable = dtable;
    g.dtable_f32 = dtable_dtype == CAKE_FP32;
    g.dtable_stride = dtable_stride;
    g.accumulate = accumulate != 0;
    g.present = q.present;
    g.fill_rows = 1;
    while (g.fill_rows < 32 && g.fill_rows * 2 * hidden * (int64_t)size <= 8192)
        g.fill_rows *= 2;
    const int64_t fill = g.fill_rows * (e.threads / 32);
    g.fill_ctas = accumulate ? 0 : (int)std::min<int64_t>((vocab + fill - 1) / fill, 1 << 20);
    g.ready = e.cluster && !accumulate ? q.ready + (t_waits.withhold == 1 ? 2 : 0) : nullptr;
    g.wait_ns = t_waits.ns;
    g.status = q.status;
    g.partials = reinterpret_cast<float *>(at + 2 * e.pairs_bytes);
    g.meta = reinterpret_cast<uint32_t *>(at + 2 * e.pairs_bytes + e.part_bytes);
    g.cut = g.meta + 2 * (size_t)e.windows;
    g.cuts = q.ready + 1;
    r = launch_embed_segments(g, s);
    if (r == cudaSuccess)
        r = launch_embed_join(g, s);
    return cuda_status(r);
}
