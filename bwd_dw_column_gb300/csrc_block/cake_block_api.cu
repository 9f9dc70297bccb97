// cake_block_api.cu -- the C ABI of a block's operators between the norms:
// argument validation, workspace layout and dispatch to the launchers.  Host
// code only.
#include <algorithm>
#include <cmath>

#include <cuda_runtime.h>

#include "../../include/cake_block_test.h"
#include "../csrc_step/cake_call.h"
#include "cake_block_launch.h"

using namespace cake;

namespace {

// The limit of the kernels' waits, and whether a part of the first copy is withheld (cake_block_wait_test).
struct Waits {
    uint64_t ns = kWaitLimitNs;
    int withhold = 0;
};
thread_local Waits t_waits;

// ------------------------------------------------------------------ dropout

cake_status check_p(double p, const uint64_t *rng)
{
    if (!(p >= 0.0 && p <= 1.0))
        return CAKE_ERR_INVALID;
    return (reinterpret_cast<uintptr_t>(rng) & 7u) ? CAKE_ERR_UNSUPPORTED : CAKE_OK;
}

DropoutRng dropout_rng(double p, uint64_t seed, uint64_t offset, const uint64_t *rng)
{
    const uint32_t cut = (uint32_t)std::nearbyint(p * 65536.0);
    DropoutRng r{seed, offset, rng, cut, cut < 65536 ? (float)(65536.0 / (65536 - (int)cut)) : 0.0f, {}};
    for (uint32_t i = 0; i < 10; ++i) {
        r.keys[2 * i] = (uint32_t)seed + i * 0x9E3779B9u;
        r.keys[2 * i + 1] = (uint32_t)(seed >> 32) + i * 0xBB67AE85u;
    }
    return r;
}

Layout rows_layout(const DropoutNormPlan &plan, const cake_shape *shape, uint32_t rows, int ntens)
{
    Layout L{};
    L.H = (int)shape->hidden;
    L.nvec = L.H / 8;
    L.warps_per_row = plan.W;
    L.groups = plan.groups;
    L.rows_per_group = 32 / plan.lanes;
    L.lanes_per_row = plan.lanes;
    L.stages = plan.stages;
    L.lo_bytes = plan.lo_bytes;
    L.ntens = ntens;
    L.rows = rows;
    L.nh = (uint32_t)shape->heads;
    L.rows_per_cta = plan.rows_per_cta;
    L.inv_h = 1.0f / (float)L.H;
    return L;
}

cake_status check_weight(const void *w, int dtype)
{
    if (!good_dtype(dtype) || !w)
        return CAKE_ERR_INVALID;
    return aligned16(w) ? CAKE_OK : CAKE_ERR_UNSUPPORTED;
}

uint64_t weight_bytes(int64_t n, int dtype) { return (uint64_t)n * (dtype == CAKE_FP32 ? 4 : 2); }

} // namespace

extern "C" cake_status cake_block_wait_test(uint32_t wait_limit_us, int withhold)
{
    if (wait_limit_us > 1000000 || withhold < 0 || withhold > 1 || (wait_limit_us == 0 && withhold))
        return CAKE_ERR_INVALID;
    t_waits.ns = wait_limit_us ? (uint64_t)wait_limit_us * 1000u : kWaitLimitNs;
    t_waits.withhold = withhold;
    return CAKE_OK;
}

extern "C" cake_status cake_dropout_norm_plan(const cake_shape *shape, int tensors, int backward, int64_t plan[9])
{
    uint32_t rows = 0;
    const cake_status st = check_shape(shape, &rows);
    if (st != CAKE_OK)
        return st;
    if (!plan || rows == 0 || tensors < 2 || tensors > 3)
        return CAKE_ERR_INVALID;
    const DropoutNormPlan p = dropout_norm_plan((int)shape->hidden, rows, tensors, backward != 0);
    const int64_t got[9] = {p.vpt,  p.lanes,        p.W,        p.groups,       p.stages,
                            p.ctas, p.rows_per_cta, p.lo_bytes, (int64_t)p.smem};
    std::copy(got, got + 9, plan);
    return CAKE_OK;
}

extern "C" cake_status cake_dropout(const cake_shape *shape, const cake_tensor *x, const cake_tensor *residual, double p,
                                    uint64_t seed, uint64_t offset, const uint64_t *rng, const cake_tensor *y,
                                    cake_stream_t stream)
{
    uint32_t rows = 0;
    cake_status st = check_shape(shape, &rows);
    if (st != CAKE_OK || (st = check_p(p, rng)) != CAKE_OK || rows == 0)
        return st;
    if ((st = check_tensor(x, shape)) != CAKE_OK || (has(residual) && (st = check_tensor(residual, shape)) != CAKE_OK) ||
        (st = check_out_tensor(y, shape)) != CAKE_OK)
        return st;
    for (const cake_tensor *i : {x, residual})
        if (has(i) && meet(memory(y, shape), memory(i, shape)) && !same_view(y, i, shape))
            return CAKE_ERR_INVALID;
    if (meet(memory(y, shape), memory(rng, 16)))
        return CAKE_ERR_INVALID;
    DropoutParams q{};
    q.r = dropout_rng(p, seed, offset, rng);
    q.x = make_view(x, shape);
    q.residual = make_view(residual, shape);
    q.y = make_view(y, shape);
    q.nh = (uint32_t)shape->heads;
    q.nvec = (uint32_t)(shape->hidden / 8);
    q.reciprocal = (uint32_t)(((uint64_t(1) << 31) + q.nvec - 1) / q.nvec);
    q.vecs = (uint64_t)rows * q.nvec;
    return cuda_status(launch_dropout(q, cu(stream)));
}

extern "C" cake_status cake_dropout_norm_fwd(const cake_shape *shape, const cake_tensor *x, const cake_tensor *residual,
                                             const void *w, cake_dtype w_dtype, double p, uint64_t seed,
                                             uint64_t offset, const uint64_t *rng, float eps, const cake_tensor *y,
                                             const cake_tensor *h_new, float *rstd, cake_stream_t stream)
{
    uint32_t rows = 0;
    cake_status st = check_shape(shape, &rows);
    if (st != CAKE_OK || (st = check_p(p, rng)) != CAKE_OK)
        return st;
    if (!(eps >= 0.0f) || !good_dtype(w_dtype))
        return CAKE_ERR_INVALID;
    if (rows == 0)
        return CAKE_OK;
    if ((st = check_weight(w, w_dtype)) != CAKE_OK || (st = check_tensor(x, shape)) != CAKE_OK ||
        (st = check_tensor(residual, shape)) != CAKE_OK || (st = check_out_tensor(y, shape)) != CAKE_OK ||
        (st = check_out_tensor(h_new, shape)) != CAKE_OK || (st = check_rows_f32(rstd)) != CAKE_OK)
        return st;
    // a row is written after it is read: y and h_new may be an input's view exactly
    const Memory written[3] = {memory(rstd, (uint64_t)rows * 4), memory(y, shape), memory(h_new, shape)};
    const Memory lists[2] = {memory(w, weight_bytes(shape->hidden, w_dtype)), memory(rng, 16)};
    const Memory ins[2] = {memory(x, shape), memory(residual, shape)};
    if (any_meet(written, 3, lists, 2) || any_meet(written, 1, ins, 2))
        return CAKE_ERR_INVALID;
    for (const cake_tensor *o : {y, h_new})
        for (const cake_tensor *i : {x, residual})
            if (meet(memory(o, shape), memory(i, shape)) && !same_view(o, i, shape))
                return CAKE_ERR_INVALID;
    DropoutNormParams q{};
    const DropoutNormPlan plan = dropout_norm_plan((int)shape->hidden, rows, 2, false);
    q.L = rows_layout(plan, shape, rows, 2);
    q.r = dropout_rng(p, seed, offset, rng);
    q.in[0] = make_view(x, shape);
    q.in[1] = make_view(residual, shape);
    q.out[0] = make_view(y, shape);
    q.out[1] = make_view(h_new, shape);
    q.w = w;
    q.w_f32 = w_dtype == CAKE_FP32;
    q.eps = eps;
    q.rstd_out = rstd;
    q.wait_ns = t_waits.ns;
    q.withhold = t_waits.withhold;
    if (step_status_ptr(&q.status) != cudaSuccess)
        return CAKE_ERR_CUDA;
    return cuda_status(launch_dropout_norm_fwd(q, plan, cu(stream)));
}

extern "C" size_t cake_dropout_norm_bwd_workspace_size(const cake_shape *shape)
{
    uint32_t rows = 0;
    if (check_shape(shape, &rows) != CAKE_OK || rows == 0)
        return 0;
    return (size_t)(rows < (uint32_t)kSMsBlock ? rows : kSMsBlock) * shape->hidden * sizeof(float2); // a CTA an SM
}

extern "C" cake_status cake_dropout_norm_bwd(const cake_shape *shape, const cake_tensor *dy, const cake_tensor *dh,
                                             const cake_tensor *h_new, const float *rstd, const void *w,
                                             cake_dtype w_dtype, double p, uint64_t seed, uint64_t offset,
                                             const uint64_t *rng, const cake_tensor *dx, const cake_tensor *dresidual,
                                             float *dw, void *workspace, size_t workspace_bytes, cake_stream_t stream)
{
    uint32_t rows = 0;
    cake_status st = check_shape(shape, &rows);
    if (st != CAKE_OK || (st = check_p(p, rng)) != CAKE_OK)
        return st;
    if (!good_dtype(w_dtype) || !dw)
        return CAKE_ERR_INVALID;
    if (!aligned16(dw))
        return CAKE_ERR_UNSUPPORTED;
    if (rows == 0)
        return cuda_status(cudaMemsetAsync(dw, 0, (size_t)shape->hidden * sizeof(float), cu(stream)));
    if ((st = check_weight(w, w_dtype)) != CAKE_OK || (st = check_tensor(dy, shape)) != CAKE_OK ||
        (has(dh) && (st = check_tensor(dh, shape)) != CAKE_OK) || (st = check_tensor(h_new, shape)) != CAKE_OK ||
        (st = check_rows_f32(rstd)) != CAKE_OK || (st = check_out_tensor(dx, shape)) != CAKE_OK ||
        (st = check_out_tensor(dresidual, shape)) != CAKE_OK)
        return st;
    const size_t need = cake_dropout_norm_bwd_workspace_size(shape);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != CAKE_OK)
        return st;
    const Memory written[4] = {memory(dx, shape), memory(dresidual, shape), memory(dw, (uint64_t)shape->hidden * 4),
                               memory(workspace, need)};
    const Memory read[6] = {memory(dy, shape),  memory(dh, shape), memory(h_new, shape), memory(rstd, (uint64_t)rows * 4),
                            memory(rng, 16), memory(w, weight_bytes(shape->hidden, w_dtype))};
    if (any_meet(written, 4, read, 6))
        return CAKE_ERR_INVALID;
    DropoutNormParams q{};
    const int ntens = has(dh) ? 3 : 2;
    const DropoutNormPlan plan = dropout_norm_plan((int)shape->hidden, rows, ntens, true);
    q.L = rows_layout(plan, shape, rows, ntens);
    q.r = dropout_rng(p, seed, offset, rng);
    q.in[0] = make_view(h_new, shape);
    q.in[1] = make_view(dy, shape);
    q.in[2] = make_view(dh, shape);
    q.out[0] = make_view(dx, shape);
    q.out[1] = make_view(dresidual, shape);
    q.w = w;
    q.w_f32 = w_dtype == CAKE_FP32;
    q.rstd = rstd;
    q.partials = static_cast<float2 *>(workspace);
    q.wait_ns = t_waits.ns;
    q.withhold = t_waits.withhold;
    if (step_status_ptr(&q.status) != cudaSuccess || launch_dropout_norm_bwd(q, plan, cu(stream)) != cudaSuccess)
        return CAKE_ERR_CUDA;
    ColumnSumParams s{};
    s.partials[0] = q.partials;
    s.out[0] = dw;
    s.P[0] = plan.ctas;
    s.H = (int)shape->hidden;
    return cuda_status(launch_column_sum(s, 1, cu(stream)));
}

// ------------------------------------------------------------------- rotary

namespace {

// Heads of a call's tokens: two views may be columns of one buffer, also where
// their heads are not equally spaced over it (queries and keys of one product).
bool heads_meet(const cake_tensor *a, const cake_shape &sa, const cake_tensor *b, const cake_shape &sb)
{
    const Memory x = memory(a, &sa), y = memory(b, &sb);
    if (!meet(x, y))
        return false;
    const auto by_token = [](const cake_tensor *t, const cake_shape &s) {
        Memory m = memory(t, &s);
        const int64_t span = (s.heads - 1) * t->stride_head + s.hidden; // of a token's heads
        m.step = s.heads == 1 || t->stride_head >= 0 ? (uintptr_t)(2 * t->stride_token) : 0;
        m.row = (uintptr_t)(2 * span);
        if (s.tokens > 1 && t->stride_token < span)
            m.step = 0;
        return m;
    };
    return meet(by_token(a, sa), by_token(b, sb));
}

struct RotaryCall {
    cake_shape shape[2]; // queries, keys
    uint32_t rows[2];
    int lists;
};

cake_status check_rotary(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t hidden, const cake_rotary *r,
                         RotaryCall &c)
{
    if (k_heads < 0 || !r)
        return CAKE_ERR_INVALID;
    c.shape[0] = {tokens, q_heads, hidden};
    c.shape[1] = {tokens, k_heads, hidden};
    c.lists = k_heads > 0 ? 2 : 1;
    for (int i = 0; i < c.lists; ++i) {
        const cake_status st = check_shape(&c.shape[i], &c.rows[i]);
        if (st != CAKE_OK)
            return st;
    }
    if (r->pairs < 0 || r->axes < 1 || r->style < CAKE_ROTARY_HALF || r->style > CAKE_ROTARY_ADJACENT ||
        r->axis_stride < 0 || r->token_stride < 0 || (r->positions_int64 != 0 && r->positions_int64 != 1))
        return CAKE_ERR_INVALID;
    if (hidden % 16 != 0 || hidden > 512 || r->pairs % 8 != 0 || 2 * r->pairs > hidden || r->axes > 16)
        return CAKE_ERR_UNSUPPORTED;
    if (tokens == 0 || r->pairs == 0)
        return CAKE_OK;
    if (!r->turns || !r->positions || (r->axes > 1 && !r->axis))
        return CAKE_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(r->turns) & 7u) || (reinterpret_cast<uintptr_t>(r->axis) & 3u) ||
        (reinterpret_cast<uintptr_t>(r->positions) & (r->positions_int64 ? 7u : 3u)))
        return CAKE_ERR_UNSUPPORTED;
    return CAKE_OK;
}

// The rotation's own tensors.
void rotary_memory(const cake_rotary *r, int64_t tokens, Memory (&m)[3])
{
    m[0] = m[1] = m[2] = {0, 0, 0, 0};
    if (tokens == 0 || r->pairs == 0)
        return;
    m[0] = memory(r->turns, (uint64_t)r->pairs * 8);
    m[1] = memory(r->axis, (uint64_t)r->pairs * 4);
    m[2] = memory(r->positions, (uint64_t)((r->axes - 1) * r->axis_stride + (tokens - 1) * r->token_stride + 1) *
                                    (r->positions_int64 ? 8 : 4));
}

void fill_rotary(RotaryParams &p, const cake_rotary *r, int64_t tokens, int64_t hidden)
{
    p.tokens = (uint32_t)tokens;
    p.D = (int)hidden;
    p.inv_d = 1.0f / (float)hidden;
    p.axes = 1;
    p.pairs = (int)r->pairs;
    if (r->pairs > 0) { // (without pairs none of these is looked at)
        p.axes = (int)r->axes;
        p.turns = r->turns;
        p.axis = r->axis;
        p.positions = r->positions;
    }
    p.pos_i64 = r->positions_int64;
    p.axis_stride = r->axis_stride;
    p.token_stride = r->token_stride;
}

// A list's output: in place exactly over `in`, or apart from everything in `rest`.
cake_status check_rotary_out(const RotaryCall &c, int i, const cake_tensor *out, const cake_tensor *const in[2],
                             const cake_tensor *const other[2], const cake_tensor *const outs[2])
{
    const cake_status st = check_out_tensor(out, &c.shape[i]);
    if (st != CAKE_OK)
        return st;
    for (int k = 0; k < c.lists; ++k) {
        if (heads_meet(out, c.shape[i], in[k], c.shape[k]) && !(i == k && same_view(out, in[k], &c.shape[i])))
            return CAKE_ERR_INVALID;
        if (other && heads_meet(out, c.shape[i], other[k], c.shape[k]))
            return CAKE_ERR_INVALID;
        if (k < i && heads_meet(out, c.shape[i], outs[k], c.shape[k]))
            return CAKE_ERR_INVALID;
    }
    return CAKE_OK;
}

} // namespace

extern "C" cake_status cake_rotary_fwd(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t hidden,
                                       const cake_tensor *q, const cake_tensor *k, const cake_rotary *rotary,
                                       const void *w_q, cake_dtype w_q_dtype, const void *w_k, cake_dtype w_k_dtype,
                                       float eps, const cake_tensor *q_out, const cake_tensor *k_out, float *rstd_q,
                                       float *rstd_k, cake_stream_t stream)
{
    RotaryCall c{};
    cake_status st = check_rotary(tokens, q_heads, k_heads, hidden, rotary, c);
    if (st != CAKE_OK)
        return st;
    const bool norm = w_q != nullptr;
    if ((c.lists == 2 && norm != (w_k != nullptr)) || (norm && !(eps >= 0.0f)))
        return CAKE_ERR_INVALID;
    const cake_tensor *const in[2] = {q, k}, *const out[2] = {q_out, k_out};
    const void *const w[2] = {w_q, w_k};
    const int dtype[2] = {w_q_dtype, w_k_dtype};
    float *const rstd[2] = {rstd_q, rstd_k};
    for (int i = 0; i < c.lists && norm; ++i)
        if (!good_dtype(dtype[i]))
            return CAKE_ERR_INVALID;
    if (tokens == 0)
        return CAKE_OK;
    for (int i = 0; i < c.lists; ++i)
        if ((st = check_tensor(in[i], &c.shape[i])) != CAKE_OK ||
            (norm && ((st = check_weight(w[i], dtype[i])) != CAKE_OK || (st = check_rows_f32(rstd[i])) != CAKE_OK)))
            return st;
    Memory lists[5], scalars[2] = {}, views[4] = {};
    rotary_memory(rotary, tokens, reinterpret_cast<Memory(&)[3]>(lists));
    for (int i = 0; i < 2; ++i)
        lists[3 + i] = i < c.lists && norm ? memory(w[i], weight_bytes(hidden, dtype[i])) : Memory{0, 0, 0, 0};
    for (int i = 0; i < c.lists; ++i)
        if ((st = check_rotary_out(c, i, out[i], in, nullptr, out)) != CAKE_OK)
            return st;
    for (int i = 0; i < c.lists; ++i) {
        const Memory o = memory(out[i], &c.shape[i]);
        if (any_meet(&o, 1, lists, 5))
            return CAKE_ERR_INVALID;
        views[2 * i] = o;
        views[2 * i + 1] = memory(in[i], &c.shape[i]);
        if (norm)
            scalars[i] = memory(rstd[i], (uint64_t)c.rows[i] * 4);
    }
    if (any_meet(scalars, 2, lists, 5) || any_meet(scalars, 2, views, 4))
        return CAKE_ERR_INVALID;
    RotaryParams p{};
    if (step_status_ptr(&p.status) != cudaSuccess)
        return CAKE_ERR_CUDA;
    fill_rotary(p, rotary, tokens, hidden);
    p.eps = eps;
    for (int i = 0; i < c.lists; ++i) {
        RotaryList &l = p.l[i];
        l.in = make_view(in[i], &c.shape[i]);
        l.out = make_view(out[i], &c.shape[i]);
        l.heads = (uint32_t)c.shape[i].heads;
        l.w = norm ? w[i] : nullptr;
        l.w_f32 = dtype[i] == CAKE_FP32;
        l.rstd_out = rstd[i];
    }
    rotary_plan(p);
    return cuda_status(launch_rotary(p, rotary->style == CAKE_ROTARY_ADJACENT, false, cu(stream)));
}

extern "C" size_t cake_rotary_bwd_workspace_size(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t hidden)
{
    cake_rotary none{};
    none.axes = 1;
    RotaryCall c{};
    if (check_rotary(tokens, q_heads, k_heads, hidden, &none, c) != CAKE_OK || tokens == 0)
        return 0;
    RotaryParams p{};
    fill_rotary(p, &none, tokens, hidden);
    for (int i = 0; i < c.lists; ++i)
        p.l[i].heads = (uint32_t)c.shape[i].heads;
    rotary_plan(p);
    return (size_t)(p.l[0].ctas + p.l[1].ctas) * hidden * sizeof(float2);
}

extern "C" cake_status cake_rotary_bwd(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t hidden,
                                       const cake_tensor *dq, const cake_tensor *dk, const cake_rotary *rotary,
                                       const cake_tensor *q, const cake_tensor *k, const float *rstd_q,
                                       const float *rstd_k, const void *w_q, cake_dtype w_q_dtype, const void *w_k,
                                       cake_dtype w_k_dtype, const cake_tensor *dq_out, const cake_tensor *dk_out,
                                       float *dw_q, float *dw_k, void *workspace, size_t workspace_bytes,
                                       cake_stream_t stream)
{
    RotaryCall c{};
    cake_status st = check_rotary(tokens, q_heads, k_heads, hidden, rotary, c);
    if (st != CAKE_OK)
        return st;
    const bool norm = w_q != nullptr;
    if (c.lists == 2 && norm != (w_k != nullptr))
        return CAKE_ERR_INVALID;
    const cake_tensor *const in[2] = {dq, dk}, *const out[2] = {dq_out, dk_out}, *const v[2] = {q, k};
    const void *const w[2] = {w_q, w_k};
    const int dtype[2] = {w_q_dtype, w_k_dtype};
    const float *const rstd[2] = {rstd_q, rstd_k};
    float *const dw[2] = {dw_q, dw_k};
    for (int i = 0; i < c.lists && norm; ++i)
        if (!good_dtype(dtype[i]) || !dw[i])
            return CAKE_ERR_INVALID;
    for (int i = 0; i < 2 && norm; ++i)
        if (!aligned16(dw[i]))
            return CAKE_ERR_UNSUPPORTED;
    // a sum over nothing: without tokens, and that of keys without heads
    const auto zero = [&](float *to) {
        return !norm || !to || cudaMemsetAsync(to, 0, (size_t)hidden * sizeof(float), cu(stream)) == cudaSuccess;
    };
    if (tokens == 0)
        return zero(dw_q) && zero(dw_k) ? CAKE_OK : CAKE_ERR_CUDA;
    for (int i = 0; i < c.lists; ++i)
        if ((st = check_tensor(in[i], &c.shape[i])) != CAKE_OK ||
            (norm && ((st = check_weight(w[i], dtype[i])) != CAKE_OK || (st = check_rows_f32(rstd[i])) != CAKE_OK ||
                      (st = check_tensor(v[i], &c.shape[i])) != CAKE_OK)))
            return st;
    const size_t need = norm ? cake_rotary_bwd_workspace_size(tokens, q_heads, k_heads, hidden) : 0;
    if ((st = check_workspace(workspace, workspace_bytes, need)) != CAKE_OK)
        return st;
    for (int i = 0; i < c.lists; ++i)
        if ((st = check_rotary_out(c, i, out[i], in, norm ? v : nullptr, out)) != CAKE_OK)
            return st;
    Memory lists[13] = {}, scalars[3] = {};
    rotary_memory(rotary, tokens, reinterpret_cast<Memory(&)[3]>(lists));
    for (int i = 0; i < c.lists && norm; ++i) {
        lists[3 + i] = memory(w[i], weight_bytes(hidden, dtype[i]));
        lists[5 + i] = memory(rstd[i], (uint64_t)c.rows[i] * 4);
        lists[11 + i] = memory(v[i], &c.shape[i]);
    }
    for (int i = 0; i < 2 && norm; ++i)
        scalars[i] = memory(dw[i], (uint64_t)hidden * 4);
    scalars[2] = memory(workspace, need);
    for (int i = 0; i < c.lists; ++i) {
        const Memory o = memory(out[i], &c.shape[i]);
        if (any_meet(&o, 1, lists, 7))
            return CAKE_ERR_INVALID;
        lists[7 + i] = o;
        lists[9 + i] = memory(in[i], &c.shape[i]);
    }
    if (any_meet(scalars, 3, lists, 13))
        return CAKE_ERR_INVALID;
    RotaryParams p{};
    if (step_status_ptr(&p.status) != cudaSuccess || (c.lists == 1 && !zero(dw_k)))
        return CAKE_ERR_CUDA;
    fill_rotary(p, rotary, tokens, hidden);
    for (int i = 0; i < c.lists; ++i) {
        RotaryList &l = p.l[i];
        l.in = make_view(in[i], &c.shape[i]);
        l.out = make_view(out[i], &c.shape[i]);
        l.heads = (uint32_t)c.shape[i].heads;
        if (norm) {
            l.v = make_view(v[i], &c.shape[i]);
            l.w = w[i];
            l.w_f32 = dtype[i] == CAKE_FP32;
            l.rstd = rstd[i];
        }
    }
    const bool adjacent = rotary->style == CAKE_ROTARY_ADJACENT;
    rotary_plan(p);
    if (!norm) // a rotation's gradient is rotated back
        return cuda_status(launch_rotary(p, adjacent, true, cu(stream)));
    p.l[0].partials = static_cast<float2 *>(workspace);
    p.l[1].partials = p.l[0].partials + (size_t)p.l[0].ctas * hidden;
    if (launch_rotary_bwd(p, adjacent, cu(stream)) != cudaSuccess)
        return CAKE_ERR_CUDA;
    ColumnSumParams s{};
    for (int i = 0; i < c.lists; ++i) {
        s.partials[i] = p.l[i].partials;
        s.out[i] = dw[i];
        s.P[i] = p.l[i].ctas;
    }
    s.H = (int)hidden;
    return cuda_status(launch_column_sum(s, c.lists, cu(stream)));
}

// -------------------------------------------------------------------- gated

namespace {

cake_status check_gated(int64_t tokens, int64_t hidden, int64_t ffn, int act)
{
    if (tokens < 0 || hidden < 1 || ffn < 1 || (act != CAKE_ACT_SILU && act != CAKE_ACT_GELU))
        return CAKE_ERR_INVALID;
    if (hidden % 8 != 0 || ffn % 8 != 0 || hidden > CAKE_MAX_BLOCK_WIDTH || ffn > CAKE_MAX_BLOCK_WIDTH ||
        tokens >= (int64_t(1) << 28)) // (the tiles are counted in 32 bits)
        return CAKE_ERR_UNSUPPORTED;
    return CAKE_OK;
}

// A matrix of rows x cols: data 16-byte aligned, rows of at least cols, in steps of 16 bytes.
cake_status check_matrix(const cake_tensor *t, int64_t rows, int64_t cols)
{
    if (!t || !t->data)
        return CAKE_ERR_INVALID;
    if (!aligned16(t->data) || t->stride_token % 8 != 0 || (rows > 1 && t->stride_token < cols) ||
        t->stride_token < 0 || t->stride_token >= (int64_t(1) << 36))
        return CAKE_ERR_UNSUPPORTED;
    return CAKE_OK;
}

Matrix matrix(const cake_tensor *t, int64_t rows, int64_t cols)
{
    if (!has(t))
        return {nullptr, rows, cols, cols};
    return {t->data, rows, cols, rows > 1 ? t->stride_token : cols};
}

Memory matrix_memory(const cake_tensor *t, int64_t rows, int64_t cols)
{
    if (!has(t))
        return {0, 0, 0, 0};
    const cake_shape s{rows, 1, cols};
    const cake_tensor one{t->data, t->stride_token, 0};
    return memory(&one, &s);
}


} // namespace

extern "C" cake_status cake_gated_fwd(int64_t tokens, int64_t hidden, int64_t ffn, const cake_tensor *x,
                                      const cake_tensor *w_gate, const cake_tensor *w_up, cake_act act,
                                      const cake_tensor *h, const cake_tensor *g, const cake_tensor *u,
                                      cake_stream_t stream)
{
    cake_status st = check_gated(tokens, hidden, ffn, act);
    if (st != CAKE_OK)
        return st;
    if (has(g) != has(u))
        return CAKE_ERR_INVALID;
    if (tokens == 0)
        return CAKE_OK;
    if ((st = check_matrix(x, tokens, hidden)) != CAKE_OK || (st = check_matrix(w_gate, ffn, hidden)) != CAKE_OK ||
        (st = check_matrix(w_up, ffn, hidden)) != CAKE_OK || (st = check_matrix(h, tokens, ffn)) != CAKE_OK ||
        (has(g) && ((st = check_matrix(g, tokens, ffn)) != CAKE_OK || (st = check_matrix(u, tokens, ffn)) != CAKE_OK)))
        return st;
    const Memory written[3] = {matrix_memory(h, tokens, ffn), matrix_memory(g, tokens, ffn),
                               matrix_memory(u, tokens, ffn)};
    const Memory read[3] = {matrix_memory(x, tokens, hidden), matrix_memory(w_gate, ffn, hidden),
                            matrix_memory(w_up, ffn, hidden)};
    if (any_meet(written, 3, read, 3))
        return CAKE_ERR_INVALID;
    GatedFwdCall c{};
    c.T = tokens;
    c.H = hidden;
    c.F = ffn;
    c.gelu = act == CAKE_ACT_GELU;
    c.x = matrix(x, tokens, hidden);
    c.w_gate = matrix(w_gate, ffn, hidden);
    c.w_up = matrix(w_up, ffn, hidden);
    c.h = matrix(h, tokens, ffn);
    c.g = matrix(g, tokens, ffn);
    c.u = matrix(u, tokens, ffn);
    c.wait_ns = t_waits.ns;
    c.withhold = t_waits.withhold;
    if (step_status_ptr(&c.status) != cudaSuccess)
        return CAKE_ERR_CUDA;
    return cuda_status(launch_gated_fwd(c, cu(stream)));
}

extern "C" size_t cake_gated_bwd_workspace_size(int64_t tokens, int64_t hidden, int64_t ffn)
{
    if (check_gated(tokens, hidden, ffn, CAKE_ACT_SILU) != CAKE_OK || tokens == 0)
        return 0;
    return gated_bwd_workspace(tokens, hidden, ffn);
}

extern "C" cake_status cake_gated_bwd(int64_t tokens, int64_t hidden, int64_t ffn, const cake_tensor *dh,
                                      const cake_tensor *x, const cake_tensor *g, const cake_tensor *u,
                                      const cake_tensor *w_gate, const cake_tensor *w_up, cake_act act,
                                      const cake_tensor *dx, const cake_tensor *dw_gate, const cake_tensor *dw_up,
                                      void *workspace, size_t workspace_bytes, cake_stream_t stream)
{
    cake_status st = check_gated(tokens, hidden, ffn, act);
    if (st != CAKE_OK)
        return st;
    if (has(dw_gate) != has(dw_up))
        return CAKE_ERR_INVALID;
    if ((has(dw_gate) && ((st = check_matrix(dw_gate, ffn, hidden)) != CAKE_OK ||
                          (st = check_matrix(dw_up, ffn, hidden)) != CAKE_OK)) ||
        (has(dx) && tokens > 0 && (st = check_matrix(dx, tokens, hidden)) != CAKE_OK))
        return st;
    const Memory dwg = matrix_memory(dw_gate, ffn, hidden), dwu = matrix_memory(dw_up, ffn, hidden);
    if (meet(dwg, dwu))
        return CAKE_ERR_INVALID;
    if (tokens == 0) {
        for (const cake_tensor *t : {dw_gate, dw_up})
            if (has(t)) {
                const Matrix m = matrix(t, ffn, hidden);
                if (cudaMemset2DAsync(t->data, (size_t)m.stride * 2, 0, (size_t)hidden * 2, (size_t)ffn, cu(stream)) !=
                    cudaSuccess)
                    return CAKE_ERR_CUDA;
            }
        return CAKE_OK;
    }
    if (!has(dx) && !has(dw_gate))
        return CAKE_OK;
    if ((st = check_matrix(dh, tokens, ffn)) != CAKE_OK || (st = check_matrix(x, tokens, hidden)) != CAKE_OK ||
        (st = check_matrix(g, tokens, ffn)) != CAKE_OK || (st = check_matrix(u, tokens, ffn)) != CAKE_OK ||
        (st = check_matrix(w_gate, ffn, hidden)) != CAKE_OK || (st = check_matrix(w_up, ffn, hidden)) != CAKE_OK)
        return st;
    const size_t need = gated_bwd_workspace(tokens, hidden, ffn);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != CAKE_OK)
        return st;
    const Memory written[4] = {matrix_memory(dx, tokens, hidden), dwg, dwu, memory(workspace, need)};
    const Memory read[6] = {matrix_memory(dh, tokens, ffn), matrix_memory(x, tokens, hidden),
                            matrix_memory(g, tokens, ffn),  matrix_memory(u, tokens, ffn),
                            matrix_memory(w_gate, ffn, hidden), matrix_memory(w_up, ffn, hidden)};
    if (any_meet(written, 4, read, 6))
        return CAKE_ERR_INVALID;
    GatedBwdCall c{};
    c.T = tokens;
    c.H = hidden;
    c.F = ffn;
    c.gelu = act == CAKE_ACT_GELU;
    c.dh = matrix(dh, tokens, ffn);
    c.x = matrix(x, tokens, hidden);
    c.g = matrix(g, tokens, ffn);
    c.u = matrix(u, tokens, ffn);
    c.w_gate = matrix(w_gate, ffn, hidden);
    c.w_up = matrix(w_up, ffn, hidden);
    c.dx = matrix(dx, tokens, hidden);
    c.dw_gate = matrix(dw_gate, ffn, hidden);
    c.dw_up = matrix(dw_up, ffn, hidden);
    c.workspace = static_cast<uint8_t *>(workspace);
    c.wait_ns = t_waits.ns;
    c.withhold = t_waits.withhold;
    if (step_status_ptr(&c.status) != cudaSuccess)
        return CAKE_ERR_CUDA;
    return cuda_status(launch_gated_bwd(c, cu(stream)));
}
