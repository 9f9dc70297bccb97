// cake_check.h -- validation of the C ABI's shapes and tensors, shared by the
// entry points of the library.  Host code only.
#pragma once

#include <cstdint>
#include <utility>

#include <cuda_runtime.h>

#include "../../include/cake_rmsnorm.h"
#include "../csrc/cake_params.h"

namespace cake {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline cake_status check_shape(const cake_shape *s, uint32_t *rows)
{
    if (!s || s->tokens < 0 || s->heads < 1 || s->hidden < 1)
        return CAKE_ERR_INVALID;
    if (s->hidden % 8 != 0 || s->hidden > CAKE_MAX_HIDDEN)
        return CAKE_ERR_UNSUPPORTED;
    const int64_t r = s->tokens * s->heads;
    if (s->tokens > 0 && r / s->tokens != s->heads)
        return CAKE_ERR_UNSUPPORTED;
    if (r >= (int64_t(1) << 31))
        return CAKE_ERR_UNSUPPORTED;
    *rows = (uint32_t)r;
    return CAKE_OK;
}

// Activation tensor: non-null, 16-byte aligned base, strides multiples of 8
// elements (16 bytes) and non-negative.
inline cake_status check_tensor(const cake_tensor *t, const cake_shape *s)
{
    if (!t || !t->data)
        return CAKE_ERR_INVALID;
    if (t->stride_token < 0 || t->stride_head < 0)
        return CAKE_ERR_UNSUPPORTED;
    if (!aligned16(t->data) || t->stride_token % 8 != 0 ||
        (s->heads > 1 && t->stride_head % 8 != 0))
        return CAKE_ERR_UNSUPPORTED;
    if (s->tokens > 1 && t->stride_token < (s->heads > 1 ? 0 : s->hidden))
        return CAKE_ERR_UNSUPPORTED;
    if (s->heads > 1 && t->stride_head < s->hidden)
        return CAKE_ERR_UNSUPPORTED;
    return CAKE_OK;
}

// An output tensor: as check_tensor, and no two of its rows overlap (a
// kernel writes every row once, so rows that share memory would race).  The
// dimensions with more than one index, in ascending stride order, must each
// step past everything the smaller ones span.
inline cake_status check_out_tensor(const cake_tensor *t, const cake_shape *s)
{
    cake_status st = check_tensor(t, s);
    if (st != CAKE_OK)
        return st;
    int64_t dims[2][2] = {{s->tokens, t->stride_token}, {s->heads, t->stride_head}};
    if (dims[0][1] > dims[1][1]) {
        std::swap(dims[0][0], dims[1][0]);
        std::swap(dims[0][1], dims[1][1]);
    }
    int64_t span = s->hidden; // elements one index of the dimensions seen so far covers
    for (auto &d : dims) {
        if (d[0] <= 1)
            continue;
        if (d[1] < span)
            return CAKE_ERR_INVALID;
        span = (d[0] - 1) * d[1] + span;
    }
    return CAKE_OK;
}

// Byte range [lo, hi) a view's rows touch (strides are non-negative).
inline std::pair<uintptr_t, uintptr_t> extent(const cake_tensor *t, const cake_shape *s)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(t->data);
    const int64_t last = (s->tokens - 1) * t->stride_token + (s->heads > 1 ? (s->heads - 1) * t->stride_head : 0);
    return {lo, lo + (uintptr_t)(2 * (last + s->hidden))};
}

inline bool overlap(const cake_tensor *a, const cake_tensor *b, const cake_shape *s)
{
    if (!a || !a->data || !b || !b->data)
        return false;
    const auto ea = extent(a, s), eb = extent(b, s);
    return ea.first < eb.second && eb.first < ea.second;
}

inline bool same_view(const cake_tensor *a, const cake_tensor *b, const cake_shape *s)
{
    return a->data == b->data && (s->tokens <= 1 || a->stride_token == b->stride_token) &&
           (s->heads <= 1 || a->stride_head == b->stride_head);
}

inline RowView make_view(const cake_tensor *t, const cake_shape *s)
{
    RowView v{};
    if (!t || !t->data)
        return v;
    v.base = static_cast<const uint16_t *>(t->data);
    v.st = t->stride_token;
    v.sh = s->heads > 1 ? t->stride_head : 0;
    if (s->heads == 1) {
        v.uniform = 1;
        v.row_stride = t->stride_token;
    } else if (t->stride_token == s->heads * t->stride_head) {
        v.uniform = 1;
        v.row_stride = t->stride_head;
    } else if (s->tokens == 1) {
        v.uniform = 1;
        v.row_stride = t->stride_head;
    }
    v.dense = v.uniform && v.row_stride == s->hidden;
    return v;
}

inline cake_status cuda_status(cudaError_t e)
{
    return e == cudaSuccess ? CAKE_OK : CAKE_ERR_CUDA;
}

} // namespace cake
