// cake_call.h -- validation of a call's workspaces, weights and shared memory,
// for the operators around the norm and between the norms.  Host code only.
#pragma once

#include "cake_check.h"

namespace cake {

inline size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

inline cudaStream_t cu(cake_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

inline bool good_dtype(int d) { return d == CAKE_BF16 || d == CAKE_FP32; }

inline cake_status check_workspace(const void *ws, size_t bytes, size_t need)
{
    if (need > 0 && (!ws || bytes < need))
        return CAKE_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
        return CAKE_ERR_UNSUPPORTED;
    return CAKE_OK;
}

inline bool has(const cake_tensor *t) { return t && t->data; }

inline cake_status check_rows_f32(const void *p)
{
    if (!p)
        return CAKE_ERR_INVALID;
    return (reinterpret_cast<uintptr_t>(p) & 3u) ? CAKE_ERR_UNSUPPORTED : CAKE_OK;
}

// Memory of a call's tensors: what it writes shares none with anything else.
// Equally spaced rows: `row` bytes every `step` bytes; step 0: all of [lo, hi).
struct Memory {
    uintptr_t lo, hi, step, row;
};

inline Memory memory(const void *p, uint64_t bytes)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, p ? lo + (uintptr_t)bytes : lo, 0, 0};
}

inline Memory memory(const cake_tensor *t, const cake_shape *s)
{
    if (!has(t))
        return {0, 0, 0, 0};
    const auto e = extent(t, s);
    const RowView v = make_view(t, s);
    return {e.first, e.second, v.uniform ? (uintptr_t)(2 * v.row_stride) : 0, (uintptr_t)(2 * s->hidden)};
}

// (Rows of unlike spacing count as the whole of what they span.)
inline bool meet(const Memory &a, const Memory &b)
{
    if (!(a.lo < b.hi && b.lo < a.hi && a.lo < a.hi && b.lo < b.hi))
        return false;
    if (a.step == 0 || a.step != b.step)
        return true;
    // columns of one buffer: where b's rows lie after a's, within a row of the buffer
    const uintptr_t off = b.lo >= a.lo ? (b.lo - a.lo) % a.step : (a.step - (a.lo - b.lo) % a.step) % a.step;
    return off < a.row || off + b.row > a.step;
}

// Whether one of the `nw` written ranges meets another one or a range that is read.
inline bool any_meet(const Memory *written, int nw, const Memory *read, int nr)
{
    for (int i = 0; i < nw; ++i) {
        for (int k = 0; k < i; ++k)
            if (meet(written[i], written[k]))
                return true;
        for (int k = 0; k < nr; ++k)
            if (meet(written[i], read[k]))
                return true;
    }
    return false;
}

} // namespace cake
