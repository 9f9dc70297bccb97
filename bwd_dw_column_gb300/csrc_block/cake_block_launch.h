// cake_block_launch.h -- launch parameters and private launchers of a block's
// operators between the norms (plain structs, passed by value to the kernels).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../csrc/cake_params.h"

namespace cake {

constexpr int kSMsBlock = 152;

// ------------------------------------------------------------------ dropout

struct DropoutRng {
    uint64_t seed, offset;
    const uint64_t *rng;   // nullptr, or a seed and a number added to offset
    uint32_t cut;          // kept: 16 random bits of at least this
    float scale;           // 65536 / (65536 - cut); 0 where cut is 65536
    uint32_t keys[20];     // of the generator's ten rounds, without rng
};

struct DropoutParams {
    DropoutRng r;
    RowView x, residual, y; // residual.base == nullptr: none
    uint32_t nh, nvec;      // vectors of 8 elements of a row
    uint32_t reciprocal;    // 2^31 / nvec, rounded up
    uint64_t vecs;          // of the whole tensor
};

struct DropoutNormPlan {
    int vpt, lanes, W, groups, stages, per_sm, ctas;
    int lo_bytes;           // backward: the threads' column sums
    uint32_t rows_per_cta;
    size_t smem;
};

struct DropoutNormParams {
    Layout L;
    DropoutRng r;
    RowView in[3];          // forward: x, residual; backward: h, dy[, dh]
    RowView out[2];         // forward: y, h_new; backward: dx, dresidual
    const void *w;
    int w_f32;
    float eps;
    float *rstd_out;        // forward
    const float *rstd;      // backward
    float2 *partials;       // backward: [ctas][H] (hi, lo)
    int *status;
    uint64_t wait_ns;
    int withhold;           // tests of the waits
};

DropoutNormPlan dropout_norm_plan(int H, uint32_t rows, int ntens, bool backward);
cudaError_t launch_dropout(const DropoutParams &p, cudaStream_t stream);
cudaError_t launch_dropout_norm_fwd(const DropoutNormParams &p, const DropoutNormPlan &plan, cudaStream_t stream);
cudaError_t launch_dropout_norm_bwd(const DropoutNormParams &p, const DropoutNormPlan &plan, cudaStream_t stream);

// Column sums of (hi, lo) pairs, partials[P][H], in a fixed order; grid.y lists.
struct ColumnSumParams {
    const float2 *partials[2];
    float *out[2];
    int P[2], H;
};
cudaError_t launch_column_sum(const ColumnSumParams &p, int lists, cudaStream_t stream);

// ------------------------------------------------------------------- rotary

// Queries (list 0) and keys (list 1) go to CTAs of their own.
struct RotaryList {
    RowView in, out;        // forward: v, y; backward: dy, dv
    RowView v;              // backward: the forward's input
    uint32_t heads;
    const void *w;          // nullptr: no norm
    int w_f32;
    float *rstd_out;        // forward
    const float *rstd;      // backward
    float2 *partials;       // backward: [ctas][D] (hi, lo)
    int ctas;
    uint32_t run, rounds;   // see RotaryWalk
};

struct RotaryParams {
    RotaryList l[2];
    uint32_t tokens;
    int D, pairs, axes;
    float eps, inv_d;
    const uint64_t *turns;
    const int32_t *axis;
    const void *positions;
    int pos_i64;
    int64_t axis_stride, token_stride;
    int *status;            // [1]: an axis outside its range
};

void rotary_plan(RotaryParams &p); // sets both lists' ctas
cudaError_t launch_rotary(const RotaryParams &p, bool adjacent, bool inverse, cudaStream_t stream);
cudaError_t launch_rotary_bwd(const RotaryParams &p, bool adjacent, cudaStream_t stream);

// -------------------------------------------------------------------- gated

// A matrix of BF16 or FP32 values in memory (rows of `stride` elements).
struct Matrix {
    const void *data;
    int64_t rows, cols, stride;
};

struct GatedFwdCall {
    int64_t T, H, F;
    int gelu;
    Matrix x, w_gate, w_up, h, g, u; // g.data == nullptr: not written
    int *status;
    uint64_t wait_ns;
    int withhold;
};

struct GatedBwdCall {
    int64_t T, H, F;
    int gelu;
    Matrix dh, x, g, u, w_gate, w_up, dx, dw_gate, dw_up; // dx.data, dw_gate.data == nullptr: not wanted
    uint8_t *workspace;
    int *status;
    uint64_t wait_ns;
    int withhold;
};

size_t gated_bwd_workspace(int64_t T, int64_t H, int64_t F);
cudaError_t launch_gated_fwd(const GatedFwdCall &c, cudaStream_t stream);
cudaError_t launch_gated_bwd(const GatedBwdCall &c, cudaStream_t stream);

cudaError_t step_status_ptr(int **out);
cudaError_t ensure_smem_attr(const void *kernel, size_t smem);

// Launched while the launch before it drains: the kernels wait for that one
// before they read anything.
template <class... P, class... A>
inline cudaError_t launch_after(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                                const A &...args)
{
    if (smem > 0) {
        cudaError_t e = ensure_smem_attr((const void *)kern, smem);
        if (e != cudaSuccess)
            return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

} // namespace cake
