// cake_step_launch.h -- launch parameters and private launchers of the
// training-step operators (plain structs, passed by value to the kernels).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../csrc/cake_params.h"

namespace cake {

// ------------------------------------------------------------ sandwich norm

// A row of a sandwich norm spans a cluster of CTAs with `cols` of its columns
// each, and W warps of VPT 8-column vectors a thread in each of them; a CTA
// stages `groups` rows at a time with a producer warp.  `parts` CTAs (or
// clusters) share the rows.
struct SandwichPlan {
    int cluster, cols, vpt, W, groups, stages, per_sm, parts;
    bool half; // backward: a thread takes 4 columns more than 8 vpt
    uint32_t rows_per_cta;
    size_t smem;
};

struct SandwichLayout {
    int H, nvec, cluster, cols, W, groups, stages, ntens;
    uint32_t rows, nh, rows_per_cta;
    float inv_h;
};

struct SandwichFwdParams {
    SandwichLayout L;
    float eps, scale;
    RowView in[3];         // staged: z, x[, gate]
    RowView y, h_new;      // outputs (written through base)
    const float *gate_rows;
    const void *w_post, *w_pre;
    int post_f32, pre_f32;
    float *rstd_post, *rstd_pre;
    int *status;
    uint64_t wait_ns;
    int withhold;          // see cake_step_wait_test
};

struct SandwichBwdParams {
    SandwichLayout L;
    float scale;
    RowView in[5];         // staged: h, z, dy[, gate][, dh]
    int gate;              // 0 none, 1 a value per row, 2 a value per element
    int has_dh;
    RowView dx, dz, dgate; // outputs; dgate.base == nullptr: not wanted
    const float *gate_rows;
    float *dgate_rows;
    const float *rstd_post, *rstd_pre;
    const void *w_post, *w_pre;
    int post_f32, pre_f32;
    float2 *partials;      // [2][parts][H] (hi, lo): dw_post's, then dw_pre's
    int *status;
    uint64_t wait_ns;
    int withhold;          // see cake_step_wait_test
};

struct SandwichReduceParams {
    const float2 *partials; // [2][P][H]
    int P, H;
    float *dw[2];           // dw_post, dw_pre
};

// The build of the backward kernel that a plan takes: see sandwich_bwd_kernel.
struct SandwichBuild {
    int vpt, rw;
    bool cl, many, half;
};

SandwichBuild sandwich_build(const SandwichPlan &plan);
SandwichPlan sandwich_plan(int H, uint32_t rows, int ntens, bool backward);
cudaError_t launch_sandwich_fwd(const SandwichFwdParams &p, const SandwichPlan &plan, cudaStream_t stream);
cudaError_t launch_sandwich_bwd(const SandwichBwdParams &p, const SandwichPlan &plan, cudaStream_t stream);
cudaError_t launch_sandwich_reduce(const SandwichReduceParams &p, cudaStream_t stream);

// ----------------------------------------------- gradient norm and clipping

// Values of one chunk, the unit of work of a CTA.
constexpr int kGradChunk = 8192;
// Tensors one launch takes: they travel in the launch parameters (32 KB).
constexpr int kGradMaxTensors = 1000;
constexpr int kGradSomeTensors = 256;
constexpr int kGradFewTensors = 32;
constexpr int kGradThreads = 256;
// CTAs of the norm's launches, at most (each leaves a partial), and of the
// scaling's: GB300, 0.65 G BF16 values into FP32 812 us with 8 an SM in both,
// 793 us with 48 of the scaling's.
constexpr int kGradCtas = 152 * 8;
constexpr int kGradClipCtas = 152 * 48;

// A list of at most kGradFewTensors tensors in kGradOnePieces pieces runs in one CTA.
constexpr int kGradPiece = 512;
constexpr int kGradOneThreads = 1024;
constexpr int kGradOnePieces = 64;

struct GradDesc {
    const void *src;
    void *dst;
    int64_t count;
    uint32_t chunk0;       // the tensor's first chunk (one CTA: piece) in this launch
    uint32_t flags;        // kGrad*
};
constexpr uint32_t kGradSrcF32 = 1, kGradDstF32 = 2, kGradVector = 4; // kGradVector: 16-byte accesses are aligned

template <int N>
struct GradParams {
    int n;
    int npartials;         // clip: partials of the whole norm
    uint32_t chunks;
    float max_norm, eps;
    int in_place;          // clip: nothing to write where coef is 1
    float *norm;           // clip: where CTA 0 of the first launch writes the norm (else nullptr)
    double *partials;      // norm: this launch's [ctas]; clip: all
    GradDesc t[N];
};

template <int N>
cudaError_t launch_grad_sumsq(const GradParams<N> &p, int ctas, cudaStream_t stream);
template <int N>
cudaError_t launch_grad_clip(const GradParams<N> &p, int ctas, cudaStream_t stream);
cudaError_t launch_grad_one(const GradParams<kGradFewTensors> &p, bool clip, cudaStream_t stream);
cudaError_t launch_grad_final(const double *partials, int n, float *norm, cudaStream_t stream);

// ---------------------------------------------------------------- embedding

struct EmbedFwdParams {
    const void *ids;
    int ids_i64;
    uint32_t tokens;
    int nvec;              // H / 8
    const void *table;
    int table_f32;
    int64_t vocab, table_stride;
    float scale;
    uint16_t *y;
    int64_t y_stride;
    int *status;
};

// Sorting: keys (id, token), the tokens without a gradient under key `vocab`.
constexpr int kSortThreads = 256;
constexpr int kSortPerThread = 8;
constexpr int kSortBlock = kSortThreads * kSortPerThread; // keys ranked together
constexpr int kSortMaxTiles = 304;
constexpr int kSortMaxBits = 8;                            // bits of a pass
constexpr int kSegMaxThreads = 128;                        // of a CTA of the sums
constexpr int kSegMaxWindow = 128;                         // sorted positions of such a CTA
constexpr int kSegMinWindow = 8;
constexpr int kClusterThreads = 1024;                      // of each CTA of the one-launch sort
constexpr int kMaxSortCluster = 16;
constexpr int64_t kClusterSortKeys = 8 * kClusterThreads * kMaxSortCluster;

struct SortParams {
    const void *ids;
    int ids_i64;
    uint32_t tokens;
    uint32_t vocab;
    int64_t padding_idx;
    uint32_t tile_keys;    // keys of a tile (a CTA's), a multiple of kSortBlock
    int tiles;
    int passes;
    int bits;              // of each pass
    uint64_t *pairs[2];    // (key << 32) | token, ping-pong
    uint32_t *hist;        // [passes][tiles][1 << bits], zero before the first pass
    uint32_t *present;     // bitmap of ids with a token, zero before the first pass (nullptr: not wanted)
    int zero_present;      // one-launch sort: zero the bitmap itself
    uint32_t *ready;       // [0] one-launch sort: set to 1 once the bitmap is complete; [1] zero for the sums;
                           // [2] tests of the waits: stays 0
    int *status;
};

struct SegmentParams {
    const uint64_t *pairs; // sorted
    uint32_t tokens;
    uint32_t vocab;
    int window;            // sorted positions of a CTA
    int windows, slices;   // CTAs of the sums: windows x column slices
    int threads;           // of such a CTA, 8 columns each
    int nvec;
    const uint16_t *dy;
    int64_t dy_stride;
    float scale;
    void *dtable;
    int dtable_f32;
    int64_t dtable_stride;
    int accumulate;
    const uint32_t *present;
    int fill_ctas;         // CTAs before the sums' that zero the rows without a token
    int fill_rows;         // rows that a warp of those takes at a time: a power of two, at most 32
    const uint32_t *ready; // those start at this flag; nullptr: after the sort
    uint64_t wait_ns;
    int *status;
    float *partials;       // [windows][2][H]: sums of the leading and the trailing piece
    uint32_t *meta;        // [windows][2]: flags and the trailing piece's id
    uint32_t *cut;         // [windows]: the windows in which a cut run starts, *cuts of them
    uint32_t *cuts;
    int join_lanes;        // threads of the join over a piece's columns, 8 each
};

cudaError_t launch_embed_fwd(const EmbedFwdParams &p, cudaStream_t stream);
cudaError_t launch_embed_cluster_sort(const SortParams &p, int ctas, cudaStream_t stream);
cudaError_t launch_embed_sort(const SortParams &p, uint64_t **sorted, cudaStream_t stream);
cudaError_t launch_embed_segments(const SegmentParams &p, cudaStream_t stream);
cudaError_t launch_embed_join(const SegmentParams &p, cudaStream_t stream);

cudaError_t step_status(int *code, int clear);
cudaError_t step_status_ptr(int **out); // two words: waits that ran out, ids outside their table

} // namespace cake
