// cake_gated.cu -- the gated feed-forward block for sm_103a: both projections,
// the activation and the product in one kernel, and its gradients.
//
//   forward   g = x Wg^T, u = x Wu^T, h = act(g) u
//   backward  dg = dh u act'(g), du = dh act(g)           (gated_grad_kernel)
//             dx = [dg du] [Wg; Wu], dWg = dg^T x, dWu = du^T x   (one launch)
//
// Products run on tcgen05 with FP32 accumulators in tensor memory.  A pair of
// CTAs (two SMs) works on tiles of 256 x 256: each CTA stages 128 rows of A and
// half of B, and one thread of the pair issues the products.  The forward's 256
// columns are 128 of g and the same 128 of u, one half of B from each weight, so
// that the epilogue finds both factors of h in its own registers.  While the
// tensor cores fill one accumulator of 256 columns, eight warps empty the other.
// No operand is transposed in memory: the copies and the descriptors take
// operands along k or across it.
//
// A few tokens leave such tiles empty and only the weights' bytes count; then
// 128 rows of each weight are the products' m and the tokens their n, and a
// cluster of CTAs shares the sum over k (gated_few_kernel).
#include <cuda.h>

#include "../csrc/cake_rows.cuh"
#include "cake_block_launch.h"
#include "cake_mma.cuh"

namespace cake {

// ---------------------------------------------------------------- activation

__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

constexpr float kGeluA = 1.5957691216057308f; // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

// act(v), and its derivative.  (1 + tanh(z)) / 2 is sigmoid(2 z).
template <bool GRAD>
__device__ __forceinline__ float activation(float v, bool gelu, float &d)
{
    if (!gelu) {
        const float s = sigmoid(v);
        if (GRAD)
            d = s * fmaf(v, 1.0f - s, 1.0f);
        return v * s;
    }
    // (beyond |v| = 16 the sigmoid is 0 or 1 in FP32, and so is the derivative)
    const float v2 = fminf(v * v, 256.0f);
    const float s = sigmoid(kGeluA * v * fmaf(kGeluB, v2, 1.0f));
    if (GRAD)
        d = fmaf(v * s * (1.0f - s), kGeluA * fmaf(3.0f * kGeluB, v2, 1.0f), s);
    return v * s;
}

// --------------------------------------------------------------------- pairs

constexpr int kPairStages = 6;
constexpr int kPairHalf = 16384;              // an operand of a stage: 128 x 64 BF16
constexpr int kPairStage = 2 * kPairHalf;
constexpr int kPairBox = 2048;                // a box of the outputs: 32 rows of 64 bytes
constexpr int kPairBoxes = 2;                 // of each epilogue warp
constexpr int kPairWriters = 8;               // epilogue warps: two to a quarter of the rows
constexpr int kPairStaging = kPairStages * kPairStage;
constexpr int kPairBars = kPairStaging + kPairWriters * kPairBoxes * kPairBox;
constexpr int kPairSmem = kPairBars + 256;
constexpr int kPairThreads = 128 + 32 * kPairWriters;
constexpr int kPairs = kSMsBlock / 2;
constexpr int kPairGroup = 8;                 // tiles of m that neighbouring units share, for their reuse in L2

// Products out[half] = sum over segments, k and an a's parts of a b.
struct PairProblem {
    CUtensorMap a[4], b[2], out[2];
    int a_mn, b_mn;       // an operand's rows lie along k in memory
    int segments, halves; // a, b by segment; or a, out by half
    int parts;            // a is a sum of so many matrices: a[segment or half][part], with b[part]
    int stack;            // instead: two of at most 64 rows, above one another in the tile
    int kblocks;          // blocks of 64 k of a segment
    int tiles_m, tiles_n; // of a half
    int splits, per_split; // of the sum over all segments
    int planes;           // FP32 parts of the outputs in out[.][plane] (splits, twice those with stack); 0: none
    int units;
    int rows, cols;       // of a half
};

struct PairParams {
    PairProblem p[2];
    CUtensorMap g, u;     // gated: outputs beside out[0]
    int save, gelu;
    // Of the first problem's units a pair takes `each`, the first `more` pairs
    // one more; of the second's these take `less`, the others `rest`.
    int pairs, each, more, less, rest;
    int *status;
    uint64_t wait_ns;
    int withhold;         // tests of the waits
};

struct PairUnit {
    const PairProblem *p;
    int half, split, m0, n0, k0, k1;
};

// The i-th unit of pair q; false: there is none.  Neighbouring pairs work on
// neighbouring units at a time.
template <bool GATED>
__device__ __forceinline__ bool pair_unit(const PairParams &P, int q, int i, PairUnit &r)
{
    const int own = P.each + (q < P.more);
    int u;
    if (i < own) {
        u = i * P.pairs + q;
        r.p = &P.p[0];
    } else {
        if (GATED)
            return false;
        i -= own;
        if (i >= (q < P.more ? P.less : P.rest))
            return false;
        u = i < P.less ? i * P.pairs + q : P.less * P.pairs + (i - P.less) * (P.pairs - P.more) + q - P.more;
        r.p = &P.p[1];
        if (u >= r.p->units)
            return false;
    }
    const PairProblem &p = *r.p;
    r.split = u % p.splits;
    int t = u / p.splits;
    const int per_half = p.tiles_m * p.tiles_n;
    r.half = t / per_half;
    t -= r.half * per_half;
    const int first = t / (kPairGroup * p.tiles_n) * kPairGroup, size = min(kPairGroup, p.tiles_m - first);
    t -= first * p.tiles_n;
    r.m0 = (first + t % size) * 256;
    r.n0 = t / size * (GATED ? 128 : 256);
    r.k0 = r.split * p.per_split;
    r.k1 = min(r.k0 + p.per_split, p.kblocks * p.segments * p.parts);
    return true;
}

// 32 rows of 64 bytes in 64-byte swizzled order, one row a lane, to the boxes' next slot and on to memory.
struct BoxWriter {
    uint32_t base;
    uint32_t n;

    template <class Store>
    __device__ __forceinline__ void put(const uint32_t (&w)[16], int lane, Store store)
    {
        if (lane == 0)
            store_wait_read<kPairBoxes - 1>(); // the slot's last store has read it
        __syncwarp();
        const uint32_t box = base + (n++ % kPairBoxes) * kPairBox, row = box + lane * 64, x = (lane >> 1) & 3;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + ((j ^ x) << 4)), "r"(w[4 * j]),
                         "r"(w[4 * j + 1]), "r"(w[4 * j + 2]), "r"(w[4 * j + 3])
                         : "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            store(box);
            store_commit();
        }
    }
};

// Warp 0 of each CTA copies, warp 1 of the first issues the products, warp 2
// holds the tensor memory, warps 4 to 11 write the outputs (each a quarter of
// the CTA's rows, as tensor memory is laid out, and half of the columns).
template <bool GATED>
__global__ void __launch_bounds__(kPairThreads, 1) gated_pair_kernel(const __grid_constant__ PairParams P)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t smem = smem_addr(smem_raw), bars = smem + kPairBars;
    const uint32_t full = bars, empty = bars + 8 * kPairStages, tfull = empty + 8 * kPairStages, tempty = tfull + 16,
                   drain = tempty + 16, tmem_at = drain + 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1;
    PairUnit u;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kPairStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull + 8 * i, 1);
            mbar_init(tempty + 8 * i, 2 * kPairWriters);
        }
        mbar_init(drain, 1);
        fence_mbar_init();
    }
    if (warp == 2) {
        tmem_alloc<2>(tmem_at, 512);
        tmem_relinquish<2>();
        tc_fence_before();
    }
    __syncwarp();
    cluster_sync_all(); // both CTAs' barriers exist, and the tensor memory is theirs
    tc_fence_after();
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tmem_at) : "memory");
    pdl_launch_dependents();
    pdl_wait();
    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            uint32_t st = 0, ph = 0, issued = 0;
            for (int i = 0; ok && pair_unit<GATED>(P, pair, i, u); ++i) {
                const PairProblem &p = *u.p;
                for (int kb = u.k0; kb < u.k1; ++kb) {
                    if (issued >= kPairStages && !(ok = mbar_wait(empty + 8 * st, ph ^ 1u, P.wait_ns)))
                        break;
                    // the first CTA's barrier counts both CTAs' copies
                    if (rank == 0)
                        mbar_arrive_expect_tx(full + 8 * st,
                                              2 * kPairStage + (P.withhold && issued == 0 ? 16 : 0));
                    const uint32_t bar = map_to_rank(full + 8 * st, 0);
                    const uint32_t sa = smem + st * kPairStage, sb = sa + kPairHalf;
                    // (the parts of a block follow one another)
                    const int part = p.parts == 2 ? kb & 1 : 0, block = p.parts == 2 ? kb >> 1 : kb;
                    const int seg = block >= p.kblocks, k = (block - seg * p.kblocks) * 64;
                    const CUtensorMap *ma = &p.a[(p.segments == 2 ? seg : u.half) * p.parts + part];
                    const int m = u.m0 + 128 * rank;
                    if (p.a_mn) {
                        tile_g2s_pair(sa, ma, m, k, bar);
                        tile_g2s_pair(sa + 8192, ma, m + 64, k, bar);
                    } else if (!GATED && p.stack) { // (the second CTA's rows lie outside: zeros)
                        tile_g2s_pair(sa, &p.a[2 * seg], k, 128 * rank, bar);
                        tile_g2s_pair(sa + 8192, &p.a[2 * seg + 1], k, 128 * rank, bar);
                    } else {
                        tile_g2s_pair(sa, ma, k, m, bar);
                    }
                    if (GATED) {
                        tile_g2s_pair(sb, &p.b[rank], k, u.n0, bar);
                    } else {
                        const CUtensorMap *mb = &p.b[seg + part]; // (two of either, never of both)
                        const int n = u.n0 + 128 * rank;
                        tile_g2s_pair(sb, mb, n, k, bar);
                        tile_g2s_pair(sb + 8192, mb, n + 64, k, bar);
                    }
                    ++issued;
                    if (++st == kPairStages) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
            }
            // no copy of the pair is left in flight
            if (rank == 0 && !ok)
                for (uint32_t j = issued > kPairStages ? issued - kPairStages : 0; j < issued; ++j)
                    (void)mbar_wait(full + 8 * (j % kPairStages), (j / kPairStages) & 1, P.wait_ns);
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            uint32_t st = 0, ph = 0;
            for (int it = 0; ok && pair_unit<GATED>(P, pair, it, u); ++it) {
                const PairProblem &p = *u.p;
                const uint32_t acc = it & 1, desc = mma_desc(256, 256, p.a_mn, p.b_mn);
                if (it >= 2 && !(ok = mbar_wait_cluster(tempty + 8 * acc, ((it >> 1) & 1) ^ 1u, P.wait_ns)))
                    break;
                tc_fence_after();
                // 16 k further, in units of 16 bytes
                const uint64_t step_a = p.a_mn ? 128 : 2, step_b = p.b_mn ? 128 : 2;
                for (int kb = u.k0; kb < u.k1; ++kb) {
                    if (!(ok = mbar_wait(full + 8 * st, ph, P.wait_ns)))
                        break;
                    tc_fence_after();
                    const uint32_t sa = smem + st * kPairStage;
                    const uint64_t da = operand_desc(sa, p.a_mn), db = operand_desc(sa + kPairHalf, p.b_mn);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        mma_bf16<2>(tmem + 256 * acc, da + q * step_a, db + q * step_b, desc, kb > u.k0 || q > 0);
                    mma_commit_pair(empty + 8 * st);
                    if (++st == kPairStages) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
                if (ok)
                    mma_commit_pair(tfull + 8 * acc);
            }
            if (!ok) { // no product is left in flight
                mma_commit_pair(drain);
                (void)mbar_wait(drain, 0, P.wait_ns);
            }
        }
    } else if (warp >= 4) {
        const int quad = warp & 3, side = (warp - 4) >> 2;
        BoxWriter box{smem + kPairStaging + (uint32_t)(warp - 4) * kPairBoxes * kPairBox, 0};
        for (int it = 0; ok && pair_unit<GATED>(P, pair, it, u); ++it) {
            const PairProblem &p = *u.p;
            const uint32_t acc = it & 1;
            ok = __all_sync(0xffffffffu, mbar_wait_cluster(tfull + 8 * acc, (it >> 1) & 1, P.wait_ns));
            if (!ok)
                break;
            tc_fence_after();
            const uint32_t t = tmem + ((uint32_t)(quad * 32) << 16) + 256 * acc;
            int row = u.m0 + 128 * (int)rank + 32 * quad, plane = u.split;
            if (!GATED && p.stack && row >= 64 && row < 128) {
                row -= 64;
                plane += p.splits;
            }
            const bool rows = row < p.rows;
            constexpr int kSide = GATED ? 2 : 4; // chunks of 32 columns
            for (int c = kSide * side; c < kSide * (side + 1); ++c) {
                const int col = u.n0 + 32 * c;
                if (!rows || col >= p.cols)
                    break;
                uint32_t w[16];
                if constexpr (GATED) {
                    uint32_t g[32], v[32];
                    tmem_ld32(t + 32 * c, g);
                    tmem_ld32(t + 128 + 32 * c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float d;
                        const float a = activation<false>(__uint_as_float(g[2 * j]), P.gelu, d);
                        const float b = activation<false>(__uint_as_float(g[2 * j + 1]), P.gelu, d);
                        w[j] = pack_bf16(a * __uint_as_float(v[2 * j]), b * __uint_as_float(v[2 * j + 1]));
                    }
                    box.put(w, lane, [&](uint32_t at) { tile_s2g(&p.out[0], col, row, at); });
                    if (P.save) {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            w[j] = pack_bf16(__uint_as_float(g[2 * j]), __uint_as_float(g[2 * j + 1]));
                        box.put(w, lane, [&](uint32_t at) { tile_s2g(&P.g, col, row, at); });
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            w[j] = pack_bf16(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
                        box.put(w, lane, [&](uint32_t at) { tile_s2g(&P.u, col, row, at); });
                    }
                } else {
                    uint32_t v[32];
                    tmem_ld32(t + 32 * c, v);
                    tmem_wait_ld();
                    if (p.planes == 0) {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            w[j] = pack_bf16(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
                        box.put(w, lane, [&](uint32_t at) { tile_s2g(&p.out[u.half], col, row, at); });
                    } else {
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                w[j] = v[16 * s + j];
                            if (col + 16 * s < p.cols)
                                box.put(w, lane,
                                        [&](uint32_t at) { tile_s2g(&p.out[u.half], col + 16 * s, row, plane, at); });
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_remote(map_to_rank(tempty + 8 * acc, 0));
        }
        if (lane == 0)
            store_wait_read<0>(); // (the launch's end completes the writes)
    }
    if (!ok) {
        // Nothing of the pair is left in flight when its CTAs leave: copies of
        // the second CTA may be on no barrier that it can wait for, and take
        // some microseconds at most.
        if (lane == 0)
            set_status(P.status, kStatusTimeout);
        for (int i = 0; i < 1000; ++i)
            __nanosleep(1000);
    }
    __syncwarp();
    cluster_sync_all();
    if (warp == 2)
        tmem_free<2>(tmem, 512);
}

// ---------------------------------------------------------------- few tokens

constexpr int kFewThreads = 256;
// GB300, pairs of CTAs against this kernel: 4096 to 8192 at 64 tokens 29 us and 26,
// at 128 30 and 29.9; 1024 to 1024 10.3 and 7.3, 10.5 and 9.5.
constexpr int kFewMostTokens = 128;
constexpr int kFewWeights = 32768; // of a stage: 128 rows of each weight, 64 k

struct FewParams {
    CUtensorMap x, w_gate, w_up;
    uint16_t *h, *g, *u;   // g == nullptr: not written
    int64_t h_stride, g_stride, u_stride;
    int T, F, kblocks;
    int n;                 // T rounded up to 16
    int columns;           // of tensor memory
    int stages, per_rank;  // blocks of k of a CTA of the cluster
    int ahead;             // of these brought to L2 while the launch before drains: weights that it
                           // writes are written in L2 too, so what is read after the wait is whole
    int gelu;
    int *status;
    uint64_t wait_ns;
    int withhold;
};

// Outputs from the cluster's sums: every one is four neighbours of f, `first`
// and every `step`-th after it are this thread's, U of them with the parts of R
// CTAs on their way at once.
template <int U, int R>
__device__ __forceinline__ void few_outputs(const FewParams &P, uint32_t smem, int f0, int first, int step, int C)
{
    const int total = P.T * 32; // [n][128] in fours, in the order of i
    for (int i0 = first; i0 < total; i0 += U * step) {
        float4 g[U], u[U];
#pragma unroll
        for (int k = 0; k < U; ++k)
            g[k] = u[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int r0 = 0; r0 < C; r0 += R) { // in the order of k
            float4 x[R][U], y[R][U];
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int k = 0; k < U; ++k)
                    if (r0 + r < C && i0 + k * step < total) {
                        const uint32_t at = map_to_rank(smem, r0 + r) + 16 * (uint32_t)(i0 + k * step);
                        x[r][k] = ld_cluster_f4(at);
                        y[r][k] = ld_cluster_f4(at + (uint32_t)P.n * 512);
                    }
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int k = 0; k < U; ++k)
                    if (r0 + r < C) {
                        const float4 a = x[r][k], b = y[r][k];
                        g[k] = make_float4(g[k].x + a.x, g[k].y + a.y, g[k].z + a.z, g[k].w + a.w);
                        u[k] = make_float4(u[k].x + b.x, u[k].y + b.y, u[k].z + b.z, u[k].w + b.w);
                    }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int i = i0 + k * step, t = i >> 5, f = f0 + 4 * (i & 31);
            if (i >= total || f >= P.F) // (F is a multiple of 8)
                continue;
            float d;
            const float h0 = activation<false>(g[k].x, P.gelu, d) * u[k].x,
                        h1 = activation<false>(g[k].y, P.gelu, d) * u[k].y,
                        h2 = activation<false>(g[k].z, P.gelu, d) * u[k].z,
                        h3 = activation<false>(g[k].w, P.gelu, d) * u[k].w;
            auto put = [&](uint16_t *m, int64_t stride, float a, float b, float c, float e) {
                *reinterpret_cast<uint2 *>(m + (int64_t)t * stride + f) = make_uint2(pack_bf16(a, b), pack_bf16(c, e));
            };
            put(P.h, P.h_stride, h0, h1, h2, h3);
            if (P.g) {
                put(P.g, P.g_stride, g[k].x, g[k].y, g[k].z, g[k].w);
                put(P.u, P.u_stride, u[k].x, u[k].y, u[k].z, u[k].w);
            }
        }
    }
}

__global__ void __launch_bounds__(kFewThreads) gated_few_kernel(const __grid_constant__ FewParams P)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ uint64_t s_bars[18];
    __shared__ uint32_t s_tmem;
    __shared__ int s_bad;
    const uint32_t smem = smem_addr(smem_raw), full = smem_addr(s_bars), empty = full + 64, done = full + 128;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank(), C = gridDim.x, f0 = blockIdx.y * 128;
    const uint32_t stage = kFewWeights + 128u * P.n;
    const int k0 = rank * P.per_rank, k1 = min(k0 + P.per_rank, P.kblocks);
    if (threadIdx.x == 0) {
        for (int i = 0; i < P.stages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        mbar_init(done, 1);
        s_bad = 0;
        fence_mbar_init();
    }
    if (warp == 2) {
        tmem_alloc<1>(smem_addr(&s_tmem), P.columns);
        tmem_relinquish<1>();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        prefetch_map(&P.x);
        for (int kb = k0; kb < min(k1, k0 + P.ahead); ++kb) {
            tile_prefetch(&P.w_gate, kb * 64, f0);
            tile_prefetch(&P.w_up, kb * 64, f0);
        }
    }
    pdl_wait();
    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            uint32_t st = 0, ph = 0, issued = 0;
            for (int kb = k0; kb < k1; ++kb, ++issued) {
                if (issued >= (uint32_t)P.stages && !(ok = mbar_wait(empty + 8 * st, ph ^ 1u, P.wait_ns)))
                    break;
                const uint32_t at = smem + st * stage, bar = full + 8 * st;
                mbar_arrive_expect_tx(bar, stage + (P.withhold && issued == 0 ? 16 : 0));
                tile_g2s(at, &P.w_gate, kb * 64, f0, bar);
                tile_g2s(at + 16384, &P.w_up, kb * 64, f0, bar);
                tile_g2s(at + kFewWeights, &P.x, kb * 64, 0, bar);
                if (++st == (uint32_t)P.stages) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            // No copy is left in flight, whichever warp's wait ran out: this warp
            // waits for the last ones itself, for as long as all waits may take.
            for (uint32_t j = issued > (uint32_t)P.stages ? issued - P.stages : 0; j < issued; ++j)
                ok = mbar_wait(full + 8 * (j % P.stages), (j / P.stages) & 1, P.wait_ns) && ok;
        }
    } else if (warp == 1) {
        if (lane == 0) {
            uint32_t st = 0, ph = 0;
            const uint32_t desc = mma_desc(128, P.n, false, false);
            for (int kb = k0; kb < k1; ++kb) {
                if (!(ok = mbar_wait(full + 8 * st, ph, P.wait_ns)))
                    break;
                tc_fence_after();
                const uint32_t at = smem + st * stage;
                const uint64_t dg = operand_desc(at, false), du = operand_desc(at + 16384, false),
                               dx = operand_desc(at + kFewWeights, false);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    mma_bf16<1>(tmem, dg + 2 * q, dx + 2 * q, desc, kb > k0 || q > 0);
                    mma_bf16<1>(tmem + P.n, du + 2 * q, dx + 2 * q, desc, kb > k0 || q > 0);
                }
                mma_commit(empty + 8 * st);
                if (++st == (uint32_t)P.stages) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            mma_commit(done);
            ok = mbar_wait(done, 0, P.wait_ns) && ok;
        }
    }
    if (!ok) {
        s_bad = 1;
        set_status(P.status, kStatusTimeout);
        // (a copy that the waits have not seen takes some microseconds more at most)
        for (int i = 0; i < 1000; ++i)
            __nanosleep(1000);
    }
    __syncthreads(); // where no wait ran out every copy has landed and every product is done: the ring is free
    tc_fence_after();
    const bool bad = s_bad;
    float *part = reinterpret_cast<float *>(smem_raw); // [gate, up][n][128]
    if (!bad) {
        // a warp's lanes are a quarter of the rows; two warps share it by columns
        const int f = (warp & 3) * 32 + lane, half = warp >> 2;
        const uint32_t t = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        for (int c = half * P.n; c < (half + 1) * P.n; c += 16) {
            uint32_t v[16];
            if (k1 > k0) {
                tmem_ld16(t + c, v);
                tmem_wait_ld();
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    v[j] = 0;
            }
#pragma unroll
            for (int j = 0; j < 16; ++j)
                part[(c + j) * 128 + f] = __uint_as_float(v[j]);
        }
        tc_fence_before();
    }
    __syncwarp();
    cluster_sync_all();
    if (!bad) {
        const int first = rank * kFewThreads + (int)threadIdx.x, step = C * kFewThreads;
        if (C == 1) // (100 tokens, 64 to 128: 6.9 us against 9.7 with one output at a time)
            few_outputs<4, 1>(P, smem, f0, first, step, C);
        else if (C == 2) // (64 tokens, 4096 to 8192: 26.0 us against 26.4 with one; 128 tokens 29.9 against 31.0)
            few_outputs<2, 2>(P, smem, f0, first, step, C);
        else // (100 tokens, 696 to 904, clusters of 5: 9.0 us against 9.9 with two)
            few_outputs<1, 4>(P, smem, f0, first, step, C);
    }
    __syncwarp();
    cluster_sync_all(); // no CTA leaves while another reads its sums
    if (warp == 2)
        tmem_free<1>(tmem, P.columns);
}

// ------------------------------------------------------------ gradients of g, u

constexpr int kGradGuThreads = 256;

struct GatedGradParams {
    const uint16_t *dh, *g, *u;
    int64_t dh_stride, g_stride, u_stride;
    uint16_t *dg, *du;     // rows of 8 nvec
    int64_t rest;          // REST: bytes from there to what their rounding left
    uint32_t nvec;
    uint64_t vecs;
    int gelu;
    // REST: the rests' factor of dWg and dWu, x with 0 for what is not finite.  The
    // values' products make such a result what it is; a rest of the other sign or of
    // 0 would turn an infinity into NaN.
    const uint16_t *x;
    int64_t x_stride;
    uint16_t *x_finite;    // rows of 8 x_nvec
    uint32_t x_nvec;
    uint64_t x_vecs;
};

__device__ __forceinline__ float2 rest_of(float2 v, uint32_t rounded)
{
    const float2 r = bf2(rounded);
    return make_float2(isfinite(r.x) ? v.x - r.x : 0.f, isfinite(r.y) ? v.y - r.y : 0.f);
}

// A word of two BF16 values, 0 for an infinity or NaN.
__device__ __forceinline__ uint32_t finite2(uint32_t w)
{
    const uint32_t e = 0x7f80u;
    return ((w & e) == e ? 0u : w & 0xffffu) | ((w & e << 16) == e << 16 ? 0u : w & 0xffff0000u);
}

template <bool REST>
__global__ void __launch_bounds__(kGradGuThreads) gated_grad_kernel(const __grid_constant__ GatedGradParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    if (REST && blockIdx.y == 1) { // x, beside the gradients (64 tokens, 4096 to 512: 12.3 us, behind them 12.5)
        for (uint64_t i = (uint64_t)blockIdx.x * kGradGuThreads + threadIdx.x; i < p.x_vecs;
             i += (uint64_t)gridDim.x * kGradGuThreads) {
            const uint64_t t = i / p.x_nvec;
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(p.x + t * p.x_stride + (i - t * p.x_nvec) * 8));
            reinterpret_cast<uint4 *>(p.x_finite)[i] = make_uint4(finite2(x.x), finite2(x.y), finite2(x.z), finite2(x.w));
        }
        return;
    }
    for (uint64_t i = (uint64_t)blockIdx.x * kGradGuThreads + threadIdx.x; i < p.vecs;
         i += (uint64_t)gridDim.x * kGradGuThreads) {
        const uint64_t t = i / p.nvec;
        const uint32_t c = (uint32_t)(i - t * p.nvec) * 8;
        const uint4 d = __ldcs(reinterpret_cast<const uint4 *>(p.dh + t * p.dh_stride + c));
        const uint4 g = __ldcs(reinterpret_cast<const uint4 *>(p.g + t * p.g_stride + c));
        const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(p.u + t * p.u_stride + c));
        uint32_t og[4], ou[4], rg[4], ru[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 dq = bf2(word(d, q)), gq = bf2(word(g, q)), uq = bf2(word(u, q));
            float d0, d1;
            const float a0 = activation<true>(gq.x, p.gelu, d0), a1 = activation<true>(gq.y, p.gelu, d1);
            const float2 vg = make_float2(dq.x * uq.x * d0, dq.y * uq.y * d1), vu = make_float2(dq.x * a0, dq.y * a1);
            og[q] = pack2(vg);
            ou[q] = pack2(vu);
            if (REST) { // (the differences are exact; of what is not finite there is none)
                rg[q] = pack2(rest_of(vg, og[q]));
                ru[q] = pack2(rest_of(vu, ou[q]));
            }
        }
        uint4 *const dg = reinterpret_cast<uint4 *>(p.dg) + i, *const du = reinterpret_cast<uint4 *>(p.du) + i;
        *dg = make_uint4(og[0], og[1], og[2], og[3]);
        *du = make_uint4(ou[0], ou[1], ou[2], ou[3]);
        if (REST) {
            dg[p.rest / 16] = make_uint4(rg[0], rg[1], rg[2], rg[3]);
            du[p.rest / 16] = make_uint4(ru[0], ru[1], ru[2], ru[3]);
        }
    }
}

// Sum of a split product's FP32 parts in their order, rounded to BF16.  REST:
// where that is not finite the parts of the rounded gradients are the result, as
// what an infinite factor makes of the rests' parts may be NaN.
struct JoinParams {
    const float *part[2];  // [planes] of rows x cols, dense
    int64_t plane;         // elements from one to the next
    int planes;
    int values;            // REST: the first of them, of the rounded gradients
    uint16_t *out[2];
    int64_t stride[2];
    uint32_t nvec;
    uint64_t vecs;         // of one output
};

__device__ __forceinline__ float4 finite_or(float4 v, float4 w)
{
    return make_float4(isfinite(v.x) ? v.x : w.x, isfinite(v.y) ? v.y : w.y, isfinite(v.z) ? v.z : w.z,
                       isfinite(v.w) ? v.w : w.w);
}

template <bool REST>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ JoinParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    const int o = blockIdx.y;
    for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < p.vecs; i += (uint64_t)gridDim.x * 256) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a, va = a, vb = a;
        const float *at = p.part[o] + i * 8;
        for (int s = 0; s < p.planes; ++s, at += p.plane) {
            const float4 x = __ldcs(reinterpret_cast<const float4 *>(at)),
                         y = __ldcs(reinterpret_cast<const float4 *>(at) + 1);
            a = make_float4(a.x + x.x, a.y + x.y, a.z + x.z, a.w + x.w);
            b = make_float4(b.x + y.x, b.y + y.y, b.z + y.z, b.w + y.w);
            if (REST && s == p.values - 1) {
                va = a;
                vb = b;
            }
        }
        if (REST) {
            a = finite_or(a, va);
            b = finite_or(b, vb);
        }
        const uint64_t r = i / p.nvec;
        reinterpret_cast<uint4 *>(p.out[o] + r * p.stride[o])[i - r * p.nvec] =
            make_uint4(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w), pack_bf16(b.x, b.y), pack_bf16(b.z, b.w));
    }
}

// ------------------------------------------------------------------- launch

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder of tensor maps (the library does not link the driver).
static EncodeTiled encoder()
{
    static const EncodeTiled f = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &r) !=
                cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<EncodeTiled>(fn);
    }();
    return f;
}

// BF16 tiles of 64 columns in 128-byte swizzled rows: operands.
static bool operand_map(CUtensorMap *m, const Matrix &x, int box_rows)
{
    const cuuint64_t dims[2] = {(cuuint64_t)x.cols, (cuuint64_t)x.rows}, strides[1] = {(cuuint64_t)x.stride * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, one[2] = {1, 1};
    return encoder() && encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(x.data), dims, strides,
                                  box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Boxes of 32 rows of 64 bytes, swizzled: outputs.
static bool output_map(CUtensorMap *m, const Matrix &x)
{
    const cuuint64_t dims[2] = {(cuuint64_t)x.cols, (cuuint64_t)x.rows}, strides[1] = {(cuuint64_t)x.stride * 2};
    const cuuint32_t box[2] = {32, 32}, one[2] = {1, 1};
    return encoder() && encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(x.data), dims, strides,
                                  box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                                  CU_TENSOR_MAP_L2_PROMOTION_NONE,
                                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same of `splits` planes of FP32 values.
static bool parts_map(CUtensorMap *m, const Matrix &x, int64_t plane, int splits)
{
    const cuuint64_t dims[3] = {(cuuint64_t)x.cols, (cuuint64_t)x.rows, (cuuint64_t)splits};
    const cuuint64_t strides[2] = {(cuuint64_t)x.stride * 4, (cuuint64_t)plane * 4};
    const cuuint32_t box[3] = {16, 32, 1}, one[3] = {1, 1, 1};
    return encoder() && encoder()(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void *>(x.data), dims, strides,
                                  box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                                  CU_TENSOR_MAP_L2_PROMOTION_NONE,
                                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class P>
static cudaError_t launch_cluster(void (*kern)(P), dim3 grid, int cluster, int threads, size_t smem,
                                  cudaStream_t stream, const P &p)
{
    cudaError_t e = ensure_smem_attr((const void *)kern, smem);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kern, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

static int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

static cudaError_t launch_few(const GatedFwdCall &c, cudaStream_t stream)
{
    FewParams P{};
    P.T = (int)c.T;
    P.F = (int)c.F;
    P.kblocks = ceil_div(c.H, 64);
    P.n = ceil_div(c.T, 16) * 16;
    P.columns = 32;
    while (P.columns < 2 * P.n)
        P.columns *= 2;
    // CTAs that share k: as many as run at a time, two an SM where their stages
    // are small.  Clusters leave some SMs of their processing clusters without
    // one: GB300, one token, 2048 to 6144 (48 tiles), clusters of 4, 5 and 6
    // CTAs 11.5, 10.8 and 16.3 us; 64 tokens, 4096 to 8192 (64 tiles, one CTA an
    // SM), clusters of 1, 2 and 3 31, 26 and 35 us.
    const int per_sm = P.n <= 32 ? 2 : 1, tiles = ceil_div(c.F, 128), fit = kSMsBlock * per_sm * 27 / 32;
    int cluster = 1;
    while (cluster < 8 && tiles * (cluster + 1) <= fit && P.kblocks >= 2 * (cluster + 1))
        ++cluster;
    P.per_rank = ceil_div(P.kblocks, cluster);
    P.ahead = 4; // (a token 10.8 us against 11.1)
    const size_t stage = kFewWeights + 128 * (size_t)P.n;
    P.stages = (int)((per_sm == 2 ? 112 * 1024 : 224 * 1024) / stage);
    P.stages = P.stages > 8 ? 8 : P.stages;
    size_t smem = P.stages * stage;
    if (smem < (size_t)P.n * 1024) // the sums
        smem = (size_t)P.n * 1024;
    if (!operand_map(&P.x, c.x, P.n) || !operand_map(&P.w_gate, c.w_gate, 128) || !operand_map(&P.w_up, c.w_up, 128))
        return cudaErrorInvalidValue;
    P.h = (uint16_t *)c.h.data;
    P.g = (uint16_t *)c.g.data;
    P.u = (uint16_t *)c.u.data;
    P.h_stride = c.h.stride;
    P.g_stride = c.g.stride;
    P.u_stride = c.u.stride;
    P.gelu = c.gelu;
    P.status = c.status;
    P.wait_ns = c.wait_ns;
    P.withhold = c.withhold;
    return launch_cluster(gated_few_kernel, dim3((unsigned)cluster, (unsigned)tiles), cluster, kFewThreads, smem,
                          stream, P);
}

// Shares of n1 units that take c1 and n2 that take c2 (0: none) among the
// pairs: the time of the longest.
static int64_t share_units(PairParams &P, int n1, int64_t c1, int n2, int64_t c2)
{
    P.pairs = n1 + n2 < kPairs ? n1 + n2 : kPairs;
    P.each = n1 / P.pairs;
    P.more = n1 % P.pairs;
    P.less = P.rest = 0;
    int64_t best = -1;
    for (int less = 0; less <= n2; ++less) {
        const int rest = (int)(((int64_t)n2 - (int64_t)less * P.more + P.pairs - P.more - 1) / (P.pairs - P.more));
        if (rest < less)
            break;
        const int64_t a = P.more ? c1 * (P.each + 1) + c2 * less : 0, b = c1 * P.each + c2 * rest;
        const int64_t t = a > b ? a : b;
        if (best < 0 || t < best) {
            best = t;
            P.less = less;
            P.rest = rest;
        }
    }
    return best;
}

static dim3 pair_grid(const PairParams &P) { return dim3((unsigned)(2 * P.pairs)); }

cudaError_t launch_gated_fwd(const GatedFwdCall &c, cudaStream_t stream)
{
    if (c.T <= kFewMostTokens)
        return launch_few(c, stream);
    PairParams P{};
    PairProblem &p = P.p[0];
    if (!operand_map(&p.a[0], c.x, 128) || !operand_map(&p.b[0], c.w_gate, 128) ||
        !operand_map(&p.b[1], c.w_up, 128) || !output_map(&p.out[0], c.h) ||
        (c.g.data && (!output_map(&P.g, c.g) || !output_map(&P.u, c.u))))
        return cudaErrorInvalidValue;
    p.segments = p.halves = p.parts = p.splits = 1;
    p.kblocks = p.per_split = ceil_div(c.H, 64);
    p.tiles_m = ceil_div(c.T, 256);
    p.tiles_n = ceil_div(c.F, 128);
    p.units = p.tiles_m * p.tiles_n;
    share_units(P, p.units, p.kblocks, 0, 0);
    p.rows = (int)c.T;
    p.cols = (int)c.F;
    P.save = c.g.data != nullptr;
    P.gelu = c.gelu;
    P.status = c.status;
    P.wait_ns = c.wait_ns;
    P.withhold = c.withhold;
    return launch_cluster(gated_pair_kernel<true>, pair_grid(P), 2, kPairThreads, kPairSmem, stream, P);
}

// A unit's time in blocks of k: its own, and what its outputs take where those
// are more (BF16; FP32 parts, which are read again).
static int64_t unit_time(const PairProblem &p)
{
    const int out = p.planes ? 8 : 4;
    return p.per_split + (p.per_split < out ? out - p.per_split : 0) + 1;
}

static void split_sum(PairProblem &p, int splits)
{
    const int kblocks = p.kblocks * p.segments * p.parts;
    p.per_split = (kblocks + splits - 1) / splits;
    p.splits = (kblocks + p.per_split - 1) / p.per_split;
    p.planes = p.stack ? 2 * p.splits : p.splits > 1 ? p.splits : 0;
    p.units = p.halves * p.tiles_m * p.tiles_n * p.splits;
}

// Sums over k of few tiles are split, as far as that makes the longest share
// shorter by more than the parts' way through memory takes (a sixteenth of a
// block of k for each tile's part).
static void split_sums(PairProblem &a, PairProblem &b)
{
    int64_t best = -1;
    int sa = 1, sb = 1;
    static constexpr int kSplits[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16};
    for (int i : kSplits)
        for (int k : kSplits) {
            if ((i > 1 && (a.kblocks * a.segments * a.parts < 4 * i || a.halves * a.tiles_m * a.tiles_n >= kPairs)) ||
                (k > 1 && (b.kblocks * b.segments * b.parts < 4 * k || b.halves * b.tiles_m * b.tiles_n >= kPairs)))
                continue;
            split_sum(a, i);
            split_sum(b, k);
            PairParams P;
            const int64_t parts = (a.planes ? a.units : 0) + (b.planes ? b.units : 0);
            const int64_t t = 16 * share_units(P, a.units, unit_time(a), b.units, unit_time(b)) + parts;
            if (best < 0 || t < best) {
                best = t;
                sa = i;
                sb = k;
            }
        }
    split_sum(a, sa);
    split_sum(b, sb);
}

// Tokens up to which the gradients of g and u go into the products as two BF16
// matrices each, the rounded values and the rounded rest (2^-16 of the value).
// One rounding of them costs a result about as much as its own (333 and 8192
// tokens: 2.3e-3 of its norm against 1.7e-3 with exact ones), and more where a
// handful of gradients carries it (2 tokens: 2.7e-3).  A second part takes as
// many products again, which are the time of large calls.  Here the weights'
// bytes are, and for dx both parts lie in one tile of 128 rows.
constexpr int64_t kTwoPartTokens = 64;

struct BwdPlan {
    PairProblem dx, dw;
    int parts;
    size_t gu_bytes, dx_bytes, dw_bytes, x_bytes;
};

// The plan goes by the sizes alone; a thread keeps its last one, as a training
// loop asks for the same again.
static const BwdPlan &plan_bwd(int64_t T, int64_t H, int64_t F)
{
    static thread_local BwdPlan b;
    static thread_local int64_t last[3];
    if (last[0] == T && last[1] == H && last[2] == F)
        return b;
    b = BwdPlan{};
    PairProblem &x = b.dx, &w = b.dw;
    b.parts = w.parts = T <= kTwoPartTokens ? 2 : 1;
    x.parts = 1;
    x.stack = b.parts == 2;
    x.segments = 2;
    x.halves = 1;
    x.a_mn = 0;
    x.b_mn = 1;
    x.kblocks = ceil_div(F, 64);
    x.tiles_m = ceil_div(T, 256);
    x.tiles_n = ceil_div(H, 256);
    x.rows = (int)T;
    x.cols = (int)H;
    w.segments = 1;
    w.halves = 2;
    w.a_mn = w.b_mn = 1;
    w.kblocks = ceil_div(T, 64);
    w.tiles_m = ceil_div(F, 256);
    w.tiles_n = ceil_div(H, 256);
    w.rows = (int)F;
    w.cols = (int)H;
    split_sums(x, w);
    b.gu_bytes = ((size_t)T * F * 2 + 255) & ~(size_t)255;
    b.dx_bytes = ((size_t)x.planes * T * H * 4 + 255) & ~(size_t)255;
    b.dw_bytes = ((size_t)w.planes * 2 * F * H * 4 + 255) & ~(size_t)255;
    b.x_bytes = b.parts == 2 ? ((size_t)T * H * 2 + 255) & ~(size_t)255 : 0;
    last[0] = T;
    last[1] = H;
    last[2] = F;
    return b;
}

size_t gated_bwd_workspace(int64_t T, int64_t H, int64_t F)
{
    const BwdPlan &b = plan_bwd(T, H, F);
    return 2 * b.parts * b.gu_bytes + b.dx_bytes + b.dw_bytes + b.x_bytes;
}

static cudaError_t launch_join(const JoinParams &j, int outputs, cudaStream_t stream)
{
    const uint64_t ctas = (j.vecs + 255) / 256;
    const dim3 grid((unsigned)(ctas < (1 << 20) ? ctas : 1 << 20), (unsigned)outputs);
    return launch_after(j.values < j.planes ? join_kernel<true> : join_kernel<false>, grid, 256, 0, stream, j);
}

cudaError_t launch_gated_bwd(const GatedBwdCall &c, cudaStream_t stream)
{
    const BwdPlan &b = plan_bwd(c.T, c.H, c.F);
    uint8_t *ws = c.workspace;
    Matrix gu[4]; // dg's parts, du's parts
    for (int i = 0; i < 2 * b.parts; ++i)
        gu[i] = {ws + i * b.gu_bytes, c.T, c.F, c.F};
    ws += 2 * b.parts * b.gu_bytes;
    float *part_x = reinterpret_cast<float *>(ws);
    float *part_w = reinterpret_cast<float *>(ws + b.dx_bytes);
    const Matrix x_finite{ws + b.dx_bytes + b.dw_bytes, c.T, c.H, c.H};
    const auto gu_maps = [&](PairProblem &p, int box_rows) {
        bool ok = true;
        for (int i = 0; i < 2 * b.parts; ++i)
            ok = ok && operand_map(&p.a[i], gu[i], box_rows);
        return ok;
    };
    GatedGradParams q{};
    q.dh = (const uint16_t *)c.dh.data;
    q.g = (const uint16_t *)c.g.data;
    q.u = (const uint16_t *)c.u.data;
    q.dh_stride = c.dh.stride;
    q.g_stride = c.g.stride;
    q.u_stride = c.u.stride;
    q.dg = (uint16_t *)gu[0].data;
    q.du = (uint16_t *)gu[b.parts].data;
    q.rest = (int64_t)b.gu_bytes;
    q.nvec = (uint32_t)(c.F / 8);
    q.vecs = (uint64_t)c.T * q.nvec;
    q.gelu = c.gelu;
    if (b.parts == 2 && c.dw_gate.data) {
        q.x = (const uint16_t *)c.x.data;
        q.x_stride = c.x.stride;
        q.x_finite = (uint16_t *)x_finite.data;
        q.x_nvec = (uint32_t)(c.H / 8);
        q.x_vecs = (uint64_t)c.T * q.x_nvec;
    }
    const uint64_t most = q.vecs > q.x_vecs ? q.vecs : q.x_vecs, ctas = (most + kGradGuThreads - 1) / kGradGuThreads;
    const dim3 grid((unsigned)(ctas < (1 << 20) ? ctas : 1 << 20), q.x ? 2 : 1);
    cudaError_t e = launch_after(b.parts == 2 ? gated_grad_kernel<true> : gated_grad_kernel<false>, grid,
                                 kGradGuThreads, 0, stream, q);
    if (e != cudaSuccess)
        return e;
    PairParams P{};
    int n = 0;
    if (c.dx.data) {
        PairProblem &p = P.p[n++] = b.dx;
        const Matrix part{part_x, c.T, c.H, c.H};
        if (!gu_maps(p, p.stack ? 64 : 128) || !operand_map(&p.b[0], c.w_gate, 64) || !operand_map(&p.b[1], c.w_up, 64) ||
            !(p.planes ? parts_map(&p.out[0], part, c.T * c.H, p.planes) : output_map(&p.out[0], c.dx)))
            return cudaErrorInvalidValue;
    }
    if (c.dw_gate.data) {
        PairProblem &p = P.p[n++] = b.dw;
        const Matrix part_g{part_w, c.F, c.H, c.H}, part_u{part_w + c.F * c.H, c.F, c.H, c.H};
        if (!gu_maps(p, 64) || !operand_map(&p.b[0], c.x, 64) ||
            (p.parts == 2 && !operand_map(&p.b[1], x_finite, 64)) ||
            !(p.planes ? parts_map(&p.out[0], part_g, 2 * c.F * c.H, p.planes) &&
                             parts_map(&p.out[1], part_u, 2 * c.F * c.H, p.planes)
                       : output_map(&p.out[0], c.dw_gate) && output_map(&p.out[1], c.dw_up)))
            return cudaErrorInvalidValue;
    }
    share_units(P, P.p[0].units, unit_time(P.p[0]), n > 1 ? P.p[1].units : 0, n > 1 ? unit_time(P.p[1]) : 0);
    P.status = c.status;
    P.wait_ns = c.wait_ns;
    P.withhold = c.withhold;
    e = launch_cluster(gated_pair_kernel<false>, pair_grid(P), 2, kPairThreads, kPairSmem, stream, P);
    if (e == cudaSuccess && c.dx.data && b.dx.planes) {
        JoinParams j{};
        j.part[0] = part_x;
        j.plane = c.T * c.H;
        j.planes = b.dx.planes;
        j.values = b.dx.splits;
        j.out[0] = (uint16_t *)c.dx.data;
        j.stride[0] = c.dx.stride;
        j.nvec = (uint32_t)(c.H / 8);
        j.vecs = (uint64_t)c.T * j.nvec;
        e = launch_join(j, 1, stream);
    }
    if (e == cudaSuccess && c.dw_gate.data && b.dw.planes) {
        JoinParams j{};
        j.part[0] = part_w;
        j.part[1] = part_w + c.F * c.H;
        j.plane = 2 * c.F * c.H;
        j.planes = j.values = b.dw.planes;
        j.out[0] = (uint16_t *)c.dw_gate.data;
        j.out[1] = (uint16_t *)c.dw_up.data;
        j.stride[0] = c.dw_gate.stride;
        j.stride[1] = c.dw_up.stride;
        j.nvec = (uint32_t)(c.H / 8);
        j.vecs = (uint64_t)c.F * j.nvec;
        e = launch_join(j, 2, stream);
    }
    return e;
}

} // namespace cake
