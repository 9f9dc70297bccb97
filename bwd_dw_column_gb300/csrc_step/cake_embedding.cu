// cake_embedding.cu -- embedding lookup and its gradient by sorted tokens,
// for sm_103a.
//
//   y_t = bf16(scale * table[ids_t])
//   dtable_v = [dtable_v +] scale * sum over t with ids_t = v of dy_t
//
// The gradient: (1) the tokens are sorted by id with a stable radix sort, so
// that the rows of one id follow one another in ascending t; (2) CTAs take
// windows of sorted positions and slices of the columns, and sum each run of
// equal ids in FP32; a run that spreads far over several windows leaves a
// partial sum per window, and (3) those are joined in window order.  Rows
// without a token are zeroed by further CTAs of step 2.  All orders depend on
// the ids alone, and every row of dtable has one writer.
//
// HBM bounds the lookup and, where there are many tokens or rows, the gradient
// (GB300: T = 65536, H = 5120 lookup 140 us; the whole gradient of 131072 x 2048
// from 8192 tokens 159 us, 7.0 TB/s; 65536 tokens added at H = 4096 179 to 185
// us, of which the sort is 20 us and the join 9 us).
#include <mutex>

#include "../csrc/cake_device.cuh"
#include "cake_step_launch.h"

namespace cake {

// A word for each code, so that an id outside its table (whose outputs are
// defined) never hides a wait that ran out (whose outputs are not).
__device__ int g_step_status[2]; // timeouts, ids outside their table

constexpr int kStatusInvalid = 1; // == CAKE_ERR_INVALID
constexpr int kStatusTimeout = 5; // == CAKE_ERR_TIMEOUT

__device__ __forceinline__ int64_t load_id(const void *ids, int i64, uint32_t t)
{
    return i64 ? __ldg(static_cast<const long long *>(ids) + t) : (int64_t)__ldg(static_cast<const int *>(ids) + t);
}

// ------------------------------------------------------------------ forward

constexpr int kEmbedThreads = 256;

// A warp takes 128 vectors (2 KB of output) of a row.
template <bool F32>
__global__ void __launch_bounds__(kEmbedThreads) embed_fwd_kernel(const __grid_constant__ EmbedFwdParams p)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const uint32_t per_row = (uint32_t)((p.nvec + 127) / 128);
    const uint64_t items = (uint64_t)p.tokens * per_row;
    const uint64_t warps = (uint64_t)gridDim.x * (kEmbedThreads / 32);
    for (uint64_t w = (uint64_t)blockIdx.x * (kEmbedThreads / 32) + (threadIdx.x >> 5); w < items; w += warps) {
        const uint32_t t = (uint32_t)(w / per_row);
        const int v0 = (int)(w - (uint64_t)t * per_row) * 128 + lane;
        const int64_t id = load_id(p.ids, p.ids_i64, t);
        const bool live = id >= 0 && id < p.vocab;
        if (id >= p.vocab && v0 == 0)
            set_status(p.status + 1, kStatusInvalid);
        uint4 raw[4][F32 ? 2 : 1];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int v = v0 + 32 * k;
#pragma unroll
            for (int i = 0; i < (F32 ? 2 : 1); ++i)
                raw[k][i] = make_uint4(0, 0, 0, 0);
            if (live && v < p.nvec) {
                if (F32) {
                    const uint4 *s = reinterpret_cast<const uint4 *>(static_cast<const float *>(p.table) +
                                                                     id * p.table_stride) + 2 * v;
                    raw[k][0] = __ldg(s);
                    raw[k][F32 ? 1 : 0] = __ldg(s + 1);
                } else {
                    raw[k][0] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.table) +
                                                                      id * p.table_stride) + v);
                }
            }
        }
        uint4 *y = reinterpret_cast<uint4 *>(p.y + (int64_t)t * p.y_stride);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float f[8];
            if (F32) {
                const uint4 a = raw[k][0], b = raw[k][F32 ? 1 : 0];
                f[0] = __uint_as_float(a.x), f[1] = __uint_as_float(a.y), f[2] = __uint_as_float(a.z);
                f[3] = __uint_as_float(a.w), f[4] = __uint_as_float(b.x), f[5] = __uint_as_float(b.y);
                f[6] = __uint_as_float(b.z), f[7] = __uint_as_float(b.w);
            } else {
                unpack8(raw[k][0], f);
            }
#pragma unroll
            for (int q = 0; q < 8; ++q)
                f[q] = live ? __fmul_rn(f[q], p.scale) : 0.f;
            if (v0 + 32 * k < p.nvec)
                __stcs(y + v0 + 32 * k, pack8(f));
        }
    }
}

// --------------------------------------------------------------------- sort
//
// Least-significant-digit radix sort.  A tile is a CTA's contiguous keys.
// Pass p's histogram of the digits per tile is complete before the pass
// starts: the count kernel makes the first, and each pass, as it places a
// key, counts its next digit for the tile it lands in (integer atomics: the
// counts do not depend on their order).  A tile's first place for a digit is
// then the count of all smaller digits plus that of the same digit in
// earlier tiles, which every CTA sums for itself.

__device__ __forceinline__ uint64_t make_pair(const SortParams &p, uint32_t t)
{
    const int64_t id = load_id(p.ids, p.ids_i64, t);
    const bool live = id >= 0 && id < (int64_t)p.vocab && id != p.padding_idx;
    const uint32_t key = live ? (uint32_t)id : p.vocab; // tokens without a gradient sort last
    if (id >= (int64_t)p.vocab)
        set_status(p.status + 1, kStatusInvalid);
    return ((uint64_t)key << 32) | t;
}

// Sets the keys' bits in the bitmap of ids with a token: one lane for the equal
// keys of a step, and none for a bit that is set already (a common id's).
template <int N>
__device__ __forceinline__ void mark_present(const SortParams &p, const uint32_t (&key)[N])
{
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const bool one = (__match_any_sync(0xffffffffu, key[j]) & ((1u << (threadIdx.x & 31)) - 1)) == 0;
        uint32_t *w = p.present + (key[j] >> 5);
        const uint32_t bit = 1u << (key[j] & 31);
        if (one && key[j] < p.vocab && !(__ldcg(w) & bit))
            atomicOr(w, bit);
    }
}

// Ranks a warp's 32 x N keys among those of the warp with the same digit, in
// order (key j of lane l is the warp's key 32 j + l), and leaves the counts of
// its digits in cnt, which is zero before.  Equal digits of the 32 keys of a
// step find each other by a ballot per bit.  Keys that are not `in` count for
// nothing.
template <int N>
__device__ __forceinline__ void rank_keys(const uint64_t (&key)[N], const bool (&in)[N], int shift, int bits,
                                          uint32_t *cnt, uint32_t (&rank)[N])
{
    const int lane = threadIdx.x & 31;
    uint32_t same[N], dig[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        dig[j] = (uint32_t)(key[j] >> (32 + shift)) & ((1u << bits) - 1);
        same[j] = __ballot_sync(0xffffffffu, in[j]);
    }
    for (int b = 0; b < bits; ++b)
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const bool one = (dig[j] >> b) & 1u;
            const uint32_t ones = __ballot_sync(0xffffffffu, one);
            same[j] &= one ? ones : ~ones;
        }
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const uint32_t below = __popc(same[j] & ((1u << lane) - 1));
        uint32_t old = 0;
        if (in[j])
            old = cnt[dig[j]];
        rank[j] = old + below;
        __syncwarp();
        if (in[j] && below == 0)
            cnt[dig[j]] = old + __popc(same[j]);
        __syncwarp();
    }
}

// One cluster sorts up to 8192 keys a CTA (PER a thread) in shared memory, in
// one launch: in every pass each CTA ranks its keys, tells the others its
// digits' counts, and puts its keys into the shared memory of the CTA where
// they belong.  Latencies bound it, and an SM's rate of scattered stores and
// atomics, a cycle or two each; so the keys are spread over as many CTAs as a
// cluster may have (GB300, ncu: 8192 keys 14 us on 8 CTAs, 48 us on one; 65536
// keys 21 us on 16 CTAs, 46 us on 8; a launch per pass 44 and 36 us).
//
// The bitmap is complete after the first pass's barrier; a flag says so and
// the dependent kernel may start then, to zero rows while the sort goes on.
constexpr int kClusterWarps = kClusterThreads / 32;

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, uint64_t v)
{
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

template <int PER>
struct ClusterSortSmem {
    uint64_t keys[2][PER * kClusterThreads];
    uint32_t cnt[kClusterWarps][1 << kSortMaxBits];
    uint32_t tot[2][kMaxSortCluster][1 << kSortMaxBits]; // by pass parity: every CTA's counts
    uint32_t base[1 << kSortMaxBits];
    uint32_t scan[8];
};

template <int PER>
__global__ void __launch_bounds__(kClusterThreads, 1) embed_cluster_sort_kernel(const __grid_constant__ SortParams p)
{
    constexpr uint32_t kKeys = PER * kClusterThreads; // of a CTA
    extern __shared__ __align__(16) uint8_t smem_raw[];
    ClusterSortSmem<PER> &m = *reinterpret_cast<ClusterSortSmem<PER> *>(smem_raw);
    const int bins = 1 << p.bits, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t C = gridDim.x, rank_c = cluster_ctarank();
    pdl_wait();
    const uint32_t first = rank_c * kKeys + warp * 32 * PER + lane; // key j: first + 32 j
    if (p.present && p.zero_present)
        for (uint32_t i = blockIdx.x * kClusterThreads + threadIdx.x; i < (p.vocab + 31) / 32;
             i += C * kClusterThreads)
            p.present[i] = 0;
    if (rank_c == 0 && threadIdx.x == 0) {
        p.ready[0] = 0;
        p.ready[1] = 0; // the sums' count of cut runs
    }
    const bool mark = p.present != nullptr;
    uint64_t key[PER];
    {
        uint32_t k32[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const uint32_t t = first + 32 * j;
            key[j] = t < p.tokens ? make_pair(p, t) : ~0ull; // past the end: sorts last
            k32[j] = (uint32_t)(key[j] >> 32);
        }
        cluster_sync_all(); // the bitmap is zero
        if (mark)
            mark_present<PER>(p, k32);
    }
    for (int pass = 0; pass < p.passes; ++pass) {
        const int shift = pass * p.bits;
        for (int i = lane; i < bins; i += 32)
            m.cnt[warp][i] = 0;
        __syncwarp();
        bool in[PER];
        uint32_t rank[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j)
            in[j] = true;
        rank_keys<PER>(key, in, shift, p.bits, m.cnt[warp], rank);
        __syncthreads();
        // each warp's first place within the CTA's keys of a digit, and their count to every CTA
        if (threadIdx.x < bins) {
            uint32_t at = 0;
#pragma unroll 8
            for (int w = 0; w < kClusterWarps; ++w) {
                const uint32_t c = m.cnt[w][threadIdx.x];
                m.cnt[w][threadIdx.x] = at;
                at += c;
            }
            const uint32_t to = smem_addr(&m.tot[pass & 1][rank_c][threadIdx.x]);
            for (uint32_t c = 0; c < C; ++c)
                st_cluster_u32(map_to_rank(to, c), at);
        }
        cluster_sync_all();
        if (pass == 0 && rank_c == 0 && threadIdx.x == 0) {
            __threadfence();
            atomicExch(p.ready, 1u);
        }
        // a digit's first place of this CTA: all smaller digits, and its own in earlier CTAs
        uint32_t all = 0, before = 0;
        if (threadIdx.x < bins)
            for (uint32_t c = 0; c < C; ++c) {
                const uint32_t v = m.tot[pass & 1][c][threadIdx.x];
                all += v;
                before += c < rank_c ? v : 0;
            }
        if (warp < 8) {
            uint32_t incl = all;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
                incl += lane >= o ? v : 0;
            }
            if (lane == 31)
                m.scan[warp] = incl;
            before += incl - all;
        }
        __syncthreads();
        // only now: a launch that starts earlier could meet the flag and the bitmap
        // of the workspace's last call
        if (pass == 0)
            pdl_launch_dependents();
        if (threadIdx.x < bins) {
            for (int w = 0; w < warp; ++w)
                before += m.scan[w];
            m.base[threadIdx.x] = before;
        }
        __syncthreads();
        // to the CTA and place where it belongs
        const uint32_t out = smem_addr(m.keys[pass & 1]);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const uint32_t d = (uint32_t)(key[j] >> (32 + shift)) & (bins - 1);
            const uint32_t at = m.base[d] + m.cnt[warp][d] + rank[j];
            st_cluster_u64(map_to_rank(out + 8 * (at % kKeys), at / kKeys), key[j]);
        }
        cluster_sync_all();
#pragma unroll
        for (int j = 0; j < PER; ++j)
            key[j] = m.keys[pass & 1][warp * 32 * PER + 32 * j + lane];
    }
#pragma unroll
    for (int j = 0; j < PER; ++j)
        if (first + 32 * j < p.tokens)
            p.pairs[0][first + 32 * j] = key[j];
}

__global__ void __launch_bounds__(kSortThreads) embed_count_kernel(const __grid_constant__ SortParams p)
{
    __shared__ uint32_t h[1 << kSortMaxBits];
    const int bins = 1 << p.bits;
    for (int i = threadIdx.x; i < bins; i += kSortThreads)
        h[i] = 0;
    __syncthreads();
    const uint32_t lo = blockIdx.x * p.tile_keys, hi = min(p.tokens, lo + p.tile_keys);
    for (uint32_t t0 = lo; t0 < hi; t0 += kSortBlock) {
        uint32_t key[kSortPerThread];
#pragma unroll
        for (int j = 0; j < kSortPerThread; ++j) {
            const uint32_t t = t0 + j * kSortThreads + threadIdx.x;
            key[j] = t < hi ? (uint32_t)(make_pair(p, t) >> 32) : 0xffffffffu;
        }
        if (p.present)
            mark_present<kSortPerThread>(p, key);
#pragma unroll
        for (int j = 0; j < kSortPerThread; ++j)
            if (key[j] != 0xffffffffu)
                atomicAdd(&h[key[j] & (bins - 1)], 1u);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < bins; i += kSortThreads)
        p.hist[(size_t)blockIdx.x * bins + i] = h[i];
}

__global__ void __launch_bounds__(kSortThreads)
    embed_place_kernel(const __grid_constant__ SortParams p, int pass, const uint64_t *src, uint64_t *dst)
{
    constexpr int kWarps = kSortThreads / 32;
    __shared__ uint32_t base[1 << kSortMaxBits];           // next place of each digit for this tile
    __shared__ uint32_t cnt[kWarps][1 << kSortMaxBits];    // each warp's counts, then its first place
    __shared__ uint32_t scan[kSortThreads];
    const int bins = 1 << p.bits, shift = pass * p.bits;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t *hist = p.hist + (size_t)pass * p.tiles * bins;
    uint32_t *next_hist = pass + 1 < p.passes ? p.hist + (size_t)(pass + 1) * p.tiles * bins : nullptr;

    // Thread (g, d) sums digit d over every (kSortThreads / bins)-th tile, then
    // thread d < bins over the g.
    const int groups = kSortThreads / bins, g = threadIdx.x / bins, gd = threadIdx.x - g * bins;
    {
        uint32_t part = 0, part_before = 0;
#pragma unroll 8
        for (int t = g; t < p.tiles; t += groups) {
            const uint32_t c = __ldcg(hist + (size_t)t * bins + gd);
            part += c;
            part_before += t < (int)blockIdx.x ? c : 0;
        }
        cnt[0][threadIdx.x] = part; // (kWarps rows of 256: two of them serve here)
        cnt[1][threadIdx.x] = part_before;
    }
    __syncthreads();
    uint32_t before = 0, all = 0;
    const int d = threadIdx.x;
    if (d < bins)
        for (int k = 0; k < groups; ++k) {
            all += cnt[0][k * bins + d];
            before += cnt[1][k * bins + d];
        }
    scan[d] = all;
    __syncthreads();
    for (int o = 1; o < kSortThreads; o <<= 1) {
        const uint32_t v = d >= o ? scan[d - o] : 0;
        __syncthreads();
        scan[d] += v;
        __syncthreads();
    }
    if (d < bins)
        base[d] = scan[d] - all + before;

    __syncthreads();
    const uint32_t lo = blockIdx.x * p.tile_keys, hi = min(p.tokens, lo + p.tile_keys);
    for (uint32_t b0 = lo; b0 < hi; b0 += kSortBlock) {
        for (int i = threadIdx.x; i < kWarps * bins; i += kSortThreads)
            cnt[i / bins][i % bins] = 0;
        __syncthreads();
        // a warp's keys are contiguous and taken in order
        uint64_t key[kSortPerThread];
        uint32_t rank[kSortPerThread];
        bool in[kSortPerThread];
#pragma unroll
        for (int j = 0; j < kSortPerThread; ++j) {
            const uint32_t t = b0 + warp * 32 * kSortPerThread + j * 32 + lane;
            in[j] = t < hi;
            key[j] = in[j] ? (src ? __ldcg(src + t) : make_pair(p, t)) : ~0ull;
        }
        rank_keys<kSortPerThread>(key, in, shift, p.bits, cnt[warp], rank);
        __syncthreads();
        if (d < bins) {
            uint32_t at = base[d];
            for (int w = 0; w < kWarps; ++w) {
                const uint32_t c = cnt[w][d];
                cnt[w][d] = at;
                at += c;
            }
            base[d] = at;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kSortPerThread; ++j) {
            const uint32_t t = b0 + warp * 32 * kSortPerThread + j * 32 + lane;
            if (t < hi) {
                const uint32_t k32 = (uint32_t)(key[j] >> 32);
                const uint32_t at = cnt[warp][(k32 >> shift) & (bins - 1)] + rank[j];
                dst[at] = key[j];
                if (next_hist)
                    atomicAdd(next_hist + (size_t)(at / p.tile_keys) * bins + ((k32 >> (shift + p.bits)) & (bins - 1)),
                              1u);
            }
        }
        __syncthreads();
    }
}

// ----------------------------------------------------------------- segments
//
// CTA (window w, slice s) sums columns of the rows whose sorted positions are
// in [w * window, (w + 1) * window).  Runs that end within `overrun` positions
// after their window (at most a window) are finished by the window in which
// they start.  A run that goes further is cut at the window boundaries: its
// first window leaves a "trailing" partial and enters itself in the list of cut
// runs, the windows that it fills leave a partial each, and the last a
// "leading" one.
constexpr uint32_t kMostOverrun = 32;
// meta[w][0]
constexpr uint32_t kMetaLead = 1;   // the window starts with a piece of an earlier window's run: partial 0
constexpr uint32_t kMetaLeadOn = 2; // ... that goes on in the next window
constexpr uint32_t kMetaTrail = 4;  // the window's last run goes on in the next window: partial 1

// Eight values of row id of dtable as they were before.
__device__ __forceinline__ void load_row8(const SegmentParams &p, uint32_t id, int col, uint4 (&a)[2])
{
    if (p.dtable_f32) {
        const uint4 *o = reinterpret_cast<const uint4 *>(static_cast<const float *>(p.dtable) +
                                                         (int64_t)id * p.dtable_stride + col);
        a[0] = o[0];
        a[1] = o[1];
    } else {
        a[0] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.dtable) +
                                                (int64_t)id * p.dtable_stride + col);
    }
}

// Row id of dtable: scale * s [+ what it was].
template <bool ACC>
__device__ __forceinline__ void store_row8(const SegmentParams &p, uint32_t id, int col, const float (&s)[8],
                                           const uint4 (&was)[2])
{
    float v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
        v[q] = __fmul_rn(s[q], p.scale);
    if (p.dtable_f32) {
        if (ACC) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                v[q] = __fadd_rn(v[q], __uint_as_float(word(was[q >> 2], q & 3)));
        }
        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.dtable) + (int64_t)id * p.dtable_stride + col);
        o[0] = make_float4(v[0], v[1], v[2], v[3]);
        o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        if (ACC) {
            float a[8];
            unpack8(was[0], a);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                v[q] = __fadd_rn(v[q], a[q]);
        }
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.dtable) + (int64_t)id * p.dtable_stride + col) = pack8(v);
    }
}

// Zeroes the rows of dtable whose id has no token: a warp takes as many rows as
// make 8 KB, 32 at most.  (Warps that come and go: 165 us for 131072 x 2048 FP32
// values, against 174 and 216 us with 16 and 6 CTAs an SM in a loop.)
__device__ void fill_rows(const SegmentParams &p, uint32_t part, uint32_t parts)
{
    const uint32_t lane = threadIdx.x & 31, R = (uint32_t)p.fill_rows;
    const uint64_t step = (uint64_t)parts * (blockDim.x / 32) * R;
    const uint32_t vecs = p.dtable_f32 ? 2 * p.nvec : p.nvec;
    const int64_t stride = p.dtable_stride * (p.dtable_f32 ? 4 : 2);
    for (uint64_t v0 = ((uint64_t)part * (blockDim.x / 32) + (threadIdx.x >> 5)) * R; v0 < p.vocab; v0 += step) {
        const uint32_t has = __ldcg(p.present + (v0 >> 5)) >> (v0 & 31); // (R rows lie in one word)
        const uint32_t n = min((uint64_t)R, p.vocab - v0);
        uint8_t *row0 = static_cast<uint8_t *>(p.dtable) + (int64_t)v0 * stride;
        if (vecs >= 32) {
            for (uint32_t r = 0; r < n; ++r)
                if (!((has >> r) & 1u))
                    for (uint32_t i = lane; i < vecs; i += 32)
                        __stcs(reinterpret_cast<uint4 *>(row0 + r * stride) + i, make_uint4(0, 0, 0, 0));
        } else {
            for (uint32_t i = lane; i < n * vecs; i += 32) {
                const uint32_t r = i / vecs;
                if (!((has >> r) & 1u))
                    __stcs(reinterpret_cast<uint4 *>(row0 + r * stride) + (i - r * vecs), make_uint4(0, 0, 0, 0));
            }
        }
    }
}

// ACC: adds to dtable.  The rows that it adds to are loaded together with the
// rows of dy, half as many at a time (GB300, T = 65536, H = 4096: a load at
// each run's end instead took 172 us).
template <bool ACC>
__global__ void __launch_bounds__(kSegMaxThreads) embed_segment_kernel(const __grid_constant__ SegmentParams p)
{
    constexpr int kSegBatch = ACC ? 4 : 8; // rows in flight
    if (blockIdx.x < (uint32_t)p.fill_ctas) {
        if (p.ready) {
            // the bitmap is complete, the sort perhaps not yet; one thread waits and
            // answers for the CTA, so that no row is left out without a report
            int late = 0;
            if (threadIdx.x == 0) {
                const uint64_t t0 = globaltimer_ns();
                while (ld_acquire_gpu(p.ready) == 0 && !late)
                    late = globaltimer_ns() - t0 > p.wait_ns;
                if (late)
                    set_status(p.status, kStatusTimeout);
            }
            if (__syncthreads_or(late))
                return;
        } else {
            pdl_wait();
        }
        fill_rows(p, blockIdx.x, p.fill_ctas);
        return;
    }
    pdl_wait();
    const uint32_t block = blockIdx.x - (uint32_t)p.fill_ctas;
    __shared__ uint32_t ids[kSegMaxWindow + kMostOverrun + 2], tok[kSegMaxWindow + kMostOverrun + 2];
    __shared__ int limits[2];
    const uint32_t w = block / p.slices, slice = block - w * p.slices;
    const uint32_t lo = w * p.window;
    const uint32_t W = min((uint32_t)p.window, p.tokens - lo); // positions of this window
    const uint32_t overrun = min((uint32_t)p.window, kMostOverrun);
    const uint32_t ext = min(p.tokens - lo, (uint32_t)p.window + overrun + 1); // and those looked at
    // ids[1 + i], tok[1 + i]: position lo + i; ids[0]: the position before
    for (uint32_t i = threadIdx.x; i < ext; i += blockDim.x) {
        const uint64_t pr = __ldcg(p.pairs + lo + i);
        ids[1 + i] = (uint32_t)(pr >> 32);
        tok[1 + i] = (uint32_t)pr;
    }
    if (threadIdx.x == 0) {
        ids[0] = lo > 0 ? (uint32_t)(__ldcg(p.pairs + lo - 1) >> 32) : 0xffffffffu;
        limits[0] = (int)W;
        limits[1] = (int)ext;
    }
    __syncthreads();
    // the leading run: positions equal to the one before the window
    // (limits[0]: its length within W); the trailing run's end (limits[1])
    for (uint32_t i = threadIdx.x; i < ext; i += blockDim.x) {
        if (i < W && ids[1 + i] != ids[0])
            atomicMin(&limits[0], (int)i);
        if (i >= W && ids[1 + i] != ids[W])
            atomicMin(&limits[1], (int)i);
    }
    __syncthreads();
    const uint32_t lead = lo > 0 ? (uint32_t)limits[0] : 0;
    uint32_t end = W; // one past the last position summed here
    uint32_t flags = 0;
    // the window's last run goes on by this many positions
    const uint32_t over = (uint32_t)limits[1] - W;
    const bool goes_on = W == (uint32_t)p.window && over > 0;
    uint32_t first = lead, lead_end = lead;
    if (lead == W) {
        // one run of an earlier window fills this one; the window before has
        // finished it if it ends within the overrun
        if (W > overrun || goes_on) {
            first = 0;
            flags = kMetaLead;
            if (goes_on && over <= overrun)
                end = W + over;
            else if (goes_on)
                flags |= kMetaLeadOn;
            lead_end = end;
        }
    } else {
        if (lead > overrun) {
            first = 0;
            flags = kMetaLead;
        }
        if (goes_on && over <= overrun)
            end = W + over;
        else if (goes_on)
            flags |= kMetaTrail;
    }
    if (slice == 0 && threadIdx.x == 0) {
        p.meta[2 * w] = flags;
        p.meta[2 * w + 1] = ids[W];
        if ((flags & kMetaTrail) && ids[W] < p.vocab)
            p.cut[atomicAdd(p.cuts, 1u)] = w; // (their order changes no result)
    }

    const int col = 8 * ((int)(slice * blockDim.x) + (int)threadIdx.x);
    if (col >= 8 * p.nvec)
        return;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    float *lead_part = p.partials + ((size_t)w * 2) * 8 * p.nvec + col, *trail_part = lead_part + 8 * p.nvec;
    for (uint32_t b = first; b < end; b += kSegBatch) {
        uint4 r[kSegBatch], was[kSegBatch][2];
#pragma unroll
        for (int k = 0; k < kSegBatch; ++k) {
            r[k] = was[k][0] = was[k][1] = make_uint4(0, 0, 0, 0);
            const uint32_t i = b + k;
            if (i < end && ids[1 + i] < p.vocab) {
                r[k] = __ldcs(reinterpret_cast<const uint4 *>(p.dy + (int64_t)tok[1 + i] * p.dy_stride + col));
                if (ACC && (i + 1 == end || ids[2 + i] != ids[1 + i]))
                    load_row8(p, ids[1 + i], col, was[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < kSegBatch; ++k) {
            const uint32_t i = b + k;
            if (i < end) {
                const uint32_t id = ids[1 + i];
                if (id >= p.vocab) // only tokens without a gradient from here on
                    return;
                float f[8];
                unpack8(r[k], f);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    s[q] = __fadd_rn(s[q], f[q]);
                const bool last = i + 1 == end || ids[2 + i] != id;
                if (last) {
                    const bool is_lead = (flags & kMetaLead) && i < lead_end;
                    const bool is_trail = (flags & kMetaTrail) && i + 1 == end;
                    if (is_lead || is_trail) {
                        float4 *o = reinterpret_cast<float4 *>(is_lead ? lead_part : trail_part);
                        o[0] = make_float4(s[0], s[1], s[2], s[3]);
                        o[1] = make_float4(s[4], s[5], s[6], s[7]);
                    } else {
                        store_row8<ACC>(p, id, col, s, was[k]);
                    }
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        s[q] = 0.f;
                }
            }
        }
    }
}

// Adds the first n of N pieces, `step` apart, in order.
template <int N>
__device__ __forceinline__ void add_pieces(const float4 *piece, size_t step, uint32_t n, float (&s)[8])
{
    float4 v[N][2];
#pragma unroll
    for (int k = 0; k < N; ++k)
        if ((uint32_t)k < n) {
            v[k][0] = __ldcg(piece + (size_t)k * step);
            v[k][1] = __ldcg(piece + (size_t)k * step + 1);
        }
#pragma unroll
    for (int k = 0; k < N; ++k)
        if ((uint32_t)k < n) {
            const float f[8] = {v[k][0].x, v[k][0].y, v[k][0].z, v[k][0].w,
                                v[k][1].x, v[k][1].y, v[k][1].z, v[k][1].w};
#pragma unroll
            for (int q = 0; q < 8; ++q)
                s[q] = __fadd_rn(s[q], f[q]);
        }
}

// Joins the partials of the cut runs: a CTA takes an eighth of a run's columns
// (64 to 1024 of them), its G groups of L threads every G-th of the run's pieces
// each, and the groups' sums are added in their order.  A common id's run has
// hundreds of pieces where windows are short (GB300, ncu, T = 65536 with
// frequencies of 1/k: H = 64 7 us, H = 512 11 us; with the pieces of a run one
// after another 21 and 25 us).
constexpr int kJoinThreads = 256;
constexpr int kJoinCtas = 152 * 4;

__global__ void __launch_bounds__(kJoinThreads, 4) embed_join_kernel(const __grid_constant__ SegmentParams p)
{
    __shared__ int last;
    __shared__ __align__(16) float part[8 * kJoinThreads]; // [G][8 L]
    pdl_wait();
    const uint32_t L = (uint32_t)p.join_lanes, G = kJoinThreads / L, blocks = ((uint32_t)p.nvec + L - 1) / L;
    const uint64_t items = (uint64_t)__ldcg(p.cuts) * blocks;
    const int H = 8 * p.nvec;
    const uint32_t g = threadIdx.x / L, c = threadIdx.x - g * L;
    for (uint64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const uint32_t run = (uint32_t)(item / blocks), block = (uint32_t)(item - (uint64_t)run * blocks);
        const uint32_t w = __ldcg(p.cut + run);
        const uint32_t id = __ldcg(p.meta + 2 * w + 1);
        // the run's pieces are those of windows w + 1 .. w + n
        uint32_t n = 0;
        for (;; n += 4 * kJoinThreads) {
            if (threadIdx.x == 0)
                last = 4 * kJoinThreads;
            __syncthreads();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t i = q * kJoinThreads + threadIdx.x, u = w + 1 + n + i;
                if (u >= (uint32_t)p.windows || !(__ldcg(p.meta + 2 * u) & kMetaLeadOn))
                    atomicMin(&last, (int)i);
            }
            __syncthreads();
            const int l = last;
            __syncthreads();
            if (l < 4 * kJoinThreads) {
                n += l + 1;
                break;
            }
        }
        const int col = 8 * (int)(L * block + c);
        uint4 was[2] = {};
        if (g == 0 && col < H && p.accumulate)
            load_row8(p, id, col, was);
        float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (col < H) {
            const size_t step = (size_t)2 * H / 4; // from window to window
            if (g == 0) // the piece of window w itself
                add_pieces<1>(reinterpret_cast<const float4 *>(p.partials + ((size_t)w * 2 + 1) * H + col), step, 1, s);
            const float4 *piece =
                reinterpret_cast<const float4 *>(p.partials + (size_t)(w + 1) * 2 * H + col) + (size_t)g * step;
            const uint32_t m = g < n ? (n - g + G - 1) / G : 0;
            // four at a time and four CTAs an SM (H = 512: 52 us in all, 56 with eight
            // at a time, which leave room for two CTAs)
            for (uint32_t u = 0; u < m; u += 4)
                add_pieces<4>(piece + (size_t)u * G * step, G * step, min(4u, m - u), s);
        }
        float4 *o = reinterpret_cast<float4 *>(part + 8 * threadIdx.x);
        o[0] = make_float4(s[0], s[1], s[2], s[3]);
        o[1] = make_float4(s[4], s[5], s[6], s[7]);
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < 8 * L; i += kJoinThreads) {
            float t = part[i];
            for (uint32_t k = 1; k < min(n, G); ++k)
                t = __fadd_rn(t, part[8 * L * k + i]);
            part[i] = t;
        }
        __syncthreads();
        if (g == 0 && col < H) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                s[q] = part[8 * c + q];
            if (p.accumulate)
                store_row8<true>(p, id, col, s, was);
            else
                store_row8<false>(p, id, col, s, was);
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ launch

// A launch may start while the one before it in the stream drains; the kernels
// wait for its end before they touch memory.
template <class P>
static cudaError_t launch_dependent(void (*kern)(P), const P &p, int ctas, int threads, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_embed_fwd(const EmbedFwdParams &p, cudaStream_t stream)
{
    const uint64_t items = (uint64_t)p.tokens * ((p.nvec + 127) / 128);
    // an item a warp: CTAs that come and go keep more rows on their way than
    // resident ones in a loop (GB300, T = 65536, H = 5120: 144 against 164 us)
    const uint64_t want = (items + kEmbedThreads / 32 - 1) / (kEmbedThreads / 32);
    const int ctas = (int)(want < (1u << 30) ? want : (1u << 30));
    return launch_dependent(p.table_f32 ? embed_fwd_kernel<true> : embed_fwd_kernel<false>, p, ctas, kEmbedThreads,
                            stream);
}

cudaError_t ensure_smem_attr(const void *kernel, size_t smem);

template <int PER>
static cudaError_t launch_cluster_sort(const SortParams &p, int ctas, cudaStream_t stream)
{
    const void *kern = (const void *)embed_cluster_sort_kernel<PER>;
    cudaError_t e = ensure_smem_attr(kern, sizeof(ClusterSortSmem<PER>));
    if (e == cudaSuccess && ctas > 8)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kClusterThreads);
    cfg.dynamicSmemBytes = sizeof(ClusterSortSmem<PER>);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, embed_cluster_sort_kernel<PER>, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_embed_cluster_sort(const SortParams &p, int ctas, cudaStream_t stream)
{
    const uint32_t per = (p.tokens + ctas * kClusterThreads - 1) / (ctas * kClusterThreads);
    return per <= 1   ? launch_cluster_sort<1>(p, ctas, stream)
           : per <= 2 ? launch_cluster_sort<2>(p, ctas, stream)
           : per <= 4 ? launch_cluster_sort<4>(p, ctas, stream)
           : per <= 8 ? launch_cluster_sort<8>(p, ctas, stream)
                      : cudaErrorInvalidValue;
}

cudaError_t launch_embed_sort(const SortParams &p, uint64_t **sorted, cudaStream_t stream)
{
    embed_count_kernel<<<p.tiles, kSortThreads, 0, stream>>>(p);
    const uint64_t *src = nullptr;
    for (int pass = 0; pass < p.passes; ++pass) {
        uint64_t *dst = p.pairs[pass & 1];
        embed_place_kernel<<<p.tiles, kSortThreads, 0, stream>>>(p, pass, src, dst);
        src = dst;
    }
    *sorted = p.pairs[(p.passes - 1) & 1];
    return cudaGetLastError();
}

cudaError_t launch_embed_segments(const SegmentParams &p, cudaStream_t stream)
{
    return launch_dependent(p.accumulate ? embed_segment_kernel<true> : embed_segment_kernel<false>, p,
                            p.windows * p.slices + p.fill_ctas, p.threads, stream);
}

cudaError_t launch_embed_join(const SegmentParams &p, cudaStream_t stream)
{
    SegmentParams q = p;
    q.join_lanes = 8;
    while (q.join_lanes < 128 && 8 * q.join_lanes < p.nvec)
        q.join_lanes *= 2;
    const uint64_t most = (uint64_t)p.windows * ((p.nvec + q.join_lanes - 1) / q.join_lanes);
    return launch_dependent(embed_join_kernel, q, most < kJoinCtas ? (int)most : kJoinCtas, kJoinThreads, stream);
}

// Device address of the status word, looked up once per device.
cudaError_t step_status_ptr(int **out)
{
    static std::mutex mu;
    static int *addr[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 64)
        return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> g(mu);
    if (!addr[dev]) {
        e = cudaGetSymbolAddress((void **)&addr[dev], g_step_status);
        if (e != cudaSuccess)
            return e;
    }
    *out = addr[dev];
    return cudaSuccess;
}

cudaError_t step_status(int *code, int clear)
{
    int words[2] = {};
    cudaError_t e = cudaMemcpyFromSymbol(words, g_step_status, sizeof(words));
    if (e == cudaSuccess && clear) {
        const int zero[2] = {};
        e = cudaMemcpyToSymbol(g_step_status, zero, sizeof(zero));
    }
    *code = words[0] ? words[0] : words[1];
    return e;
}

} // namespace cake
