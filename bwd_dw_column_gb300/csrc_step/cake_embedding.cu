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
#include <mutex>

#include "../csrc/cake_device.cuh"
#include "cake_step_launch.h"

namespace cake {

__device__ int g_step_status;

constexpr int kStatusInvalid = 1; // == CAKE_ERR_INVALID

__device__ __forceinline__ int64_t load_id(const void *ids, int i64, uint32_t t)
{
    return i64 ? __ldg(static_cast<const long long *>(ids) + t) : (int64_t)__ldg(static_cast<const int *>(ids) + t);
}

// ------------------------------------------------------------------ forward

constexpr int kEmbedThreads = 256;

// One warp per 32 x 4 vectors of a row.
__global__ void __launch_bounds__(kEmbedThreads) embed_fwd_kernel(const __grid_constant__ EmbedFwdParams p)
{
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
            set_status(p.status, kStatusInvalid);
        uint4 out[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int v = v0 + 32 * k;
            float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (live && v < p.nvec) {
                if (p.table_f32) {
                    const float4 *s =
                        reinterpret_cast<const float4 *>(static_cast<const float *>(p.table) + id * p.table_stride) +
                        2 * v;
                    const float4 a = __ldg(s), b = __ldg(s + 1);
                    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
                    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
                } else {
                    unpack8(__ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.table) +
                                                                  id * p.table_stride) +
                                  v),
                            f);
                }
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    f[q] = __fmul_rn(f[q], p.scale);
            }
            out[k] = pack8(f);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (v0 + 32 * k < p.nvec)
                __stcs(reinterpret_cast<uint4 *>(p.y + (int64_t)t * p.y_stride) + v0 + 32 * k, out[k]);
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
    return ((uint64_t)key << 32) | t;
}

__global__ void __launch_bounds__(kSortThreads) embed_count_kernel(const __grid_constant__ SortParams p)
{
    __shared__ uint32_t h[1 << kSortMaxBits];
    const int bins = 1 << p.bits;
    for (int i = threadIdx.x; i < bins; i += kSortThreads)
        h[i] = 0;
    __syncthreads();
    const uint32_t lo = blockIdx.x * p.tile_keys, hi = min(p.tokens, lo + p.tile_keys);
    for (uint32_t t = lo + threadIdx.x; t < hi; t += kSortThreads) {
        const uint64_t pr = make_pair(p, t);
        const uint32_t key = (uint32_t)(pr >> 32);
        if (key < p.vocab) {
            if (!((__ldcg(p.present + (key >> 5)) >> (key & 31)) & 1u)) // a common id is set once
                atomicOr(p.present + (key >> 5), 1u << (key & 31));
        } else if (load_id(p.ids, p.ids_i64, t) >= (int64_t)p.vocab) {
            set_status(p.status, kStatusInvalid);
        }
        atomicAdd(&h[key & (bins - 1)], 1u);
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

    // bins <= kSortThreads: thread d owns digit d
    uint32_t before = 0, all = 0;
    const int d = threadIdx.x;
    if (d < bins)
        for (int t = 0; t < p.tiles; ++t) {
            const uint32_t c = __ldcg(hist + (size_t)t * bins + d);
            all += c;
            before += t < (int)blockIdx.x ? c : 0;
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

    const uint32_t lo = blockIdx.x * p.tile_keys, hi = min(p.tokens, lo + p.tile_keys);
    for (uint32_t b0 = lo; b0 < hi; b0 += kSortBlock) {
        for (int i = threadIdx.x; i < kWarps * bins; i += kSortThreads)
            cnt[i / bins][i % bins] = 0;
        __syncthreads();
        // a warp's keys are contiguous and taken in order; equal digits of
        // the 32 keys of a step find each other by match
        uint64_t key[kSortPerThread];
        uint32_t rank[kSortPerThread];
#pragma unroll
        for (int j = 0; j < kSortPerThread; ++j) {
            const uint32_t t = b0 + warp * 32 * kSortPerThread + j * 32 + lane;
            const bool in = t < hi;
            key[j] = in ? (src ? __ldcg(src + t) : make_pair(p, t)) : ~0ull;
            // keys past the end get a digit of their own and are not counted
            const uint32_t dig = in ? (uint32_t)(key[j] >> (32 + shift)) & (bins - 1) : (uint32_t)bins;
            const uint32_t same = __match_any_sync(0xffffffffu, dig);
            const uint32_t below = __popc(same & ((1u << lane) - 1));
            uint32_t old = 0;
            if (in)
                old = cnt[warp][dig];
            rank[j] = old + below;
            __syncwarp();
            if (in && below == 0)
                cnt[warp][dig] = old + __popc(same);
            __syncwarp();
        }
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
// in [w * window, (w + 1) * window).  Runs that end within kOverrun positions
// after their window are finished by the window in which they start.  A run
// that goes further is cut at the window boundaries: its first window leaves
// a "trailing" partial, the windows that it fills one each, and the last a
// "leading" one.
constexpr int kSegThreads = 128;                // 8 columns a thread
constexpr int kSegCols = 8 * kSegThreads;
constexpr int kSegMaxWindow = 128;
constexpr int kOverrun = 32;
constexpr int kSegBatch = 8;                    // rows in flight
// meta[w][0]
constexpr uint32_t kMetaLead = 1;   // the window starts with a piece of an earlier window's run: partial 0
constexpr uint32_t kMetaLeadOn = 2; // ... that goes on in the next window
constexpr uint32_t kMetaTrail = 4;  // the window's last run goes on in the next window: partial 1

__device__ __forceinline__ void store_row8(const SegmentParams &p, uint32_t id, int col, const float (&s)[8])
{
    float v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
        v[q] = __fmul_rn(s[q], p.scale);
    if (p.dtable_f32) {
        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.dtable) + (int64_t)id * p.dtable_stride + col);
        if (p.accumulate) {
            const float4 a = o[0], b = o[1];
            v[0] = __fadd_rn(v[0], a.x), v[1] = __fadd_rn(v[1], a.y), v[2] = __fadd_rn(v[2], a.z);
            v[3] = __fadd_rn(v[3], a.w), v[4] = __fadd_rn(v[4], b.x), v[5] = __fadd_rn(v[5], b.y);
            v[6] = __fadd_rn(v[6], b.z), v[7] = __fadd_rn(v[7], b.w);
        }
        o[0] = make_float4(v[0], v[1], v[2], v[3]);
        o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint4 *o = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.dtable) + (int64_t)id * p.dtable_stride + col);
        if (p.accumulate) {
            float a[8];
            unpack8(*o, a);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                v[q] = __fadd_rn(v[q], a[q]);
        }
        *o = pack8(v);
    }
}

// Zeroes the rows of dtable whose id has no token: a warp per row.
__device__ void fill_rows(const SegmentParams &p, uint32_t part, uint32_t parts)
{
    const int lane = threadIdx.x & 31;
    const uint32_t warps = parts * (kSegThreads / 32);
    const int vecs = p.dtable_f32 ? 2 * p.nvec : p.nvec;
    for (uint32_t v = part * (kSegThreads / 32) + (threadIdx.x >> 5); v < p.vocab; v += warps) {
        if ((__ldcg(p.present + (v >> 5)) >> (v & 31)) & 1u)
            continue;
        uint4 *o = p.dtable_f32
                       ? reinterpret_cast<uint4 *>(static_cast<float *>(p.dtable) + (int64_t)v * p.dtable_stride)
                       : reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.dtable) + (int64_t)v * p.dtable_stride);
        for (int i = lane; i < vecs; i += 32)
            __stcs(o + i, make_uint4(0, 0, 0, 0));
    }
}

__global__ void __launch_bounds__(kSegThreads) embed_segment_kernel(const __grid_constant__ SegmentParams p)
{
    const uint32_t sums = (uint32_t)p.windows * p.slices;
    if (blockIdx.x >= sums) {
        fill_rows(p, blockIdx.x - sums, p.fill_ctas);
        return;
    }
    __shared__ uint32_t ids[kSegMaxWindow + kOverrun + 2], tok[kSegMaxWindow + kOverrun + 2];
    __shared__ int limits[2];
    const uint32_t w = blockIdx.x / p.slices, slice = blockIdx.x - w * p.slices;
    const uint32_t lo = w * p.window;
    const uint32_t W = min((uint32_t)p.window, p.tokens - lo); // positions of this window
    const uint32_t ext = min(p.tokens - lo, (uint32_t)p.window + kOverrun + 1); // and those looked at
    // ids[1 + i], tok[1 + i]: position lo + i; ids[0]: the position before
    for (uint32_t i = threadIdx.x; i < ext; i += kSegThreads) {
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
    for (uint32_t i = threadIdx.x; i < ext; i += kSegThreads) {
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
        if (W > kOverrun || goes_on) {
            first = 0;
            flags = kMetaLead;
            if (goes_on && over <= kOverrun)
                end = W + over;
            else if (goes_on)
                flags |= kMetaLeadOn;
            lead_end = end;
        }
    } else {
        if (lead > kOverrun) {
            first = 0;
            flags = kMetaLead;
        }
        if (goes_on && over <= kOverrun)
            end = W + over;
        else if (goes_on)
            flags |= kMetaTrail;
    }
    if (slice == 0 && threadIdx.x == 0) {
        p.meta[2 * w] = flags;
        p.meta[2 * w + 1] = ids[W];
    }

    const int col = (int)slice * kSegCols + 8 * (int)threadIdx.x;
    if (col >= 8 * p.nvec)
        return;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    float *lead_part = p.partials + ((size_t)w * 2) * 8 * p.nvec + col, *trail_part = lead_part + 8 * p.nvec;
    for (uint32_t b = first; b < end; b += kSegBatch) {
        uint4 r[kSegBatch];
#pragma unroll
        for (int k = 0; k < kSegBatch; ++k) {
            r[k] = make_uint4(0, 0, 0, 0);
            if (b + k < end && ids[1 + b + k] < p.vocab)
                r[k] = __ldcs(reinterpret_cast<const uint4 *>(p.dy + (int64_t)tok[1 + b + k] * p.dy_stride + col));
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
                        store_row8(p, id, col, s);
                    }
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        s[q] = 0.f;
                }
            }
        }
    }
}

// Joins the partials of the runs that were cut: the CTA of the window in
// which such a run starts adds the following windows' pieces in order.
__global__ void __launch_bounds__(kSegThreads) embed_join_kernel(const __grid_constant__ SegmentParams p)
{
    const uint32_t w = blockIdx.x / p.slices, slice = blockIdx.x - w * p.slices;
    if (!(__ldcg(p.meta + 2 * w) & kMetaTrail))
        return;
    const uint32_t id = __ldcg(p.meta + 2 * w + 1);
    const int H = 8 * p.nvec;
    const int col = (int)slice * kSegCols + 8 * (int)threadIdx.x;
    if (col >= H || id >= p.vocab)
        return;
    const float *t = p.partials + ((size_t)w * 2 + 1) * H + col;
    float s[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
        s[q] = __ldcg(t + q);
    for (uint32_t u = w + 1; u < (uint32_t)p.windows; ++u) {
        const uint32_t f = __ldcg(p.meta + 2 * u);
        const float *a = p.partials + (size_t)u * 2 * H + col;
#pragma unroll
        for (int q = 0; q < 8; ++q)
            s[q] = __fadd_rn(s[q], __ldcg(a + q));
        if (!(f & kMetaLeadOn))
            break;
    }
    store_row8(p, id, col, s);
}

// ------------------------------------------------------------------ launch

cudaError_t launch_embed_fwd(const EmbedFwdParams &p, cudaStream_t stream)
{
    const uint64_t items = (uint64_t)p.tokens * ((p.nvec + 127) / 128);
    const uint64_t want = (items + kEmbedThreads / 32 - 1) / (kEmbedThreads / 32);
    const int ctas = (int)(want < 152 * 8 * 8 ? want : 152 * 8 * 8);
    embed_fwd_kernel<<<ctas, kEmbedThreads, 0, stream>>>(p);
    return cudaGetLastError();
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
    embed_segment_kernel<<<p.windows * p.slices + p.fill_ctas, kSegThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_embed_join(const SegmentParams &p, cudaStream_t stream)
{
    embed_join_kernel<<<p.windows * p.slices, kSegThreads, 0, stream>>>(p);
    return cudaGetLastError();
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
    cudaError_t e = cudaMemcpyFromSymbol(code, g_step_status, sizeof(int));
    if (e == cudaSuccess && clear) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_step_status, &zero, sizeof(int));
    }
    return e;
}

} // namespace cake
