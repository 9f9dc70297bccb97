// cake_sandwich.cu -- the sandwich norm for sm_103a: the norm after a block,
// its gate, the residual scale and addition, and the norm before the next
// block, forward and backward.
//
// Forward, per row: z -> rstd_post -> h = bf16(x + scale g n) -> rstd_pre -> y.
// Backward, per row, with a = dy w_pre and b = g w_post (g per element, or 1):
//   S1 = sum a h,  S2 = sum (dh + rstd_pre a) b z,  S3 = sum b h z
//   c2 = rstd_pre S1 / H,     t = dh + rstd_pre a - k2 h,  k2 = rstd_pre^2 c2
//   sum t b z = S2 - k2 S3,   dz = scale g_row rstd_post (b t - k1 z),
//   k1 = rstd_post^2 (S2 - k2 S3) / H,  row gate: dgate = scale rstd_post (S2 - k2 S3)
// so that one pass and one reduction over the row give every scalar, instead
// of a pass for c2 and, after it, one for the mean of dn w_post zh.  Rounding
// errors are of the same order: t is linear in k2, and both forms round terms
// of the magnitudes |dh|, rstd_pre |a| and |k2 h|.
//
// Both kernels stream rows through shared memory as the RMSNorm kernels do
// (a producer warp with bulk copies, row groups of W warps as consumers,
// bounded waits).  HBM bounds the forward (GB300, T = 16384, H = 6144, a gate a
// row: 124 us, 0.96 of the copy rate); the backward is held by its warps'
// instruction latencies a little below that (T = 65536, H = 4096: 533 us, 0.89).
#include "../csrc/cake_rows.cuh"
#include "cake_step_launch.h"

namespace cake {

cudaError_t ensure_smem_attr(const void *kernel, size_t smem);

constexpr int kSMsStep = 152;
constexpr int kSwMaxStages = 16;
constexpr int kSwMaxTile = 15;            // rows of a stage, at most
constexpr int kSwSlots = 4;               // backward: rows whose partial sums may be in use
constexpr int kSwMaxJoined = 7;           // groups whose rows span several warps, at most
constexpr int kSwMaxRowWarps = 16;        // warps of a row over its cluster, at most
constexpr int kSwMaxCluster = 4;
constexpr int kSwClustersOf4 = 36;        // that a GB300 holds at a time
// Shared memory before the weights: the ring's barriers (256 bytes), the row
// sums' barriers (512), a flag (64), the row sums' partials, the rows' scalars.
constexpr int kSwRed = 832;
constexpr int kSwRedBytes = 4096;
constexpr int kSwScalarsAt = kSwRed + kSwRedBytes;
constexpr int kSwFixed = (kSwScalarsAt + kSwMaxStages * kSwMaxTile * 16 + 127) / 128 * 128;

// Room for the warps of a row in a slot of partial sums: 8 or 16; 1: rows of
// one warp, which need no slots.
__host__ __device__ constexpr int row_warps(int n) { return n == 1 ? 1 : n <= 8 ? 8 : 16; }

struct SwSmem {
    Smem s;               // barriers, reduction slots, flag, ring
    uint64_t *sums;       // [groups][slots] backward: a row's partial sums are written
    float4 *scalars;      // [stages][tile rows] (rstd_post, rstd_pre, row gate, -)
    float *w[2];          // w_post, w_pre as FP32, two planes each (see stage_weight)
};

__device__ __forceinline__ SwSmem sw_carve(uint8_t *base, const SandwichLayout &L)
{
    SwSmem m;
    m.s.full = reinterpret_cast<uint64_t *>(base);
    m.s.empty = m.s.full + L.stages;
    m.sums = reinterpret_cast<uint64_t *>(base + 256);
    m.s.flag = reinterpret_cast<int *>(base + 768);
    m.s.red = reinterpret_cast<float *>(base + kSwRed);
    m.scalars = reinterpret_cast<float4 *>(base + kSwScalarsAt);
    m.w[0] = reinterpret_cast<float *>(base + kSwFixed);
    m.w[1] = m.w[0] + weight_smem_bytes(L.cols) / 4;
    m.s.ring = base + kSwFixed + 2 * weight_smem_bytes(L.cols);
    m.s.tens_bytes = (uint32_t)L.groups * L.cols * 2;
    m.s.stage_bytes = m.s.tens_bytes * L.ntens;
    return m;
}

// The layout in the form that the shared pieces of the row pipeline take.
__device__ __forceinline__ Layout sw_rows_layout(const SandwichLayout &L, int nvec)
{
    Layout r = {};
    r.H = 8 * nvec;
    r.nvec = nvec;
    r.warps_per_row = L.W;
    r.groups = L.groups;
    r.stages = L.stages;
    return r;
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// The 8 weights of vector v (plane 0: columns 0-3 of the vectors, plane 1: 4-7).
__device__ __forceinline__ void sw_weight(const float *w, int nvec, int v, float2 (&w2)[4])
{
    const float4 a = reinterpret_cast<const float4 *>(w)[v], b = reinterpret_cast<const float4 *>(w)[nvec + v];
    w2[0] = make_float2(a.x, a.y);
    w2[1] = make_float2(a.z, a.w);
    w2[2] = make_float2(b.x, b.y);
    w2[3] = make_float2(b.z, b.w);
}

// Store to the shared memory of a CTA of the cluster, counted as 4 bytes on
// an mbarrier there.  Unlike a store and a releasing arrival, it does not wait
// for this thread's earlier stores to global memory (GB300, H = 4096: that
// release took the backward from 371 to 606 us at T = 32768).
__device__ __forceinline__ void st_async_f32(uint32_t cluster_addr, float v, uint32_t cluster_bar)
{
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(cluster_addr),
                 "r"(__float_as_uint(v)), "r"(cluster_bar)
                 : "memory");
}

__device__ __forceinline__ uint4 *out_row(const RowView &v, uint32_t r, uint32_t nh)
{
    return reinterpret_cast<uint4 *>(const_cast<uint16_t *>(v.base) + row_off(v, r, nh));
}

// Producer warp: streams vectors [v0, v0 + nvec) of the CTA's rows of every
// staged tensor into the ring;
// a row's scalars go along through plain shared stores, loaded a tile ahead
// and published by the arrival on the stage's full barrier.
template <int NT>
__device__ __forceinline__ void sw_produce(const SwSmem &m, const SandwichLayout &L, const RowView (&in)[NT],
                                           const float *sc0, const float *sc1, const float *sc2, int v0, int nvec,
                                           uint32_t r0, uint32_t r_end, int *status, uint64_t wait_ns, int withhold)
{
    const uint32_t lane = threadIdx.x & 31;
    const uint64_t pol = policy_evict_first();
    const uint32_t row_bytes = (uint32_t)nvec * 16, tile = (uint32_t)L.groups, pitch = (uint32_t)L.cols * 2;
    auto scalars = [&](uint32_t row0) {
        float4 v = make_float4(0.f, 0.f, 1.f, 0.f);
        if (lane < tile && row0 + lane < r_end) {
            if (sc0)
                v.x = __ldg(sc0 + row0 + lane);
            if (sc1)
                v.y = __ldg(sc1 + row0 + lane);
            if (sc2)
                v.z = __ldg(sc2 + row0 + lane);
        }
        return v;
    };
    // tests of the waits: 16 bytes of the first stage that never come
    if (lane == 0 && (withhold == 1 || (withhold == 2 && blockIdx.x == 0)))
        asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], 16;" ::"r"(smem_addr(&m.s.full[0]))
                     : "memory");
    float4 next = scalars(r0);
    uint32_t st = 0, ph = 0, it = 0;
    for (uint32_t row0 = r0; row0 < r_end; row0 += tile, ++it) {
        if (it >= (uint32_t)L.stages &&
            !__all_sync(0xffffffffu, mbar_wait(smem_addr(&m.s.empty[st]), ph ^ 1u, wait_ns))) {
            if (lane == 0)
                set_status(status, kStatusTimeout);
            break;
        }
        const uint32_t n = min(tile, r_end - row0);
        const uint32_t bar = smem_addr(&m.s.full[st]);
        if (lane < n)
            m.scalars[st * kSwMaxTile + lane] = next;
        __syncwarp();
        if (lane == 0)
            mbar_arrive_expect_tx(bar, (uint32_t)L.ntens * n * row_bytes);
        __syncwarp();
        const uint32_t dst0 = smem_addr(m.s.ring) + st * m.s.stage_bytes;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (t >= L.ntens)
                break;
            const uint32_t dst = dst0 + t * m.s.tens_bytes;
            if (in[t].dense && L.cluster == 1) {
                if (lane == 0)
                    bulk_g2s(dst, in[t].base + (int64_t)row0 * in[t].row_stride, n * row_bytes, bar, pol);
            } else if (lane < n) {
                bulk_g2s(dst + lane * pitch, in[t].base + row_off(in[t], row0 + lane, L.nh) + 8 * v0, row_bytes, bar,
                         pol);
            }
        }
        next = scalars(row0 + tile);
        if (++st == (uint32_t)L.stages) {
            st = 0;
            ph ^= 1u;
        }
    }
    // no copy of this CTA is left in flight
    const uint32_t first = it > (uint32_t)L.stages ? it - L.stages : 0;
    for (uint32_t j = first; j < it; ++j)
        if (!mbar_wait(smem_addr(&m.s.full[j % L.stages]), (j / L.stages) & 1, wait_ns) && lane == 0)
            set_status(status, kStatusTimeout);
}

// ------------------------------------------------------------------ forward

constexpr int kSwFwdThreads = 416;  // 12 consumer warps and the producer
constexpr int kSwWideThreads = 544; // 16: rows of more than 6144 columns

template <int VPT, bool GATE, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) sandwich_fwd_kernel(const __grid_constant__ SandwichFwdParams p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const SandwichLayout &L = p.L;
    const SwSmem m = sw_carve(smem_raw, L);
    const int nvec = L.cols / 8;
    const Layout RL = sw_rows_layout(L, nvec);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t r0 = blockIdx.x * L.rows_per_cta, r_end = min(L.rows, r0 + L.rows_per_cta);
    init_ring(m.s, RL);
    pdl_wait();
    if (warp == L.groups * L.W) {
        sw_produce(m, L, p.in, nullptr, nullptr, p.gate_rows, 0, nvec, r0, r_end, p.status, p.wait_ns,
                   p.withhold);
        return;
    }
    const int gid = warp / L.W, wig = warp - gid * L.W, gtid = wig * 32 + lane, vstride = 32 * L.W;
    {
        Smem sw = m.s;
        sw.wsm = m.w[0];
        stage_weight(sw, RL, p.w_post, p.post_f32);
        sw.wsm = m.w[1];
        stage_weight(sw, RL, p.w_pre, p.pre_f32);
    }
    bool abort = false;
    uint32_t slot = 0, st = 0, ph = 0;
    const uint32_t tile = (uint32_t)L.groups;
    for (uint32_t row0 = r0; row0 < r_end && !abort; row0 += tile) {
        abort = !mbar_wait(smem_addr(&m.s.full[st]), ph, p.wait_ns);
        const uint32_t r = row0 + gid;
        if (r < r_end) { // uniform across the group
            const uint8_t *stage = m.s.ring + st * m.s.stage_bytes + (size_t)gid * L.cols * 2;
            const uint4 *zs = reinterpret_cast<const uint4 *>(stage);
            const uint4 *xs = reinterpret_cast<const uint4 *>(stage + m.s.tens_bytes);
            const uint4 *gs = reinterpret_cast<const uint4 *>(stage + 2 * m.s.tens_bytes);
            const float sg = __fmul_rn(p.scale, m.scalars[st * kSwMaxTile + gid].z);
            uint4 z[VPT];
            float2 ss = both(0.f);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = k * vstride + gtid;
                z[k] = v < nvec ? zs[v] : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float2 a = bf2(word(z[k], q));
                    ss = fma2(a, a, ss);
                }
            }
            float tot = group_sum(__fadd_rn(ss.x, ss.y), m.s, RL, gid, wig, lane, slot++, abort);
            const float r1 = 1.0f / sqrtf(__fadd_rn(__fmul_rn(tot, L.inv_h), p.eps));
            uint4 h[VPT];
            ss = both(0.f);
            uint4 *hrow = out_row(p.h_new, r, L.nh);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = k * vstride + gtid;
                h[k] = make_uint4(0, 0, 0, 0);
                if (v < nvec) {
                    const uint4 x = xs[v];
                    uint4 g = make_uint4(0, 0, 0, 0);
                    if (GATE)
                        g = gs[v];
                    float2 w2[4];
                    sw_weight(m.w[0], nvec, v, w2);
                    uint32_t o[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float2 n = mul2(mul2(bf2(word(z[k], q)), both(r1)), w2[q]);
                        const float2 f = GATE ? mul2(both(sg), bf2(word(g, q))) : both(sg);
                        o[q] = pack2(fma2(f, n, bf2(word(x, q))));
                        const float2 a = bf2(o[q]);
                        ss = fma2(a, a, ss);
                    }
                    h[k] = make_uint4(o[0], o[1], o[2], o[3]);
                    if (!abort)
                        __stcs(hrow + v, h[k]);
                }
            }
            tot = group_sum(__fadd_rn(ss.x, ss.y), m.s, RL, gid, wig, lane, slot++, abort);
            const float r2 = 1.0f / sqrtf(__fadd_rn(__fmul_rn(tot, L.inv_h), p.eps));
            uint4 *yrow = out_row(p.y, r, L.nh);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = k * vstride + gtid;
                if (v < nvec && !abort) {
                    float2 w2[4];
                    sw_weight(m.w[1], nvec, v, w2);
                    uint32_t o[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        o[q] = pack2(mul2(mul2(bf2(word(h[k], q)), both(r2)), w2[q]));
                    __stcs(yrow + v, make_uint4(o[0], o[1], o[2], o[3]));
                }
            }
            if (gtid == 0 && !abort) {
                p.rstd_post[r] = r1;
                p.rstd_pre[r] = r2;
            }
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(smem_addr(&m.s.empty[st]));
        if (++st == (uint32_t)L.stages) {
            st = 0;
            ph ^= 1u;
        }
    }
    if (abort && lane == 0)
        set_status(p.status, kStatusTimeout);
}

// ----------------------------------------------------------------- backward

// Kahan-compensated hi += a * b of column pairs; lo holds the part of the
// last term that hi has not taken up.
__device__ __forceinline__ void kahan2(float2 &hi, float2 &lo, float2 a, float2 b)
{
    const float2 y = fma2(a, b, lo);
    const float2 t = add2(hi, y);
    lo = add2(sub2(hi, t), y);
    hi = t;
}

// The three sums of a row over a warp: lanes [8 n, 8 n + 8) end with sum n
// (n = 3: zero).  Each of the first two steps halves the values that a lane
// still carries, so three sums take 6 shuffles instead of 15.
__device__ __forceinline__ float warp_sum3(float v0, float v1, float v2, int lane)
{
    const bool up = lane & 16, hi = lane & 8;
    float a = up ? v2 : v0, b = up ? 0.f : v1;
    a = __fadd_rn(a, __shfl_xor_sync(0xffffffffu, up ? v0 : v2, 16));
    b = __fadd_rn(b, __shfl_xor_sync(0xffffffffu, up ? v1 : 0.f, 16));
    float r = hi ? b : a;
    r = __fadd_rn(r, __shfl_xor_sync(0xffffffffu, hi ? a : b, 8));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
        r = __fadd_rn(r, __shfl_xor_sync(0xffffffffu, r, o));
    return r;
}

// mbar_wait with one answer for the whole warp: its lanes go on, or give up, together.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns)
{
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, limit_ns));
}

__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(kSuspendHintNs)
        : "memory");
    return ok != 0;
}

// warp_wait for a phase that other CTAs of the cluster complete: it acquires
// their writes at the cluster's scope.
__device__ __forceinline__ bool warp_wait_cluster(uint32_t bar, uint32_t parity, uint64_t limit_ns)
{
    bool ok = try_wait_cluster(bar, parity);
    if (!ok) {
        const uint64_t t0 = globaltimer_ns();
        for (uint32_t i = 1; !ok; ++i) {
            ok = try_wait_cluster(bar, parity);
            if (!ok && (i & 3u) == 0 && globaltimer_ns() - t0 > limit_ns)
                break;
        }
    }
    return __all_sync(0xffffffffu, ok);
}

// GATE: 0 none, 1 a value per row, 2 a value per element.  CL: rows span a
// cluster.  RW: row_warps of the layout.
//
// A thread holds the two column sums of 8 VPT columns as Kahan pairs, 32 VPT
// registers, which is why it takes no more than 16 columns.  With 12 consumer
// warps of 128 registers an SM then holds 6144 columns of rows.  A warp's own
// latencies bound its rate (GB300, ncu at H = 4096 on 8 warps: issue slots 43 %
// used, 5.2 cycles a warp and instruction), so rows that leave warps unused at
// this width, or do not fit three stages, are split over a cluster of 2 or 4
// CTAs, each with its share of the columns and, so, of the weights.
//
// Order of work: first pass of row j + 1 (its three sums and dw_pre), then
// the second pass of row j (its outputs and dw_post).  The sums of a row
// travel between the row's warps, in every CTA of its cluster, through shared
// memory behind an mbarrier that a warp arrives on after its first pass and
// tests after the next row's, so that no warp waits for a reduction.  A warp
// writes row j + 2's sums only after row j's have all come to its CTA, which
// needs every warp of the row to have read row j - 2's: four slots, each with
// a barrier of its own, hold the rows that may be in use, also where sums
// reach one CTA of a cluster later than another.
constexpr int kSwBwdWarps = 12;     // consumer warps; four more hold the producer
constexpr int kSwBwdManyWarps = 15; // ... or fifteen at 128 registers, and the producer
constexpr int kSwBwdThreads = 32 * (kSwBwdWarps + 4);
static_assert(kSwBwdThreads == 32 * (kSwBwdManyWarps + 1), "both forms launch 16 warps");

// MANY: up to 15 consumer warps instead of 12, for rows of 2, 5 or 7 warps, of
// which 12 hold fewer, and for threads of 8 or 12 columns, whose sums take fewer
// registers (GB300, 2^27 values: H = 2560 272 us against 307, 5120 282 against
// 322, 7168 292 against 328, 256 265 against 283; 1024 with an element gate 338
// against 349).
//
// HALF: a thread takes 4 columns more, the half vectors behind the row's first
// 32 W vectors: 12 columns a thread.
template <int VPT, int GATE, bool CL, int RW, bool MANY = false, bool HALF = false>
__global__ void __launch_bounds__(kSwBwdThreads, 1) sandwich_bwd_kernel(const __grid_constant__ SandwichBwdParams p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const SandwichLayout &L = p.L;
    const SwSmem m = sw_carve(smem_raw, L);
    const int C = CL ? L.cluster : 1;
    const uint32_t rank = CL ? cluster_ctarank() : 0, cid = CL ? blockIdx.x / C : blockIdx.x;
    const int v0 = (int)rank * (L.cols / 8), nvec = CL ? min(L.cols / 8, L.nvec - v0) : L.nvec; // this CTA's vectors
    const Layout RL = sw_rows_layout(L, nvec);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t r0 = cid * L.rows_per_cta, r_end = min(L.rows, r0 + L.rows_per_cta);
    if (threadIdx.x < kSwSlots * L.groups) // in a cluster: one arrival, and the bytes that come
        mbar_init(smem_addr(m.sums + threadIdx.x), CL ? 1 : L.W);
    for (int i = threadIdx.x; i < kSwRedBytes / 4; i += blockDim.x)
        m.s.red[i] = 0.f; // the parts of warps that a row does not have stay zero
    if (CL && threadIdx.x < kSwSlots * L.groups)
        fence_mbar_init();
    init_ring(m.s, RL);
    if (CL)
        cluster_sync_all(); // every CTA's barriers and slots exist before a remote access
    pdl_wait();
    // Registers: 16 warps start with 128 each; the last four give 72 up, and
    // the twelve consumer warps take 24 more (12 x 152 + 4 x 56 = 16 x 128).
    constexpr int kProducer = MANY ? kSwBwdManyWarps : kSwBwdWarps;
    if (warp >= kProducer) {
        if (!MANY)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == kProducer)
            sw_produce(m, L, p.in, p.rstd_post, p.rstd_pre, p.gate_rows, v0, nvec, r0, r_end, p.status, p.wait_ns,
                       p.withhold);
        __syncwarp();
        if (CL)
            cluster_sync_all();
        return;
    }
    if (!MANY)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
    if (warp >= L.groups * L.W) { // no row for this warp
        if (CL)
            cluster_sync_all();
        return;
    }
    const int gid = warp / L.W, wig = warp - gid * L.W, gtid = wig * 32 + lane, vstride = 32 * L.W;
    const bool has_dh = p.has_dh;
    constexpr bool joined = RW > 1;
    {
        Smem sw = m.s;
        sw.wsm = m.w[0];
        stage_weight(sw, RL, static_cast<const uint8_t *>(p.w_post) + v0 * (p.post_f32 ? 32 : 16), p.post_f32);
        sw.wsm = m.w[1];
        stage_weight(sw, RL, static_cast<const uint8_t *>(p.w_pre) + v0 * (p.pre_f32 ? 32 : 16), p.pre_f32);
    }
    // Piece k of the thread's columns is vector k * vstride + gtid, or half
    // vector gtid behind all of those: index(k) counts in vectors or halves.
    constexpr int K = VPT + HALF;
    auto is_half = [](int k) { return HALF && k == VPT; };
    auto index = [&](int k) { return is_half(k) ? 2 * VPT * vstride + gtid : k * vstride + gtid; };
    auto inside = [&](int k, int v) { return v < (is_half(k) ? 2 * nvec : nvec); };
    auto at = [&](const uint4 *row, int k, int v) { // the piece's address
        return is_half(k) ? reinterpret_cast<const uint4 *>(reinterpret_cast<const uint2 *>(row) + v) : row + v;
    };
    auto load = [&](const uint4 *from, int k) {
        if (!is_half(k))
            return *from;
        const uint2 a = *reinterpret_cast<const uint2 *>(from);
        return make_uint4(a.x, a.y, 0, 0);
    };
    auto store = [&](uint4 *row, int k, int v, const uint32_t(&o)[4]) {
        if (is_half(k))
            __stcs(reinterpret_cast<uint2 *>(row) + v, make_uint2(o[0], o[1]));
        else
            __stcs(row + v, make_uint4(o[0], o[1], o[2], o[3]));
    };
    auto weight = [&](int which, int k, int v, float2(&w2)[4]) {
        if (is_half(k)) {
            const float4 a = reinterpret_cast<const float4 *>(m.w[which])[(v & 1) * nvec + (v >> 1)];
            w2[0] = make_float2(a.x, a.y);
            w2[1] = make_float2(a.z, a.w);
        } else {
            sw_weight(m.w[which], nvec, v, w2);
        }
    };
    float2 hi1[K][4], lo1[K][4], hi2[K][4], lo2[K][4]; // dw_post, dw_pre
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            hi1[k][q] = lo1[k][q] = hi2[k][q] = lo2[k][q] = both(0.f);

    const uint32_t tile = (uint32_t)L.groups, tb = m.s.tens_bytes / 16;
    const uint32_t dh_off = (GATE == 2 ? 4 : 3) * tb;
    const uint32_t ntiles = r_end > r0 ? (r_end - r0 + tile - 1) / tile : 0;
    const uint4 *gbase = reinterpret_cast<const uint4 *>(m.s.ring + (size_t)gid * L.cols * 2);
    const uint32_t sbytes = m.s.stage_bytes / 16;
    float *red = m.s.red + gid * kSwSlots * 4 * RW; // a slot: [4 sums][RW]
    float own = 0.f; // rows of one warp: the sums of the row between its passes
    bool abort = false;
    uint32_t st1 = 0, ph1 = 0; // ring slot of the first pass
    for (uint32_t j = 0; j <= ntiles && !abort; ++j) {
        float mine = 0.f;
        if (j < ntiles) {
            abort = !warp_wait(smem_addr(&m.s.full[st1]), ph1, p.wait_ns);
            if (r0 + j * tile + gid < r_end && !abort) { // uniform across the warp
                const float2 rn = both(m.scalars[st1 * kSwMaxTile + gid].y);
                float2 s1 = both(0.f), s2 = both(0.f), s3 = both(0.f);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int v = index(k);
                    if (inside(k, v)) {
                        const uint4 *row = at(gbase + st1 * sbytes, k, v);
                        const uint4 h = load(row, k), z = load(row + tb, k), d = load(row + 2 * tb, k);
                        uint4 g = make_uint4(0, 0, 0, 0), e = make_uint4(0, 0, 0, 0);
                        if (GATE == 2)
                            g = load(row + 3 * tb, k);
                        if (has_dh)
                            e = load(row + dh_off, k);
                        float2 w1[4], w2[4];
                        weight(0, k, v, w1);
                        weight(1, k, v, w2);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            if (is_half(k) && q >= 2)
                                continue;
                            const float2 hq = bf2(word(h, q)), dq = bf2(word(d, q));
                            const float2 a = mul2(dq, w2[q]);
                            const float2 bz =
                                mul2(bf2(word(z, q)), GATE == 2 ? mul2(w1[q], bf2(word(g, q))) : w1[q]);
                            s1 = fma2(a, hq, s1);
                            s2 = fma2(fma2(rn, a, bf2(word(e, q))), bz, s2);
                            s3 = fma2(bz, hq, s3);
                            kahan2(hi2[k][q], lo2[k][q], mul2(dq, hq), rn);
                        }
                    }
                }
                mine = warp_sum3(__fadd_rn(s1.x, s1.y), __fadd_rn(s2.x, s2.y), __fadd_rn(s3.x, s3.y), lane);
                if (joined) {
                    float *at = red + ((j & 3) * 4 + (lane >> 3)) * RW + (CL ? cluster_ctarank() * L.W : 0) + wig;
                    const uint32_t bar = smem_addr(m.sums + kSwSlots * gid + (j & 3));
                    if (CL) {
                        // to every CTA of the cluster, each sum by a lane that holds it
                        if (wig == 0 && lane == 0)
                            mbar_arrive_expect_tx(bar, 12u * L.W * C);
                        if ((lane & 7) < C && lane < 24)
                            st_async_f32(map_to_rank(smem_addr(at), lane & 7), mine, map_to_rank(bar, lane & 7));
                    } else {
                        if ((lane & 7) == 0)
                            *at = mine;
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(bar);
                    }
                }
            }
            if (++st1 == (uint32_t)L.stages) {
                st1 = 0;
                ph1 ^= 1u;
            }
        }
        if (j > 0) {
            const uint32_t i = j - 1, r = r0 + i * tile + gid;
            // the second pass's slot, one before the first pass's
            const uint32_t back = j < ntiles ? 2 : 1, st2 = st1 >= back ? st1 - back : st1 + L.stages - back;
            if (r < r_end) {
                float t3 = own;
                if (joined) {
                    const uint32_t bar = smem_addr(m.sums + kSwSlots * gid + (i & 3));
                    if (!(CL ? warp_wait_cluster(bar, (i >> 2) & 1, p.wait_ns)
                             : warp_wait(bar, (i >> 2) & 1, p.wait_ns)))
                        abort = true;
                    // eight lanes to a sum
                    const float *from = red + (i & 3) * 4 * RW;
                    if (RW == 8) {
                        t3 = from[lane];
                    } else {
                        const float2 a = reinterpret_cast<const float2 *>(from)[lane];
                        t3 = __fadd_rn(a.x, a.y);
                    }
#pragma unroll
                    for (int o = 4; o > 0; o >>= 1)
                        t3 = __fadd_rn(t3, __shfl_xor_sync(0xffffffffu, t3, o));
                }
                const float t1 = __shfl_sync(0xffffffffu, t3, 0), t2 = __shfl_sync(0xffffffffu, t3, 8);
                t3 = __shfl_sync(0xffffffffu, t3, 16);
                const float4 sc = m.scalars[st2 * kSwMaxTile + gid];
                const float k2 = __fmul_rn(__fmul_rn(__fmul_rn(__fmul_rn(t1, L.inv_h), sc.y), sc.y), sc.y);
                const float dot = __fmaf_rn(-k2, t3, t2);
                const float2 nk2 = both(-k2), rn = both(sc.y);
                const float s_r = __fmul_rn(GATE == 1 ? __fmul_rn(p.scale, sc.z) : p.scale, sc.x);
                const float k1 = __fmul_rn(__fmul_rn(__fmul_rn(dot, L.inv_h), sc.x), sc.x);
                const float2 sr = both(s_r), nks = both(-__fmul_rn(k1, s_r));
                if (GATE == 1 && p.dgate_rows && gtid == 0 && (!CL || cluster_ctarank() == 0) && !abort)
                    p.dgate_rows[r] = __fmul_rn(__fmul_rn(p.scale, sc.x), dot);
                // (the rank is read again where it is needed: a register less over the loop)
                const int vo = CL ? (int)cluster_ctarank() * (L.cols / 8) : 0;
                uint4 *dx = out_row(p.dx, r, L.nh) + vo, *dz = out_row(p.dz, r, L.nh) + vo;
                uint4 *dg = GATE == 2 && p.dgate.base ? out_row(p.dgate, r, L.nh) + vo : nullptr;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int v = index(k);
                    if (inside(k, v) && !abort) {
                        const uint4 *row = at(gbase + st2 * sbytes, k, v);
                        const uint4 h = load(row, k), z = load(row + tb, k), d = load(row + 2 * tb, k);
                        uint4 g = make_uint4(0, 0, 0, 0), e = make_uint4(0, 0, 0, 0);
                        if (GATE == 2)
                            g = load(row + 3 * tb, k);
                        if (has_dh)
                            e = load(row + dh_off, k);
                        float2 w1[4], w2[4];
                        weight(0, k, v, w1);
                        weight(1, k, v, w2);
                        uint32_t ox[4], oz[4], og[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            if (is_half(k) && q >= 2)
                                continue;
                            const float2 zq = bf2(word(z, q));
                            const float2 a = mul2(bf2(word(d, q)), w2[q]);
                            const float2 t = fma2(nk2, bf2(word(h, q)), fma2(rn, a, bf2(word(e, q))));
                            ox[q] = pack2(t);
                            const float2 st = mul2(sr, t);
                            const float2 mt = GATE == 2 ? mul2(st, bf2(word(g, q))) : st;
                            oz[q] = pack2(fma2(mt, w1[q], mul2(nks, zq)));
                            if (GATE == 2)
                                og[q] = pack2(mul2(mul2(st, zq), w1[q]));
                            kahan2(hi1[k][q], lo1[k][q], mt, zq);
                        }
                        store(dx, k, v, ox);
                        store(dz, k, v, oz);
                        if (GATE == 2 && dg)
                            store(dg, k, v, og);
                    }
                }
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_addr(&m.s.empty[st2]));
        }
        own = mine;
    }
    if (abort && lane == 0)
        set_status(p.status, kStatusTimeout);

    // The CTA partial: the groups' sums in group order, through the drained
    // ring ([group][w][4 nvec] float4 (hi, lo, hi, lo) of a column pair).
    const int nct = L.groups * L.W * 32, nslot = 4 * nvec;
    const int vp = CL ? (int)cluster_ctarank() * (L.cols / 8) : 0;
    float4 *comb = reinterpret_cast<float4 *>(m.s.ring);
    consumer_sync(RL);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int v = index(k), pair = is_half(k) ? 2 * v : 4 * v;
        if (inside(k, v))
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (is_half(k) && q >= 2)
                    continue;
                comb[(size_t)(2 * gid) * nslot + pair + q] =
                    make_float4(hi1[k][q].x, lo1[k][q].x, hi1[k][q].y, lo1[k][q].y);
                comb[(size_t)(2 * gid + 1) * nslot + pair + q] =
                    make_float4(hi2[k][q].x, lo2[k][q].x, hi2[k][q].y, lo2[k][q].y);
            }
    }
    consumer_sync(RL);
    for (int i = threadIdx.x; i < 2 * nslot; i += nct) {
        const int w = i >= nslot, c = i - w * nslot;
        float4 a = comb[i];
        for (int g = 1; g < L.groups; ++g) {
            const float4 b = comb[(size_t)2 * g * nslot + i];
            comp_add(a.x, a.y, b.x);
            a.y = __fadd_rn(a.y, b.y);
            comp_add(a.z, a.w, b.z);
            a.w = __fadd_rn(a.w, b.w);
        }
        reinterpret_cast<float4 *>(p.partials + ((size_t)w * (gridDim.x / C) + cid) * L.H)[4 * vp + c] = a;
    }
    __syncwarp();
    if (CL)
        cluster_sync_all(); // no CTA leaves while another may still write to its slots
    pdl_launch_dependents();
}

// Column sums of the CTA partials in CTA order: a warp takes 32 columns and
// every 16th CTA; the 16 sums of a column are then added in warp order.
constexpr int kSwReduceWarps = 16;

__global__ void __launch_bounds__(32 * kSwReduceWarps)
    sandwich_reduce_kernel(const __grid_constant__ SandwichReduceParams p)
{
    __shared__ float2 part[kSwReduceWarps][32];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int j = blockIdx.x * 32 + lane;
    const float2 *src = p.partials + (size_t)blockIdx.y * p.P * p.H;
    float hi = 0.f, lo = 0.f;
    if (j < p.H)
        for (int q = warp; q < p.P; q += kSwReduceWarps) {
            const float2 v = __ldcg(src + (size_t)q * p.H + j);
            comp_add(hi, lo, v.x);
            lo = __fadd_rn(lo, v.y);
        }
    part[warp][lane] = make_float2(hi, lo);
    __syncthreads();
    if (warp == 0 && j < p.H) {
        for (int w = 1; w < kSwReduceWarps; ++w) {
            comp_add(hi, lo, part[w][lane].x);
            lo = __fadd_rn(lo, part[w][lane].y);
        }
        p.dw[blockIdx.y][j] = __fadd_rn(hi, lo);
    }
}

// ------------------------------------------------------------------ launch

// The shape of a CTA.  It depends on H and the staged tensors, the number of
// CTAs on the rows too, and on nothing else, so the sums' orders do not either.
// false: such a CTA does not fit.
static bool try_plan(SandwichPlan &p, int H, int ntens, bool backward, int cluster, int groups)
{
    const int nvec = (H / 8 + cluster - 1) / cluster; // of a CTA
    p.cluster = cluster;
    p.cols = 8 * nvec;
    // 8 columns a thread up to 256, 16 beyond; the backward of rows of one CTA
    // takes 12 where they leave fewer lanes without work (GB300, 2^27 values:
    // H = 264 321 us against 444, 384 253 against 310, 640 321 against 404, 1032 283
    // against 348, 1152 261 against 317, 1664 279 against 313; the copy takes 238)
    p.half = backward && H <= 2048 && nvec > 32 && (nvec + 47) / 48 * 48 < (nvec + 63) / 64 * 64;
    p.vpt = nvec <= 32 || p.half ? 1 : 2;
    p.W = p.half ? (nvec + 47) / 48 : (nvec + 32 * p.vpt - 1) / (32 * p.vpt);
    p.groups = groups;
    const bool many = p.vpt == 1 || ((p.W == 2 || p.W == 5 || p.W == 7) && cluster <= 2);
    if (p.groups * p.W > (!backward ? 16 : many ? kSwBwdManyWarps : kSwBwdWarps))
        return false;
    if (backward && cluster == 1 && p.W > 8) // (a cluster of 2 leaves fewer warps without work)
        return false;
    // CTAs per SM: the backward's takes all registers, 28 of the forward's warps fit
    p.per_sm = backward ? 1 : 28 / (p.groups * p.W + 1) >= 2 ? 2 : 1;
    const size_t fixed = (size_t)kSwFixed + 2 * weight_smem_bytes(p.cols);
    const size_t stage = (size_t)ntens * p.groups * p.cols * 2;
    // the backward holds two rows of a group at once and a third is to be
    // on its way; the forward works on one
    const int want = backward ? 3 : 2;
    for (;; --p.per_sm) {
        const size_t room = 228 * 1024 / p.per_sm - 1024; // 1 KB of each CTA is the system's
        p.stages = room > fixed ? (int)((room - fixed) / stage) : 0;
        if (p.stages >= want || p.per_sm == 1)
            break;
    }
    // three stages of the forward against four to eight, GB300, 2^27 values:
    // H = 256 174 us against 192, H = 2560 180 against 187; the others the same
    const int most = backward ? kSwMaxStages : 3;
    if (p.stages > most)
        p.stages = most;
    p.smem = fixed + (size_t)p.stages * stage;
    const size_t comb = fixed + (size_t)(backward ? p.groups : 0) * p.cols * 16;
    if (comb > p.smem)
        p.smem = comb;
    if (p.smem > 227 * 1024 || p.cols * (cluster - 1) >= H)
        return false;
    if (p.W * cluster > 1 && (p.groups > kSwMaxJoined || p.W * cluster > kSwMaxRowWarps ||
                              p.groups * kSwSlots * 16 * row_warps(p.W * cluster) > kSwRedBytes))
        return false;
    return p.stages >= want;
}

SandwichPlan sandwich_plan(int H, uint32_t rows, int ntens, bool backward)
{
    SandwichPlan p{};
    if (!backward) {
        const int W = H <= 256 ? 1 : (H + 511) / 512;
        try_plan(p, H, ntens, false, 1, W >= 12 ? 1 : 12 / W);
    } else {
        // The most columns in work on an SM, up to the 6144 that keep HBM
        // busy; of equals the smallest cluster.  Weights, as measured on GB300
        // with 2^27 values without a gate (copy rate: 238 us): three stages
        // against four 296 and 263 us at H = 2048 (with an element gate seven
        // groups of three against six of four 381 and 368 us at H = 840), a single
        // group against two 290 and 266 us at H = 6144; 36 clusters of 4 fit the
        // 152 SMs.
        int best = 0;
        for (int c = 1; c <= (H > 2048 ? kSwMaxCluster : 1); c *= 2)
            for (int g = kSwMaxTile; g >= 1; --g) {
                SandwichPlan q{};
                if (!try_plan(q, H, ntens, true, c, g))
                    continue;
                int score = q.cols * q.groups * q.per_sm;
                score = score > 6144 ? 6144 : score;
                if (q.stages < 4)
                    score = score * 85 / 100;
                if (q.groups * q.per_sm == 1)
                    score = score * 93 / 100;
                score = c == 4 ? score * 93 / 100 : c == 2 ? score * 97 / 100 : score;
                if (score > best) {
                    best = score;
                    p = q;
                }
            }
    }
    const uint32_t tile = (uint32_t)p.groups;
    uint32_t ctas = (rows + tile - 1) / tile; // clusters, where a row has one
    const uint32_t most = p.cluster == 4 ? kSwClustersOf4 : (uint32_t)kSMsStep * p.per_sm / p.cluster;
    if (ctas > most)
        ctas = most;
    p.rows_per_cta = ctas ? (rows + ctas - 1) / ctas : 0;
    p.parts = p.rows_per_cta ? (int)((rows + p.rows_per_cta - 1) / p.rows_per_cta) : 0;
    return p;
}

template <class P>
static cudaError_t launch_rows(void (*kern)(P), const P &p, const SandwichPlan &plan, int threads, cudaStream_t stream)
{
    cudaError_t e = ensure_smem_attr((const void *)kern, plan.smem);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(plan.parts * plan.cluster));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = plan.smem;
    cfg.stream = stream;
    // started while the launch before it drains (GB300: 2 to 4 us less a call where calls follow one another)
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)plan.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = plan.cluster > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kern, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_sandwich_fwd(const SandwichFwdParams &p, const SandwichPlan &plan, cudaStream_t stream)
{
    const bool g = p.L.ntens == 3;
    const int threads = 32 * (plan.groups * plan.W + 1);
    if (plan.vpt == 1)
        return g ? launch_rows(sandwich_fwd_kernel<1, true, kSwFwdThreads>, p, plan, threads, stream)
                 : launch_rows(sandwich_fwd_kernel<1, false, kSwFwdThreads>, p, plan, threads, stream);
    if (plan.W <= 12)
        return g ? launch_rows(sandwich_fwd_kernel<2, true, kSwFwdThreads>, p, plan, threads, stream)
                 : launch_rows(sandwich_fwd_kernel<2, false, kSwFwdThreads>, p, plan, threads, stream);
    return g ? launch_rows(sandwich_fwd_kernel<2, true, kSwWideThreads>, p, plan, threads, stream)
             : launch_rows(sandwich_fwd_kernel<2, false, kSwWideThreads>, p, plan, threads, stream);
}

SandwichBuild sandwich_build(const SandwichPlan &plan)
{
    SandwichBuild b;
    b.vpt = plan.vpt;
    b.rw = row_warps(plan.W * plan.cluster);
    b.cl = plan.cluster > 1;
    b.many = plan.vpt == 1 || plan.groups * plan.W > kSwBwdWarps;
    b.half = plan.half;
    return b;
}

template <int GATE, int VPT, bool CL, int RW, bool MANY, bool HALF>
static bool launch_build(const SandwichBuild &b, const SandwichBwdParams &p, const SandwichPlan &plan,
                         cudaStream_t stream, cudaError_t &e)
{
    if (b.vpt != VPT || b.cl != CL || b.rw != RW || b.many != MANY || b.half != HALF)
        return false;
    e = launch_rows(sandwich_bwd_kernel<VPT, GATE, CL, RW, MANY, HALF>, p, plan, kSwBwdThreads, stream);
    return true;
}

// The builds that some width's plan takes.
template <int GATE>
static cudaError_t launch_bwd_gate(const SandwichBwdParams &p, const SandwichPlan &plan, cudaStream_t stream)
{
    // (a row is held while the next one is read: two stages)
    if (plan.stages < 2 || plan.groups * plan.W > kSwBwdManyWarps)
        return cudaErrorInvalidValue;
    const SandwichBuild b = sandwich_build(plan);
    cudaError_t e = cudaErrorInvalidValue; // no such build
    (void)(launch_build<GATE, 1, false, 1, true, false>(b, p, plan, stream, e) ||
           launch_build<GATE, 1, false, 1, true, true>(b, p, plan, stream, e) ||
           launch_build<GATE, 1, false, 8, true, true>(b, p, plan, stream, e) ||
           launch_build<GATE, 2, false, 1, false, false>(b, p, plan, stream, e) ||
           launch_build<GATE, 2, false, 8, false, false>(b, p, plan, stream, e) ||
           launch_build<GATE, 2, false, 8, true, false>(b, p, plan, stream, e) ||
           launch_build<GATE, 2, true, 8, false, false>(b, p, plan, stream, e) ||
           launch_build<GATE, 2, true, 16, false, false>(b, p, plan, stream, e) ||
           launch_build<GATE, 2, true, 16, true, false>(b, p, plan, stream, e));
    return e;
}

cudaError_t launch_sandwich_bwd(const SandwichBwdParams &p, const SandwichPlan &plan, cudaStream_t stream)
{
    switch (p.gate) {
    case 0: return launch_bwd_gate<0>(p, plan, stream);
    case 1: return launch_bwd_gate<1>(p, plan, stream);
    default: return launch_bwd_gate<2>(p, plan, stream);
    }
}

cudaError_t launch_sandwich_reduce(const SandwichReduceParams &p, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.H + 31) / 32), 2);
    cfg.blockDim = dim3(32 * kSwReduceWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, sandwich_reduce_kernel, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

} // namespace cake
