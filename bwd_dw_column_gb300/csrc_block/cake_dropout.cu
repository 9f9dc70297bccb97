// cake_dropout.cu -- dropout from a counter-based generator for sm_103a: alone,
// with a residual addition, and with the residual addition and the RMSNorm
// after it, forward and backward.
//
// The random bits of 8 neighbouring elements (a thread's 16-byte vector) are
// one block of Philox4x32-10 (Salmon, Moraes, Dror, Shaw 2011): ten rounds of
// two 32 x 32 -> 64 bit products.  Sixteen bits an element make that about 9
// instructions an element; with 32 it would be twice as much.  Nothing of the
// mask is stored or read, so HBM bounds every kernel here.
#include <type_traits>

#include "../csrc/cake_rows.cuh"
#include "cake_block_launch.h"

namespace cake {

// The generator's key and the counter's upper half.  DEV false: known to the
// host, with the keys of all rounds among the kernel's parameters, where the
// rounds take them as constants; DEV true: read from the device and counted up
// from round to round.
template <bool DEV>
struct Philox {
    const DropoutRng &r;
    uint32_t k0, k1, o0, o1;

    __device__ __forceinline__ explicit Philox(const DropoutRng &rng) : r(rng)
    {
        uint64_t seed = r.seed, off = r.offset;
        if (DEV) {
            seed = r.rng[0];
            off += r.rng[1];
        }
        k0 = (uint32_t)seed;
        k1 = (uint32_t)(seed >> 32);
        o0 = (uint32_t)off;
        o1 = (uint32_t)(off >> 32);
    }

    // 16 bits for each of the 8 elements of vector b, lowest first.
    __device__ __forceinline__ uint4 block(uint64_t b) const
    {
        uint32_t x = (uint32_t)b, y = (uint32_t)(b >> 32), z = o0, w = o1;
#pragma unroll
        for (int i = 0; i < 10; ++i) {
            const uint64_t p0 = (uint64_t)x * 0xD2511F53u, p1 = (uint64_t)z * 0xCD9E8D57u;
            x = (uint32_t)(p1 >> 32) ^ y ^ (DEV ? k0 + i * 0x9E3779B9u : r.keys[2 * i]);
            z = (uint32_t)(p0 >> 32) ^ w ^ (DEV ? k1 + i * 0xBB67AE85u : r.keys[2 * i + 1]);
            y = (uint32_t)p1;
            w = (uint32_t)p0;
        }
        return make_uint4(x, y, z, w);
    }
};

// The vector's bits, all zero where every element is dropped (cut = 65536).
template <bool DEV>
__device__ __forceinline__ uint4 random_bits(const Philox<DEV> &s, uint64_t b)
{
    return s.r.cut < 65536 ? s.block(b) : make_uint4(0, 0, 0, 0);
}

// scale * v where kept, 0 elsewhere; `limit` is the cut in the upper half of a word.
__device__ __forceinline__ float2 dropped(float2 v, uint32_t bits, uint32_t limit, float2 scale)
{
    v = mul2(v, scale);
    return make_float2((bits << 16) >= limit ? v.x : 0.f, bits >= limit ? v.y : 0.f);
}

__device__ __forceinline__ uint32_t limit_of(const DropoutRng &r) { return r.cut < 65536 ? r.cut << 16 : 0xffffffffu; }

// -------------------------------------------------------------------- alone

// A CTA takes 1024 neighbouring vectors at a time, four a thread.  SPACING says
// how they lie in memory: 0 in one block, 1 in equally spaced rows less than 2^31
// elements apart, 2 in any.  Rows come from one division for all of them and a
// product with a reciprocal for each (GB300, 16381 x 6144: 59 us in one block,
// spaced rows 69 us by 64-bit products of every row and column).
constexpr int kDropThreads = 256;
constexpr int kDropPer = 4;
constexpr uint32_t kDropVecs = kDropThreads * kDropPer;
constexpr uint64_t kDropCtas = 1 << 20;

// Where a CTA's vectors lie in a view.
template <int SPACING>
struct DropPlace {
    const RowView &v;
    const uint4 *first;   // 0: the first vector; 1: its row's begin
    uint32_t row0, nh;

    __device__ __forceinline__ DropPlace(const RowView &view, const DropoutParams &p, uint64_t v0, uint32_t row)
        : v(view), row0(row), nh(p.nh)
    {
        first = reinterpret_cast<const uint4 *>(view.base);
        if (SPACING == 0)
            first += v0;
        if (SPACING == 1)
            first += (int64_t)row * (view.row_stride / 8);
    }

    // Vector i of the CTA's: the col-th of the q-th row from row0 on.
    __device__ __forceinline__ uint4 *at(uint32_t i, uint32_t q, uint32_t col) const
    {
        const uint4 *a = SPACING == 0 ? first + i
                         : SPACING == 1
                             ? first + (uint64_t)q * (uint32_t)(v.row_stride / 8) + col
                             : first + row_off(v, row0 + q, nh) / 8 + col;
        return const_cast<uint4 *>(a);
    }
};

template <bool RES, int SPACING, bool DEV>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(const __grid_constant__ DropoutParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    const Philox<DEV> key(p.r);
    const uint32_t limit = limit_of(p.r);
    const float2 scale = make_float2(p.r.scale, p.r.scale);
    for (uint64_t v0 = (uint64_t)blockIdx.x * kDropVecs; v0 < p.vecs; v0 += (uint64_t)gridDim.x * kDropVecs) {
        uint32_t row0 = 0, rem = 0;
        if (SPACING) {
            row0 = v0 >> 32 ? (uint32_t)(v0 / p.nvec) : (uint32_t)v0 / p.nvec;
            rem = (uint32_t)(v0 - (uint64_t)row0 * p.nvec);
        }
        const uint32_t n = p.vecs - v0 < kDropVecs ? (uint32_t)(p.vecs - v0) : kDropVecs;
        const DropPlace<SPACING> px(p.x, p, v0, row0), pe(p.residual, p, v0, row0), py(p.y, p, v0, row0);
        uint4 x[kDropPer], e[kDropPer];
        uint32_t q_of[kDropPer], col_of[kDropPer];
#pragma unroll
        for (int k = 0; k < kDropPer; ++k) {
            const uint32_t i = k * kDropThreads + threadIdx.x;
            // (rem + i) / nvec: exact below 2^31 / nvec
            q_of[k] = SPACING ? __umulhi(2 * (rem + i), p.reciprocal) : 0;
            col_of[k] = SPACING ? rem + i - q_of[k] * p.nvec : 0;
            if (i < n) {
                x[k] = __ldcs(px.at(i, q_of[k], col_of[k]));
                if (RES)
                    e[k] = __ldcs(pe.at(i, q_of[k], col_of[k]));
            }
        }
#pragma unroll
        for (int k = 0; k < kDropPer; ++k) {
            const uint32_t i = k * kDropThreads + threadIdx.x;
            if (i >= n)
                break;
            const uint4 bits = random_bits(key, v0 + i);
            uint32_t o[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float2 v = dropped(bf2(word(x[k], q)), word(bits, q), limit, scale);
                if (RES)
                    v = add2(v, bf2(word(e[k], q)));
                o[q] = pack2(v);
            }
            __stcs(py.at(i, q_of[k], col_of[k]), make_uint4(o[0], o[1], o[2], o[3]));
        }
    }
}

// ------------------------------------------------------------ with the norm

// Both kernels stream rows through shared memory as the RMSNorm kernels do (a
// producer warp with bulk copies, row groups of W warps, bounded waits).
constexpr int kDnThreads = 544; // 16 consumer warps and the producer

// Tests of the waits: 16 bytes of the first stage that never come.
__device__ __forceinline__ void withhold_bytes(const Smem &s, int withhold)
{
    if (withhold && (threadIdx.x & 31) == 0)
        asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], 16;" ::"r"(smem_addr(&s.full[0])) : "memory");
    __syncwarp();
}

// LPR < 32: rows of LPR lanes, 32 / LPR of them to a warp, which is a row group
// of its own; otherwise a row spans a group's W warps.
template <int LPR>
struct RowLanes {
    static constexpr int kRows = 32 / LPR; // of a group's stage
    int sub, tid, stride; // the thread's row among the group's; its first vector, and the step to its next

    __device__ __forceinline__ RowLanes(int lane, int gtid, int W)
        : sub(LPR < 32 ? lane / LPR : 0), tid(LPR < 32 ? lane % LPR : gtid), stride(LPR < 32 ? LPR : 32 * W)
    {
    }

    // Sum over a row's threads; `abort` is joined over the group's.
    static __device__ __forceinline__ float sum(float v, const Smem &s, const Layout &L, int gid, int wig, int lane,
                                                uint32_t slot, bool &abort)
    {
        if constexpr (LPR == 32) {
            return group_sum(v, s, L, gid, wig, lane, slot, abort);
        } else {
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1)
                v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
            abort = __any_sync(0xffffffffu, abort);
            return v;
        }
    }
};

template <int VPT, int LPR, bool DEV>
__global__ void __launch_bounds__(kDnThreads, 2)
    dropout_norm_fwd_kernel(const __grid_constant__ DropoutNormParams p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const Layout &L = p.L;
    const Smem s = carve_smem(smem_raw, L);
    const Chunk c = cta_chunk(L);
    const int W = L.warps_per_row, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    init_ring(s, L);
    pdl_launch_dependents();
    pdl_wait();
    if (warp == L.groups * W) {
        const RowView views[2] = {p.in[0], p.in[1]};
        withhold_bytes(s, p.withhold);
        produce<2>(s, L, c, views, 2, p.status, p.wait_ns);
        return;
    }
    const int gid = warp / W, wig = warp - gid * W, gtid = wig * 32 + lane, nvec = L.nvec;
    const RowLanes<LPR> own(lane, gtid, W);
    const int vstride = own.stride, ltid = own.tid;
    const Philox<DEV> key(p.r);
    const uint32_t limit = limit_of(p.r);
    const float2 scale = make_float2(p.r.scale, p.r.scale);
    stage_weight(s, L, p.w, p.w_f32);
    bool abort = false;
    uint32_t slot = 0, st = 0, ph = 0;
    for (uint32_t it = 0; it < c.ntiles && !abort; ++it) {
        const int tr = gid * RowLanes<LPR>::kRows + own.sub;
        const uint32_t first = c.r0 + it * c.tile_rows + gid * RowLanes<LPR>::kRows, r = first + own.sub;
        uint4 bits[VPT]; // before the wait: they need no data
#pragma unroll
        for (int k = 0; k < VPT; ++k)
            bits[k] = random_bits(key, (uint64_t)r * nvec + k * vstride + ltid);
        abort = !mbar_wait(smem_addr(&s.full[st]), ph, p.wait_ns);
        if (first < c.r_end) { // uniform across the group
            const bool live = LPR == 32 || r < c.r_end;
            const uint8_t *stage = s.ring + st * s.stage_bytes + (size_t)tr * L.H * 2;
            const uint4 *xs = reinterpret_cast<const uint4 *>(stage);
            const uint4 *es = reinterpret_cast<const uint4 *>(stage + s.tens_bytes);
            uint4 h[VPT];
            float2 ss = make_float2(0.f, 0.f);
            uint4 *hrow = reinterpret_cast<uint4 *>(const_cast<uint16_t *>(p.out[1].base) + row_off(p.out[1], r, L.nh));
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = k * vstride + ltid;
                h[k] = make_uint4(0, 0, 0, 0);
                if (live && v < nvec) {
                    const uint4 x = xs[v], e = es[v];
                    uint32_t o[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        o[q] = pack2(add2(dropped(bf2(word(x, q)), word(bits[k], q), limit, scale),
                                          bf2(word(e, q))));
                        const float2 a = bf2(o[q]);
                        ss = fma2(a, a, ss);
                    }
                    h[k] = make_uint4(o[0], o[1], o[2], o[3]);
                    if (!abort)
                        __stcs(hrow + v, h[k]);
                }
            }
            const float tot = own.sum(__fadd_rn(ss.x, ss.y), s, L, gid, wig, lane, slot++, abort);
            const float rs = 1.0f / sqrtf(__fadd_rn(__fmul_rn(tot, L.inv_h), p.eps));
            const float2 rs2 = make_float2(rs, rs);
            uint4 *yrow = reinterpret_cast<uint4 *>(const_cast<uint16_t *>(p.out[0].base) + row_off(p.out[0], r, L.nh));
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = k * vstride + ltid;
                if (live && v < nvec && !abort) {
                    float2 w2[4];
                    weight_pairs(s, L, v, w2);
                    uint32_t o[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        o[q] = pack2(mul2(mul2(bf2(word(h[k], q)), rs2), w2[q]));
                    __stcs(yrow + v, make_uint4(o[0], o[1], o[2], o[3]));
                }
            }
            if (live && ltid == 0 && !abort)
                p.rstd_out[r] = rs;
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(smem_addr(&s.empty[st]));
        if (++st == (uint32_t)L.stages) {
            st = 0;
            ph ^= 1u;
        }
    }
    if (abort && lane == 0)
        set_status(p.status, kStatusTimeout);
}

// A thread holds 8 VPT columns of a row.  Its terms of dw are added over 16 rows
// in registers and then to Kahan pairs in shared memory that only it uses.  With
// hh = h rstd, a = dy w and m = mean of a hh the gradient is
//   t = dh + rstd (a - hh m),
// in this order: rstd^2 is beyond FP32 for rows below 1e-19 (eps = 0).
constexpr int kDnBlock = 16;

__device__ __forceinline__ void fold_columns(float4 *at, int step, float2 (&sum)[4])
{
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float4 &v = at[q * step]; // two columns' sums, and what they have not taken up
        const float2 hi = make_float2(v.x, v.y), y = add2(sum[q], make_float2(v.z, v.w)), t = add2(hi, y),
                     lo = add2(sub2(hi, t), y);
        v = make_float4(t.x, t.y, lo.x, lo.y);
        sum[q] = make_float2(0.f, 0.f);
    }
}

template <int VPT, int LPR, bool DH, bool DEV>
__global__ void __launch_bounds__(kDnThreads, 1)
    dropout_norm_bwd_kernel(const __grid_constant__ DropoutNormParams p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const Layout &L = p.L;
    const Smem s = carve_smem(smem_raw, L);
    const Chunk c = cta_chunk(L);
    const int W = L.warps_per_row, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    init_ring(s, L);
    pdl_launch_dependents();
    pdl_wait();
    if (warp == L.groups * W) {
        const RowView views[3] = {p.in[0], p.in[1], p.in[2]};
        withhold_bytes(s, p.withhold);
        produce<3>(s, L, c, views, L.ntens, p.status, p.wait_ns);
        return;
    }
    const int gid = warp / W, wig = warp - gid * W, gtid = wig * 32 + lane, nvec = L.nvec;
    const RowLanes<LPR> own(lane, gtid, W);
    const int vstride = own.stride, ltid = own.tid, tr = gid * RowLanes<LPR>::kRows + own.sub;
    const int nct = L.groups * W * 32;
    const Philox<DEV> key(p.r);
    const uint32_t limit = limit_of(p.r);
    const float2 scale = make_float2(p.r.scale, p.r.scale);
    stage_weight(s, L, p.w, p.w_f32);
    float4 *const sums = s.lo + threadIdx.x; // [VPT][4][consumer threads]
    float2 acc[VPT][4];
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            acc[k][q] = make_float2(0.f, 0.f);
            sums[(4 * k + q) * nct] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    bool abort = false;
    uint32_t slot = 0, st = 0, ph = 0;
    for (uint32_t it = 0; it < c.ntiles && !abort; ++it) {
        const uint32_t first = c.r0 + it * c.tile_rows + gid * RowLanes<LPR>::kRows, r = first + own.sub;
        const float rs = r < c.r_end ? __ldg(p.rstd + r) : 0.f;
        uint4 bits[VPT]; // before the wait: they need no data
#pragma unroll
        for (int k = 0; k < VPT; ++k)
            bits[k] = random_bits(key, (uint64_t)r * nvec + k * vstride + ltid);
        abort = !mbar_wait(smem_addr(&s.full[st]), ph, p.wait_ns);
        if (first < c.r_end) { // uniform across the group
            const bool live = LPR == 32 || r < c.r_end;
            const uint8_t *stage = s.ring + st * s.stage_bytes + (size_t)tr * L.H * 2;
            const uint4 *hs = reinterpret_cast<const uint4 *>(stage);
            const uint4 *ds = reinterpret_cast<const uint4 *>(stage + s.tens_bytes);
            const uint4 *es = reinterpret_cast<const uint4 *>(stage + 2 * s.tens_bytes);
            const float2 rs2 = make_float2(rs, rs);
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = k * vstride + ltid;
                if (live && v < nvec) {
                    const uint4 h = hs[v], d = ds[v];
                    float2 w2[4];
                    weight_pairs(s, L, v, w2);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float2 dq = bf2(word(d, q)), hh = mul2(bf2(word(h, q)), rs2);
                        sum = fma2(mul2(dq, w2[q]), hh, sum);
                        acc[k][q] = fma2(hh, dq, acc[k][q]);
                    }
                }
            }
            const float tot = own.sum(__fadd_rn(sum.x, sum.y), s, L, gid, wig, lane, slot++, abort);
            const float m = -__fmul_rn(tot, L.inv_h);
            const float2 m2 = make_float2(m, m);
            uint4 *xrow = reinterpret_cast<uint4 *>(const_cast<uint16_t *>(p.out[0].base) + row_off(p.out[0], r, L.nh));
            uint4 *erow = reinterpret_cast<uint4 *>(const_cast<uint16_t *>(p.out[1].base) + row_off(p.out[1], r, L.nh));
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = k * vstride + ltid;
                if (live && v < nvec && !abort) {
                    const uint4 h = hs[v], d = ds[v];
                    uint4 e = make_uint4(0, 0, 0, 0);
                    if (DH)
                        e = es[v];
                    float2 w2[4];
                    weight_pairs(s, L, v, w2);
                    uint32_t ox[4], oe[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float2 a = mul2(bf2(word(d, q)), w2[q]);
                        float2 t = fma2(mul2(bf2(word(h, q)), rs2), m2, a);
                        t = DH ? fma2(rs2, t, bf2(word(e, q))) : mul2(rs2, t);
                        oe[q] = pack2(t);
                        ox[q] = pack2(dropped(t, word(bits[k], q), limit, scale));
                    }
                    __stcs(xrow + v, make_uint4(ox[0], ox[1], ox[2], ox[3]));
                    __stcs(erow + v, make_uint4(oe[0], oe[1], oe[2], oe[3]));
                }
            }
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(smem_addr(&s.empty[st]));
        if (++st == (uint32_t)L.stages) {
            st = 0;
            ph ^= 1u;
        }
        if (it % kDnBlock == kDnBlock - 1)
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                fold_columns(sums + 4 * k * nct, nct, acc[k]);
    }
    if (abort && lane == 0)
        set_status(p.status, kStatusTimeout);
    // The CTA partial: the rows' sums in their order, through the drained ring
    // ([row of a stage][4 nvec] float4 (hi, lo, hi, lo) of a column pair).
    const int nslot = 4 * nvec;
    float4 *comb = reinterpret_cast<float4 *>(s.ring);
    consumer_sync(L);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int v = k * vstride + ltid;
        fold_columns(sums + 4 * k * nct, nct, acc[k]);
        if (v < nvec)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 f = sums[(4 * k + q) * nct];
                comb[(size_t)tr * nslot + 4 * v + q] = make_float4(f.x, f.z, f.y, f.w);
            }
    }
    consumer_sync(L);
    for (int i = threadIdx.x; i < nslot; i += nct) {
        float4 a = comb[i];
        for (int g = 1; g < L.groups * RowLanes<LPR>::kRows; ++g) {
            const float4 b = comb[(size_t)g * nslot + i];
            comp_add(a.x, a.y, b.x);
            a.y = __fadd_rn(a.y, b.y);
            comp_add(a.z, a.w, b.z);
            a.w = __fadd_rn(a.w, b.w);
        }
        reinterpret_cast<float4 *>(p.partials + (size_t)blockIdx.x * L.H)[i] = a;
    }
}

// Column sums of the CTAs' partials in CTA order: a warp takes 32 columns and
// every 32nd CTA, with several of its loads on their way at once; the 32 sums
// of a column are then added in warp order.
constexpr int kColumnWarps = 32;
constexpr int kColumnAhead = 8;

__global__ void __launch_bounds__(32 * kColumnWarps) column_sum_kernel(const __grid_constant__ ColumnSumParams p)
{
    __shared__ float2 part[kColumnWarps][32];
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, list = blockIdx.y;
    const int j = blockIdx.x * 32 + lane;
    float hi = 0.f, lo = 0.f;
    if (j < p.H)
        for (int q0 = warp; q0 < p.P[list]; q0 += kColumnAhead * kColumnWarps) {
            float2 v[kColumnAhead];
#pragma unroll
            for (int i = 0; i < kColumnAhead; ++i) {
                const int q = q0 + i * kColumnWarps;
                v[i] = q < p.P[list] ? __ldcg(p.partials[list] + (size_t)q * p.H + j) : make_float2(0.f, 0.f);
            }
#pragma unroll
            for (int i = 0; i < kColumnAhead; ++i) {
                comp_add(hi, lo, v[i].x);
                lo = __fadd_rn(lo, v[i].y);
            }
        }
    part[warp][lane] = make_float2(hi, lo);
    __syncthreads();
    if (warp == 0 && j < p.H) {
        for (int w = 1; w < kColumnWarps; ++w) {
            comp_add(hi, lo, part[w][lane].x);
            lo = __fadd_rn(lo, part[w][lane].y);
        }
        p.out[list][j] = __fadd_rn(hi, lo);
    }
}

// ------------------------------------------------------------------- launch

// Shared memory of a plan's CTA for its vpt, lanes, W and groups; false: no two stages fit.
static bool fit_plan(DropoutNormPlan &p, int H, int ntens, bool backward)
{
    p.lo_bytes = backward ? p.vpt * 64 * p.groups * p.W * 32 : 0;
    const size_t fixed = kMiscBytes + weight_smem_bytes(H) + p.lo_bytes, rows = (size_t)p.groups * (32 / p.lanes),
                 stage = (size_t)ntens * rows * H * 2;
    p.per_sm = backward || rows * H >= 7000 ? 1 : 2;
    for (;; --p.per_sm) {
        const size_t room = 228 * 1024 / p.per_sm - 1024; // 1 KB of each CTA is the system's
        p.stages = room > fixed ? (int)((room - fixed) / stage) : 0;
        if (p.stages >= 2 || p.per_sm == 1)
            break;
    }
    // The forward runs one CTA an SM with three stages where that has 7000
    // columns or more in work, else two with two stages, or what brings 48 KB on
    // their way: GB300, 2^26 values (the copy takes 80 us), one and two CTAs:
    // H = 4096 83 and 96 us, H = 1024 83 and 95, H = 8192 84 and 91, but H = 6144
    // 94 and 86, H = 5120 150 and 89, H = 256 113 and 92.
    const int least = backward ? 6 : p.per_sm == 1 ? 3 : 2;
    int most = (int)((48 * 1024 + stage - 1) / stage);
    most = most > least ? most : least;
    most = most > 16 ? 16 : most;
    if (p.stages > most)
        p.stages = most;
    size_t ring = p.stages * stage;
    if (backward && ring < rows * H * 8) // the rows' column sums pass through it
        ring = rows * H * 8;
    p.smem = fixed + ring;
    return p.stages >= 2 && p.smem <= 227 * 1024;
}

// The shape of a CTA goes by H and the staged tensors alone, so the orders of
// the sums do too: the most columns in work up to the 6144 that keep HBM busy,
// those of a single row group (whose warps wait for one sum together) and of
// less than three stages counted less; of equals the fewest columns a thread.
DropoutNormPlan dropout_norm_plan(int H, uint32_t rows, int ntens, bool backward)
{
    const int nvec = H / 8;
    DropoutNormPlan p{};
    int best = -1;
    for (int vpt = 1; vpt <= (backward ? 3 : 2); ++vpt) {
        const int W = (nvec + 32 * vpt - 1) / (32 * vpt);
        for (int groups = 16 / W < kMaxRowGroupBarriers ? 16 / W : kMaxRowGroupBarriers; groups >= 1; --groups) {
            DropoutNormPlan q{};
            q.vpt = vpt;
            q.lanes = H <= 32 ? 4 : H <= 64 ? 8 : H <= 128 ? 16 : 32;
            q.W = W;
            q.groups = groups;
            if (!fit_plan(q, H, ntens, backward))
                continue;
            int score = groups * (32 / q.lanes) * H;
            score = score > 6144 ? 6144 : score;
            score = groups == 1 ? score * 8 / 10 : score;
            score = q.stages < 3 ? score * 85 / 100 : score;
            if (score > best) {
                best = score;
                p = q;
            }
        }
    }
    const uint32_t tile = (uint32_t)p.groups * (32 / p.lanes), tiles = (rows + tile - 1) / tile, most = (uint32_t)(kSMsBlock * p.per_sm);
    const uint32_t ctas = tiles < most ? tiles : most;
    p.rows_per_cta = ctas ? (rows + ctas - 1) / ctas : 0;
    p.ctas = p.rows_per_cta ? (int)((rows + p.rows_per_cta - 1) / p.rows_per_cta) : 0;
    return p;
}

cudaError_t launch_dropout(const DropoutParams &p, cudaStream_t stream)
{
    const uint64_t want = (p.vecs + kDropVecs - 1) / kDropVecs;
    const dim3 grid((unsigned)(want < kDropCtas ? want : kDropCtas));
    int spacing = 0;
    for (const RowView *v : {&p.x, &p.residual, &p.y})
        if (v->base) {
            const int own = v->dense ? 0 : v->uniform && v->row_stride < (int64_t(1) << 31) ? 1 : 2;
            spacing = own > spacing ? own : spacing;
        }
    const auto go = [&](auto dev) {
        constexpr bool D = decltype(dev)::value;
        auto kern = p.residual.base ? (spacing == 0   ? dropout_kernel<true, 0, D>
                                       : spacing == 1 ? dropout_kernel<true, 1, D>
                                                      : dropout_kernel<true, 2, D>)
                                    : (spacing == 0   ? dropout_kernel<false, 0, D>
                                       : spacing == 1 ? dropout_kernel<false, 1, D>
                                                      : dropout_kernel<false, 2, D>);
        return launch_after(kern, grid, kDropThreads, 0, stream, p);
    };
    return p.r.rng ? go(std::true_type()) : go(std::false_type());
}

cudaError_t launch_dropout_norm_fwd(const DropoutNormParams &p, const DropoutNormPlan &plan, cudaStream_t stream)
{
    const int threads = 32 * (plan.groups * plan.W + 1);
    const auto go = [&](auto dev) {
        constexpr bool D = decltype(dev)::value;
        auto kern = plan.lanes == 4    ? dropout_norm_fwd_kernel<1, 4, D>
                    : plan.lanes == 8  ? dropout_norm_fwd_kernel<1, 8, D>
                    : plan.lanes == 16 ? dropout_norm_fwd_kernel<1, 16, D>
                    : plan.vpt == 1    ? dropout_norm_fwd_kernel<1, 32, D>
                                       : dropout_norm_fwd_kernel<2, 32, D>;
        return launch_after(kern, dim3((unsigned)plan.ctas), threads, plan.smem, stream, p);
    };
    return p.r.rng ? go(std::true_type()) : go(std::false_type());
}

cudaError_t launch_dropout_norm_bwd(const DropoutNormParams &p, const DropoutNormPlan &plan, cudaStream_t stream)
{
    const int threads = 32 * (plan.groups * plan.W + 1);
    const auto go = [&](auto dev, auto dh) {
        constexpr bool D = decltype(dev)::value, E = decltype(dh)::value;
        auto kern = plan.lanes == 4    ? dropout_norm_bwd_kernel<1, 4, E, D>
                    : plan.lanes == 8  ? dropout_norm_bwd_kernel<1, 8, E, D>
                    : plan.lanes == 16 ? dropout_norm_bwd_kernel<1, 16, E, D>
                    : plan.vpt == 1    ? dropout_norm_bwd_kernel<1, 32, E, D>
                    : plan.vpt == 2    ? dropout_norm_bwd_kernel<2, 32, E, D>
                                       : dropout_norm_bwd_kernel<3, 32, E, D>;
        return launch_after(kern, dim3((unsigned)plan.ctas), threads, plan.smem, stream, p);
    };
    if (p.L.ntens == 3)
        return p.r.rng ? go(std::true_type(), std::true_type()) : go(std::false_type(), std::true_type());
    return p.r.rng ? go(std::true_type(), std::false_type()) : go(std::false_type(), std::false_type());
}

cudaError_t launch_column_sum(const ColumnSumParams &p, int lists, cudaStream_t stream)
{
    return launch_after(column_sum_kernel, dim3((unsigned)((p.H + 31) / 32), (unsigned)lists), 32 * kColumnWarps, 0,
                        stream, p);
}

} // namespace cake
