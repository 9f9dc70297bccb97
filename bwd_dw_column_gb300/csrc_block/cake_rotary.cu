// cake_rotary.cu -- the per-head norm of queries and keys with rotary positions
// of several axes for sm_103a, forward and backward.
//
// A row (a token's head) lies on LANES lanes of two 16-byte vectors each, so
// that both members of every rotated pair are a lane's own (rotary_lane).  A
// lane group walks over a token's heads, so a lane computes the sine and cosine
// of its 8 pairs once for all of them.  The angle
// is a product modulo 2^64 in units of 2^-64 turn, whole turns drop out of it
// exactly, and a sine and cosine of its upper half remain.
//
// HBM bounds both kernels: every value is read and written once (GB300, 32768
// tokens of 24 + 4 heads of 256, a quarter rotated: forward 150 us, 0.94 of the
// copy rate, backward 221, 0.96).  A thread copies its vectors of the rows ahead into slots of shared memory that only it
// reads (cp.async, so no barrier and no registers are held by what is on its
// way).
#include "../csrc/cake_rows.cuh"
#include "cake_block_launch.h"

namespace cake {

constexpr int kRotThreads = 256;
constexpr int kRotWarps = kRotThreads / 32;
constexpr int kRotFwdDepth = 4, kRotBwdDepth = 3; // rows on their way
constexpr int kStatusInvalid = 1; // == CAKE_ERR_INVALID

// ------------------------------------------------------------ copies ahead

__device__ __forceinline__ void copy16(uint32_t dst, const uint16_t *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 slot16(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// ------------------------------------------------------------- a lane's part

// A lane's columns a .. a + 7 and b .. b + 7.  Of adjacent pairs these are
// vector l of either half of the row, with four pairs in each; of the half
// style, while there are rotated columns, a vector of the first and the one of
// the second half of them that it pairs with, and beyond those a vector of
// either half of the rest.
struct RotaryLane {
    bool live, rot_a, rot_b; // has columns; rotates them
    int a, b;
    int pair_a, pair_b;      // the first pair of the lane's first and second four
    uint32_t axes;           // of its pairs, 4 bits each
};

template <bool ADJ>
__device__ __forceinline__ RotaryLane rotary_lane(const RotaryParams &p, int l)
{
    RotaryLane m;
    const int n = p.D / 16, r = p.pairs / 8;
    m.live = l < n;
    if (ADJ) {
        m.a = 8 * l;
        m.b = 8 * (n + l);
        m.rot_a = m.live && l < 2 * r;
        m.rot_b = m.live && n + l < 2 * r;
        m.pair_a = 4 * l;
        m.pair_b = 4 * (n + l);
    } else {
        m.rot_a = m.rot_b = l < r;
        m.a = m.rot_a ? 8 * l : 8 * (r + l);
        m.b = m.rot_a ? 8 * (r + l) : 8 * (n + l);
        m.pair_a = 8 * l;
        m.pair_b = 8 * l + 4;
    }
    m.axes = 0;
    if (p.axis)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int32_t x = (i < 4 ? m.rot_a : m.rot_b) ? __ldg(p.axis + (i < 4 ? m.pair_a : m.pair_b - 4) + i) : 0;
            if (x >= 0 && x < p.axes)
                m.axes |= (uint32_t)x << (4 * i);
        }
    return m;
}

// What the lanes of a group share: each one's weights as FP32 (two vectors) and
// its pairs' turns, in shared memory.
struct RotaryShared {
    float4 w[4][32];
    ulonglong2 turns[4][32];
};

// Fills it; the CTA's threads meet before they read.
template <int LANES>
__device__ __forceinline__ void rotary_shared(const RotaryParams &p, const RotaryList &l, const RotaryLane &m,
                                              RotaryShared &sh)
{
    const int i = threadIdx.x;
    if (i < LANES) {
        float w[16];
        uint64_t t[8];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int j = (k < 8 ? m.a : m.b - 8) + k;
            w[k] = !l.w || !m.live ? 0.f
                   : l.w_f32       ? __ldg(static_cast<const float *>(l.w) + j)
                                   : __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t *>(l.w) + j) << 16);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const bool rot = k < 4 ? m.rot_a : m.rot_b;
            const int pair = (k < 4 ? m.pair_a : m.pair_b - 4) + k;
            t[k] = rot ? __ldg(p.turns + pair) : 0;
            if (rot && p.axis) {
                const int32_t x = __ldg(p.axis + pair);
                if (x < 0 || x >= p.axes) { // no such axis: the pair is not turned
                    t[k] = 0;
                    set_status(p.status + 1, kStatusInvalid);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            sh.w[k][i] = make_float4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
            sh.turns[k][i] = make_ulonglong2(t[2 * k], t[2 * k + 1]);
        }
    }
    __syncthreads();
}

__device__ __forceinline__ uint64_t position(const RotaryParams &p, uint32_t axis, uint32_t t)
{
    const int64_t at = (int64_t)axis * p.axis_stride + (int64_t)t * p.token_stride;
    return p.pos_i64 ? (uint64_t)__ldg(static_cast<const long long *>(p.positions) + at)
                     : (uint64_t)(int64_t)__ldg(static_cast<const int *>(p.positions) + at);
}

// Sine and cosine of 2 pi phase / 2^32: the eighths of a turn on either side of
// a quarter by their power series about it (|x| <= pi / 4: up to x^9 and x^8,
// the next terms are 1.8e-9 and 2.5e-8), turned on by whole quarters.  The phase
// is exact, so this needs half the instructions of a general sine and cosine,
// which the keys' few heads a token have to pay for.
__device__ __forceinline__ void turn_sincos(int32_t phase, float sign, float &sine, float &cosine)
{
    const int32_t q = (int32_t)((uint32_t)phase + 0x20000000u) >> 30; // the nearest quarter, -2 .. 1
    const float x = (float)(int32_t)((uint32_t)phase - ((uint32_t)q << 30)) * 1.46291807926715968e-9f; // 2 pi / 2^32
    const float y = x * x;
    float s = fmaf(y, 1.0f / 362880.0f, -1.0f / 5040.0f);
    s = fmaf(y, s, 1.0f / 120.0f);
    s = fmaf(y, s, -1.0f / 6.0f);
    s = fmaf(x * y, s, x);
    float c = fmaf(y, 1.0f / 40320.0f, -1.0f / 720.0f);
    c = fmaf(y, c, 1.0f / 24.0f);
    c = fmaf(y, c, -0.5f);
    c = fmaf(y, c, 1.0f);
    const float a = q & 1 ? c : s, b = q & 1 ? s : c;
    // quarters 1 and 2 turn the cosine's sign, 2 and 3 the sine's
    sine = __uint_as_float(__float_as_uint(a) ^ ((uint32_t)(q & 2) << 30)) * sign;
    cosine = __uint_as_float(__float_as_uint(b) ^ ((uint32_t)((q + 1) & 2) << 30));
}

// A token's positions on their way: with several axes lane x of the group holds
// that of axis x (more axes than lanes are loaded where they are needed), else
// every lane the only one.
template <int LANES>
__device__ __forceinline__ uint64_t load_positions(const RotaryParams &p, uint32_t t)
{
    const uint32_t l = threadIdx.x % LANES;
    return t < p.tokens && p.turns ? position(p, p.axis && l < (uint32_t)p.axes ? l : 0, t) : 0;
}

// Cosines and sines of the lane's pairs at token t, in twos; `sign` -1: turned
// backwards.  The whole warp takes part.
template <int LANES>
__device__ __forceinline__ void rotary_angles(const RotaryParams &p, const RotaryShared &sh, const RotaryLane &m,
                                              uint32_t t, uint64_t positions, float sign, float2 (&c)[4],
                                              float2 (&s)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const ulonglong2 turns = sh.turns[i][threadIdx.x % LANES];
        uint64_t at[2] = {positions, positions};
        if (p.axis)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t x = (m.axes >> (4 * (2 * i + k))) & 15u;
                at[k] = __shfl_sync(0xffffffffu, (unsigned long long)positions, (int)x, LANES);
                if (p.axes > LANES && t < p.tokens)
                    at[k] = position(p, x, t);
            }
        turn_sincos((int32_t)((turns.x * at[0]) >> 32), sign, s[i].x, c[i].x); // 2^-32 turns
        turn_sincos((int32_t)((turns.y * at[1]) >> 32), sign, s[i].y, c[i].y);
    }
}

// a, b: the lane's two vectors in twos of columns.
template <bool ADJ>
__device__ __forceinline__ void rotate(const RotaryLane &m, float2 (&a)[4], float2 (&b)[4], const float2 (&c)[4],
                                       const float2 (&s)[4])
{
    if constexpr (ADJ) {
        auto one = [](float2 v, float cos, float sin) {
            return fma2(v, make_float2(cos, cos), mul2(make_float2(v.y, v.x), make_float2(-sin, sin)));
        };
        if (m.rot_a)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                a[i] = one(a[i], i & 1 ? c[i / 2].y : c[i / 2].x, i & 1 ? s[i / 2].y : s[i / 2].x);
        if (m.rot_b)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                b[i] = one(b[i], i & 1 ? c[2 + i / 2].y : c[2 + i / 2].x, i & 1 ? s[2 + i / 2].y : s[2 + i / 2].x);
    } else if (m.rot_a) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = a[i], y = b[i];
            a[i] = fma2(x, c[i], mul2(y, make_float2(-s[i].x, -s[i].y)));
            b[i] = fma2(y, c[i], mul2(x, s[i]));
        }
    }
}

__device__ __forceinline__ void unpack(const uint4 &v, float2 (&f)[4])
{
#pragma unroll
    for (int q = 0; q < 4; ++q)
        f[q] = bf2(word(v, q));
}

__device__ __forceinline__ void store_row(uint16_t *row, const RotaryLane &m, const float2 (&a)[4],
                                          const float2 (&b)[4])
{
    if (!m.live)
        return;
    __stcs(reinterpret_cast<uint4 *>(row + m.a), make_uint4(pack2(a[0]), pack2(a[1]), pack2(a[2]), pack2(a[3])));
    __stcs(reinterpret_cast<uint4 *>(row + m.b), make_uint4(pack2(b[0]), pack2(b[1]), pack2(b[2]), pack2(b[3])));
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v)
{
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
        v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// The CTA's list, and its index among that list's CTAs.
__device__ __forceinline__ const RotaryList &cta_list(const RotaryParams &p, uint32_t &cta)
{
    const bool keys = blockIdx.x >= (unsigned)p.l[0].ctas;
    cta = keys ? blockIdx.x - p.l[0].ctas : blockIdx.x;
    return p.l[keys];
}

// A step is one head of as many neighbouring tokens as a warp has lane groups;
// a list's steps run over the heads, then over the tokens.  The CTAs go over
// them together, a run of some tokens' steps for each warp at a time, so that
// what all of them read stays close together; what is left after the last whole
// round is shared out evenly.  (Lane groups beyond
// the last token work on zeros, so that every shuffle finds the whole warp.)
template <int LANES>
struct RotaryWalk {
    static constexpr uint32_t kTokens = 32 / LANES;
    uint32_t t, h;         // this lane group's token, and the head
    uint32_t left, round;  // steps of this run, its round

    // The warp's part of the steps after the last whole round.
    static __device__ __forceinline__ uint32_t rest(const RotaryParams &p, const RotaryList &L, uint32_t w,
                                                    uint32_t &first)
    {
        const uint32_t warps = (uint32_t)L.ctas * kRotWarps, begin = L.rounds * warps * L.run * L.heads;
        const uint32_t total = (p.tokens + kTokens - 1) / kTokens * L.heads - begin;
        const uint32_t per = total / warps, more = total - per * warps;
        first = begin + w * per + min(w, more);
        return per + (w < more);
    }

    __device__ __forceinline__ void start(const RotaryParams &p, const RotaryList &L, uint32_t w)
    {
        const uint32_t sub = (threadIdx.x & 31) / LANES;
        if (round < L.rounds) {
            t = (round * (uint32_t)L.ctas * kRotWarps + w) * L.run * kTokens + sub;
            h = 0;
            left = L.run * L.heads;
        } else {
            uint32_t first;
            left = rest(p, L, w, first);
            t = first / L.heads * kTokens + sub;
            h = first % L.heads;
        }
    }

    // The token after this one.
    __device__ __forceinline__ uint32_t next_token(const RotaryParams &p, const RotaryList &L, uint32_t w) const
    {
        if (left > L.heads - h)
            return t + kTokens;
        RotaryWalk n = *this;
        n.round = round + 1;
        if (n.round > L.rounds)
            return p.tokens;
        n.start(p, L, w);
        return n.t;
    }

    // To the next step; true where that is not the next head of the same token.
    __device__ __forceinline__ bool next(const RotaryParams &p, const RotaryList &L, uint32_t w)
    {
        bool jump = false;
        if (++h == L.heads) {
            h = 0;
            t += kTokens;
            jump = true;
        }
        if (--left == 0 && round < L.rounds) {
            ++round;
            start(p, L, w);
            jump = true;
        }
        return jump;
    }
};

__device__ __forceinline__ const uint16_t *row_at(const RowView &v, uint32_t t, uint32_t h)
{
    return v.base + (int64_t)t * v.st + (int64_t)h * v.sh;
}

template <int LANES, bool ADJ, bool NORM>
__global__ void __launch_bounds__(kRotThreads, 2) rotary_kernel(const __grid_constant__ RotaryParams p, float sign)
{
    extern __shared__ __align__(16) uint4 slots_raw[];
    pdl_launch_dependents();
    pdl_wait();
    uint32_t cta, none;
    const RotaryList &L = cta_list(p, cta);
    const RotaryLane m = rotary_lane<ADJ>(p, threadIdx.x % LANES);
    const uint32_t w = cta * kRotWarps + (threadIdx.x >> 5);
    const uint32_t steps = L.rounds * L.run * L.heads + RotaryWalk<LANES>::rest(p, L, w, none);
    RotaryWalk<LANES> at, ahead;
    at.round = 0;
    at.start(p, L, w);
    ahead = at;
    uint32_t left = steps;
    const uint32_t mine = smem_addr(slots_raw + threadIdx.x);
    constexpr uint32_t kHalf = kRotThreads * 16, kStage = 2 * kHalf;
    const uint16_t *in = row_at(L.in, at.t, at.h), *out = row_at(L.out, at.t, at.h);
    auto fetch = [&](uint32_t stage) {
        if (left > 0) {
            if (m.live && ahead.t < p.tokens) {
                copy16(mine + stage * kStage, in + m.a);
                copy16(mine + stage * kStage + kHalf, in + m.b);
            }
            --left;
            if (ahead.next(p, L, w))
                in = row_at(L.in, ahead.t, ahead.h);
            else
                in += L.in.sh;
        }
        copies_commit();
    };
#pragma unroll
    for (int i = 0; i < kRotFwdDepth - 1; ++i)
        fetch(i);
    uint64_t positions = load_positions<LANES>(p, at.t);
    RotaryShared &sh = *reinterpret_cast<RotaryShared *>(slots_raw + kRotFwdDepth * 2 * kRotThreads);
    rotary_shared<LANES>(p, L, m, sh);
    float2 wa[4], wb[4];
    if constexpr (NORM)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = sh.w[i][threadIdx.x % LANES];
            (i < 2 ? wa : wb)[2 * (i & 1)] = make_float2(v.x, v.y);
            (i < 2 ? wa : wb)[2 * (i & 1) + 1] = make_float2(v.z, v.w);
        }
    float2 c[4], s[4];
    bool jump = true; // another token than the step before
    for (uint32_t n = 0, stage = 0; n < steps; ++n, stage = (stage + 1) % kRotFwdDepth) {
        fetch((stage + kRotFwdDepth - 1) % kRotFwdDepth);
        const bool row = at.t < p.tokens;
        if (jump) {
            rotary_angles<LANES>(p, sh, m, at.t, positions, sign, c, s);
            positions = load_positions<LANES>(p, at.next_token(p, L, w));
        }
        copies_wait<kRotFwdDepth - 1>();
        uint4 va = make_uint4(0, 0, 0, 0), vb = va;
        if (row && m.live) {
            va = slot16(mine + stage * kStage);
            vb = slot16(mine + stage * kStage + kHalf);
        }
        float2 a[4], b[4];
        unpack(va, a);
        unpack(vb, b);
        if constexpr (NORM) {
            float2 ss = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                ss = fma2(b[i], b[i], fma2(a[i], a[i], ss));
            const float sum = lanes_sum<LANES>(__fadd_rn(ss.x, ss.y));
            const float rs = 1.0f / sqrtf(__fmaf_rn(sum, p.inv_d, p.eps));
            const float2 rs2 = make_float2(rs, rs);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = mul2(mul2(a[i], rs2), wa[i]);
                b[i] = mul2(mul2(b[i], rs2), wb[i]);
            }
            if (row && threadIdx.x % LANES == 0)
                L.rstd_out[(size_t)at.t * L.heads + at.h] = rs;
        }
        if (row) {
            rotate<ADJ>(m, a, b, c, s);
            store_row(const_cast<uint16_t *>(out), m, a, b);
        }
        jump = at.next(p, L, w);
        if (jump)
            out = row_at(L.out, at.t, at.h);
        else
            out += L.out.sh;
    }
}

// Backward with a norm.  A lane adds its 16 columns' terms of dw over 16 rows in
// registers and then to Kahan pairs in shared memory that only it uses: pairs in
// registers took 32 of them and 24 instructions a row more, and the spills that
// this cost went to L2 (GB300, 8192 tokens of 24 + 4 heads of 256: 148 us).
constexpr uint32_t kRotBlock = 16;

__device__ __forceinline__ void fold(uint32_t at, float2 (&sum)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t to = at + i * kRotThreads * 16;
        const float4 v = ld_shared_f4(to); // two columns' sums, and what they have not taken up
        const float2 hi = make_float2(v.x, v.y), y = add2(sum[i], make_float2(v.z, v.w)), t = add2(hi, y),
                     lo = add2(sub2(hi, t), y);
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(t.x), "f"(t.y), "f"(lo.x), "f"(lo.y)
                     : "memory");
        sum[i] = make_float2(0.f, 0.f);
    }
}

template <int LANES, bool ADJ>
__global__ void __launch_bounds__(kRotThreads, 2) rotary_bwd_kernel(const __grid_constant__ RotaryParams p)
{
    // the slots (later the warps' sums [warps][D] (hi, lo)), the threads' column sums, what they share
    extern __shared__ __align__(16) uint4 slots_raw[];
    pdl_launch_dependents();
    pdl_wait();
    uint32_t cta, none;
    const RotaryList &L = cta_list(p, cta);
    const RotaryLane m = rotary_lane<ADJ>(p, threadIdx.x % LANES);
    const uint32_t w = cta * kRotWarps + (threadIdx.x >> 5);
    const uint32_t steps = L.rounds * L.run * L.heads + RotaryWalk<LANES>::rest(p, L, w, none);
    RotaryWalk<LANES> at, ahead;
    at.round = 0;
    at.start(p, L, w);
    ahead = at;
    uint32_t left = steps;
    const uint32_t mine = smem_addr(slots_raw + threadIdx.x);
    constexpr uint32_t kQuarter = kRotThreads * 16, kStage = 4 * kQuarter;
    const uint16_t *dy = row_at(L.in, at.t, at.h), *v = row_at(L.v, at.t, at.h), *out = row_at(L.out, at.t, at.h);
    auto fetch = [&](uint32_t stage) {
        if (left > 0) {
            if (m.live && ahead.t < p.tokens) {
                const uint32_t to = mine + stage * kStage;
                copy16(to, dy + m.a);
                copy16(to + kQuarter, dy + m.b);
                copy16(to + 2 * kQuarter, v + m.a);
                copy16(to + 3 * kQuarter, v + m.b);
            }
            --left;
            if (ahead.next(p, L, w)) {
                dy = row_at(L.in, ahead.t, ahead.h);
                v = row_at(L.v, ahead.t, ahead.h);
            } else {
                dy += L.in.sh;
                v += L.v.sh;
            }
        }
        copies_commit();
    };
#pragma unroll
    for (int i = 0; i < kRotBwdDepth - 1; ++i)
        fetch(i);
    float2 sa[4], sb[4];
    uint4 *const sums = slots_raw + kRotBwdDepth * 4 * kRotThreads + threadIdx.x;
    const uint32_t sums_a = smem_addr(sums), sums_b = sums_a + 4 * kRotThreads * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        sa[i] = sb[i] = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        sums[i * kRotThreads] = make_uint4(0, 0, 0, 0);
    uint64_t positions = load_positions<LANES>(p, at.t);
    RotaryShared &sh = *reinterpret_cast<RotaryShared *>(slots_raw + (kRotBwdDepth * 4 + 8) * kRotThreads);
    rotary_shared<LANES>(p, L, m, sh);
    float2 c[4], s[4];
    float rs = at.t < p.tokens && steps > 0 ? __ldg(L.rstd + (size_t)at.t * L.heads + at.h) : 0.f;
    bool jump = true; // another token than the step before
    for (uint32_t n = 0, stage = 0; n < steps; ++n, stage = (stage + 1) % kRotBwdDepth) {
        fetch((stage + kRotBwdDepth - 1) % kRotBwdDepth);
        const bool row = at.t < p.tokens;
        if (jump) {
            rotary_angles<LANES>(p, sh, m, at.t, positions, -1.f, c, s);
            positions = load_positions<LANES>(p, at.next_token(p, L, w));
        }
        const float2 rs2 = make_float2(rs, rs);
        uint16_t *const to = const_cast<uint16_t *>(out);
        jump = at.next(p, L, w);
        if (jump)
            out = row_at(L.out, at.t, at.h);
        else
            out += L.out.sh;
        rs = at.t < p.tokens && n + 1 < steps ? __ldg(L.rstd + (size_t)at.t * L.heads + at.h) : 0.f; // the next row's
        copies_wait<kRotBwdDepth - 1>();
        uint4 da = make_uint4(0, 0, 0, 0), db = da, va = da, vb = da;
        if (row && m.live) {
            const uint32_t from = mine + stage * kStage;
            da = slot16(from);
            db = slot16(from + kQuarter);
            va = slot16(from + 2 * kQuarter);
            vb = slot16(from + 3 * kQuarter);
        }
        float2 a[4], b[4], x[4], y[4];
        unpack(da, a);
        unpack(db, b);
        unpack(va, x);
        unpack(vb, y);
        if (row)
            rotate<ADJ>(m, a, b, c, s);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = mul2(x[i], rs2);
            y[i] = mul2(y[i], rs2);
            sa[i] = fma2(a[i], x[i], sa[i]);
            sb[i] = fma2(b[i], y[i], sb[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const float4 f = sh.w[i / 2][threadIdx.x % LANES], g = sh.w[2 + i / 2][threadIdx.x % LANES];
            a[i] = mul2(a[i], make_float2(f.x, f.y));
            a[i + 1] = mul2(a[i + 1], make_float2(f.z, f.w));
            b[i] = mul2(b[i], make_float2(g.x, g.y));
            b[i + 1] = mul2(b[i + 1], make_float2(g.z, g.w));
            sum = fma2(b[i], y[i], fma2(a[i], x[i], sum));
            sum = fma2(b[i + 1], y[i + 1], fma2(a[i + 1], x[i + 1], sum));
        }
        if (n % kRotBlock == kRotBlock - 1) {
            fold(sums_a, sa);
            fold(sums_b, sb);
        }
        const float mean = -__fmul_rn(lanes_sum<LANES>(__fadd_rn(sum.x, sum.y)), p.inv_d);
        const float2 mean2 = make_float2(mean, mean);
        if (row) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = mul2(rs2, fma2(x[i], mean2, a[i]));
                b[i] = mul2(rs2, fma2(y[i], mean2, b[i]));
            }
            store_row(to, m, a, b);
        }
    }
    fold(sums_a, sa);
    fold(sums_b, sb);
    copies_wait<0>();
    __syncthreads(); // the slots are free
    // the warp's lane groups in order, then the CTA's warps
    auto over_groups = [&](float &hi, float &lo) {
#pragma unroll
        for (int o = LANES; o < 32; o <<= 1) {
            const float h2 = __shfl_xor_sync(0xffffffffu, hi, o), l2 = __shfl_xor_sync(0xffffffffu, lo, o);
            // the lower group's sum first, on both sides
            const bool up = threadIdx.x & o;
            float f = up ? h2 : hi, e = up ? l2 : lo;
            comp_add(f, e, up ? hi : h2);
            lo = __fadd_rn(e, up ? lo : l2);
            hi = f;
        }
    };
    float2 *part = reinterpret_cast<float2 *>(slots_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float4 v = ld_shared_f4(sums_a + i * kRotThreads * 16);
        over_groups(v.x, v.z);
        over_groups(v.y, v.w);
        if (lane < LANES && m.live) {
            float2 *to = part + warp * p.D + (i < 4 ? m.a + 2 * i : m.b + 2 * i - 8);
            to[0] = make_float2(v.x, v.z);
            to[1] = make_float2(v.y, v.w);
        }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < p.D; j += kRotThreads) {
        float2 f = part[j];
        for (int k = 1; k < kRotWarps; ++k) {
            const float2 e = part[k * p.D + j];
            comp_add(f.x, f.y, e.x);
            f.y = __fadd_rn(f.y, e.y);
        }
        L.partials[(size_t)cta * p.D + j] = f;
    }
}

// ------------------------------------------------------------------- launch

static int rotary_lanes(int D)
{
    int lanes = 2;
    while (lanes * 16 < D)
        lanes *= 2;
    return lanes;
}

// As many CTAs as run at a time, shared out by the lists' rows, a token's angles
// counted as one more; a warp has at least a step.  A run is a token's heads, or
// tokens enough for 16 steps.  GB300, 32768 tokens of 24 + 4 heads of 256: angles
// not counted 175 us forward and 233 backward, as one row 163 and 220, as two 225
// and 223; with two CTAs an SM instead of three the forward takes 150.
void rotary_plan(RotaryParams &p)
{
    const uint32_t tokens = 32 / rotary_lanes(p.D), resident = (uint32_t)kSMsBlock * 2;
    const uint64_t all = (p.l[0].heads ? (uint64_t)p.l[0].heads + 1 : 0) + (p.l[1].heads ? p.l[1].heads + 1 : 0);
    for (RotaryList &l : p.l) {
        const uint64_t groups = ((uint64_t)p.tokens + tokens - 1) / tokens, steps = groups * l.heads;
        uint64_t ctas = (steps + kRotWarps - 1) / kRotWarps;
        const uint64_t most = l.heads ? (resident * ((uint64_t)l.heads + 1) + all / 2) / all : 0;
        if (ctas > most)
            ctas = most > 0 ? most : steps > 0;
        l.ctas = (int)ctas;
        l.run = l.heads > 0 && l.heads < 16 ? 16 / l.heads : 1;
        l.rounds = ctas ? (uint32_t)(groups / (ctas * kRotWarps * l.run)) : 0;
    }
}

template <int LANES>
static cudaError_t launch_lanes(const RotaryParams &p, bool adjacent, bool inverse, cudaStream_t stream)
{
    const dim3 grid((unsigned)(p.l[0].ctas + p.l[1].ctas));
    const float sign = inverse ? -1.f : 1.f;
    const bool norm = p.l[0].w != nullptr;
    auto kern = adjacent ? (norm ? rotary_kernel<LANES, true, true> : rotary_kernel<LANES, true, false>)
                         : (norm ? rotary_kernel<LANES, false, true> : rotary_kernel<LANES, false, false>);
    return launch_after(kern, grid, kRotThreads, kRotFwdDepth * 2 * kRotThreads * 16 + sizeof(RotaryShared), stream, p, sign);
}

cudaError_t launch_rotary(const RotaryParams &p, bool adjacent, bool inverse, cudaStream_t stream)
{
    switch (rotary_lanes(p.D)) {
    case 2: return launch_lanes<2>(p, adjacent, inverse, stream);
    case 4: return launch_lanes<4>(p, adjacent, inverse, stream);
    case 8: return launch_lanes<8>(p, adjacent, inverse, stream);
    case 16: return launch_lanes<16>(p, adjacent, inverse, stream);
    default: return launch_lanes<32>(p, adjacent, inverse, stream);
    }
}

template <int LANES>
static cudaError_t launch_bwd_lanes(const RotaryParams &p, bool adjacent, cudaStream_t stream)
{
    const dim3 grid((unsigned)(p.l[0].ctas + p.l[1].ctas));
    // (the warps' sums, 64 bytes a column, fit the slots)
    const size_t smem = (kRotBwdDepth * 4 + 8) * kRotThreads * 16 + sizeof(RotaryShared);
    return launch_after(adjacent ? rotary_bwd_kernel<LANES, true> : rotary_bwd_kernel<LANES, false>, grid, kRotThreads,
                        smem, stream, p);
}

cudaError_t launch_rotary_bwd(const RotaryParams &p, bool adjacent, cudaStream_t stream)
{
    cudaError_t e;
    switch (rotary_lanes(p.D)) {
    case 2: e = launch_bwd_lanes<2>(p, adjacent, stream); break;
    case 4: e = launch_bwd_lanes<4>(p, adjacent, stream); break;
    case 8: e = launch_bwd_lanes<8>(p, adjacent, stream); break;
    case 16: e = launch_bwd_lanes<16>(p, adjacent, stream); break;
    default: e = launch_bwd_lanes<32>(p, adjacent, stream); break;
    }
    return e;
}

} // namespace cake
