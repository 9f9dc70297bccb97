// cake_rotary.cu -- the per-head norm of queries and keys with rotary positions
// of several axes for sm_103a, forward and backward.
//
// A row (a token's head) lies on LANES lanes of 16 columns each, so that both
// members of every rotated pair are a lane's own: of adjacent pairs 16 columns
// in a run, of the half style 8 in the first half and the 8 that they pair with.
// A lane group takes one token at a time and walks over its heads, so a lane
// computes the sine and cosine of its 8 pairs once for all of them.  The angle
// is a product modulo 2^64 in units of 2^-64 turn, whole turns drop out of it
// exactly, and its upper half goes to sincospif.
//
// HBM bounds both kernels: every value is read and written once.
#include "../csrc/cake_rows.cuh"
#include "cake_block_launch.h"

namespace cake {

constexpr int kRotThreads = 256;
constexpr int kRotWarps = kRotThreads / 32;
constexpr int kStatusInvalid = 1; // == CAKE_ERR_INVALID

// A lane's columns and pairs.
struct RotaryLane {
    bool live, rot;      // has columns; rotates them
    int a, b;            // its two vectors' first columns
    uint64_t turns[8];
    uint32_t axis;       // 4 bits a pair
};

template <bool ADJ>
__device__ __forceinline__ RotaryLane rotary_lane(const RotaryParams &p, int l)
{
    RotaryLane m;
    m.live = l < p.D / 16;
    m.rot = l < p.pairs / 8;
    const bool half = !ADJ && m.rot;
    m.a = half ? 8 * l : 16 * l;
    m.b = half ? p.pairs + 8 * l : 16 * l + 8;
    m.axis = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        m.turns[i] = m.rot ? __ldg(p.turns + 8 * l + i) : 0;
        if (m.rot && p.axis) {
            const int32_t x = __ldg(p.axis + 8 * l + i);
            if (x < 0 || x >= p.axes) {
                m.turns[i] = 0;
                set_status(p.status + 1, kStatusInvalid);
            } else {
                m.axis |= (uint32_t)x << (4 * i);
            }
        }
    }
    return m;
}

__device__ __forceinline__ uint64_t position(const RotaryParams &p, uint32_t axis, uint32_t t)
{
    const int64_t at = (int64_t)axis * p.axis_stride + (int64_t)t * p.token_stride;
    return p.pos_i64 ? (uint64_t)__ldg(static_cast<const long long *>(p.positions) + at)
                     : (uint64_t)(int64_t)__ldg(static_cast<const int *>(p.positions) + at);
}

// Cosines and sines of the lane's pairs at token t; `sign` -1: turned backwards.
__device__ __forceinline__ void rotary_angles(const RotaryParams &p, const RotaryLane &m, uint32_t t, float sign,
                                              float (&c)[8], float (&s)[8])
{
    if (!m.rot)
        return;
    uint64_t at = position(p, m.axis & 15u, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i > 0 && p.axis)
            at = position(p, (m.axis >> (4 * i)) & 15u, t);
        const int32_t phase = (int32_t)((m.turns[i] * at) >> 32); // 2^-32 turns
        sincospif((float)phase * 0x1p-31f, &s[i], &c[i]);
        s[i] *= sign;
    }
}

// f[0..8): the first vector, f[8..16): the second.
template <bool ADJ>
__device__ __forceinline__ void rotate(float (&f)[16], const float (&c)[8], const float (&s)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int x = ADJ ? 2 * i : i, y = ADJ ? 2 * i + 1 : 8 + i;
        const float a = f[x], b = f[y];
        f[x] = __fmaf_rn(a, c[i], -__fmul_rn(b, s[i]));
        f[y] = __fmaf_rn(b, c[i], __fmul_rn(a, s[i]));
    }
}

struct Row16 {
    uint4 a, b;
};

__device__ __forceinline__ Row16 load_row(const uint16_t *row, const RotaryLane &m)
{
    Row16 r;
    r.a = r.b = make_uint4(0, 0, 0, 0);
    if (m.live) {
        r.a = __ldcs(reinterpret_cast<const uint4 *>(row + m.a));
        r.b = __ldcs(reinterpret_cast<const uint4 *>(row + m.b));
    }
    return r;
}

__device__ __forceinline__ void unpack16(const Row16 &r, float (&f)[16])
{
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        f[2 * q] = bf16lo(word(r.a, q));
        f[2 * q + 1] = bf16hi(word(r.a, q));
        f[8 + 2 * q] = bf16lo(word(r.b, q));
        f[8 + 2 * q + 1] = bf16hi(word(r.b, q));
    }
}

__device__ __forceinline__ void store_row(uint16_t *row, const RotaryLane &m, const float (&f)[16])
{
    if (!m.live)
        return;
    __stcs(reinterpret_cast<uint4 *>(row + m.a), make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                                           pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])));
    __stcs(reinterpret_cast<uint4 *>(row + m.b), make_uint4(pack_bf16(f[8], f[9]), pack_bf16(f[10], f[11]),
                                                           pack_bf16(f[12], f[13]), pack_bf16(f[14], f[15])));
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v)
{
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
        v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// The lane's weights as FP32.
__device__ __forceinline__ void lane_weights(const RotaryList &l, const RotaryLane &m, float (&w)[16])
{
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int j = (i < 8 ? m.a : m.b - 8) + i;
        w[i] = !m.live ? 0.f
               : l.w_f32 ? __ldg(static_cast<const float *>(l.w) + j)
                         : __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t *>(l.w) + j) << 16);
    }
}

__device__ __forceinline__ int64_t head_off(const RowView &v, uint32_t t, uint32_t h)
{
    return (int64_t)t * v.st + (int64_t)h * v.sh;
}

// The CTA's list, and its index among that list's CTAs.
__device__ __forceinline__ const RotaryList &cta_list(const RotaryParams &p, uint32_t &cta)
{
    const bool keys = blockIdx.x >= (unsigned)p.l[0].ctas;
    cta = keys ? blockIdx.x - p.l[0].ctas : blockIdx.x;
    return p.l[keys];
}

// All lanes of a warp walk through the same number of rows, so that every
// shuffle finds the whole warp; a lane group without a row works on zeros.
template <int LANES, bool ADJ, bool NORM>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const __grid_constant__ RotaryParams p, float sign)
{
    pdl_wait();
    uint32_t cta;
    const RotaryList &L = cta_list(p, cta);
    const RotaryLane m = rotary_lane<ADJ>(p, threadIdx.x % LANES);
    const uint32_t group = threadIdx.x / LANES, slots = kRotThreads / LANES / L.splits;
    const uint32_t slot = group / L.splits, sub = group % L.splits;
    const uint32_t t0 = cta * L.tokens_per_cta, t_end = min(p.tokens, t0 + L.tokens_per_cta);
    float w[NORM ? 16 : 1];
    if constexpr (NORM)
        lane_weights(L, m, w);
    for (uint32_t base = t0; base < t_end; base += slots) {
        const uint32_t t = base + slot;
        const bool on = t < t_end;
        Row16 next;
        next.a = next.b = make_uint4(0, 0, 0, 0);
        if (on && sub < L.heads)
            next = load_row(L.in.base + head_off(L.in, t, sub), m);
        float c[8], s[8];
        if (on)
            rotary_angles(p, m, t, sign, c, s);
        for (uint32_t h0 = 0; h0 < L.heads; h0 += L.splits) {
            const uint32_t h = h0 + sub;
            const Row16 row = next;
            if (on && h + L.splits < L.heads)
                next = load_row(L.in.base + head_off(L.in, t, h + L.splits), m);
            float f[16];
            unpack16(row, f);
            if constexpr (NORM) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    ss = __fmaf_rn(f[i], f[i], ss);
                ss = lanes_sum<LANES>(ss);
                const float rs = 1.0f / sqrtf(__fmaf_rn(ss, p.inv_d, p.eps));
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    f[i] = __fmul_rn(__fmul_rn(f[i], rs), w[i]);
                if (on && h < L.heads && threadIdx.x % LANES == 0)
                    L.rstd_out[(size_t)t * L.heads + h] = rs;
            }
            if (on && h < L.heads) {
                if (m.rot)
                    rotate<ADJ>(f, c, s);
                store_row(const_cast<uint16_t *>(L.out.base) + head_off(L.out, t, h), m, f);
            }
        }
    }
}

// Backward with a norm.  A lane adds its 16 columns' terms of dw as Kahan pairs.
template <int LANES, bool ADJ>
__global__ void __launch_bounds__(kRotThreads) rotary_bwd_kernel(const __grid_constant__ RotaryParams p)
{
    extern __shared__ __align__(16) float2 part[]; // [warps][D]
    pdl_wait();
    uint32_t cta;
    const RotaryList &L = cta_list(p, cta);
    const RotaryLane m = rotary_lane<ADJ>(p, threadIdx.x % LANES);
    const uint32_t group = threadIdx.x / LANES, slots = kRotThreads / LANES / L.splits;
    const uint32_t slot = group / L.splits, sub = group % L.splits;
    const uint32_t t0 = cta * L.tokens_per_cta, t_end = min(p.tokens, t0 + L.tokens_per_cta);
    float w[16], hi[16], lo[16];
    lane_weights(L, m, w);
#pragma unroll
    for (int i = 0; i < 16; ++i)
        hi[i] = lo[i] = 0.f;
    for (uint32_t base = t0; base < t_end; base += slots) {
        const uint32_t t = base + slot;
        const bool on = t < t_end;
        float c[8], s[8];
        if (on)
            rotary_angles(p, m, t, -1.f, c, s);
        for (uint32_t h0 = 0; h0 < L.heads; h0 += L.splits) {
            const uint32_t h = h0 + sub;
            const bool row = on && h < L.heads;
            Row16 rd, rv;
            rd.a = rd.b = rv.a = rv.b = make_uint4(0, 0, 0, 0);
            float rs = 0.f;
            if (row) {
                rd = load_row(L.in.base + head_off(L.in, t, h), m);
                rv = load_row(L.v.base + head_off(L.v, t, h), m);
                rs = __ldg(L.rstd + (size_t)t * L.heads + h);
            }
            float d[16], v[16];
            unpack16(rd, d);
            unpack16(rv, v);
            if (row && m.rot)
                rotate<ADJ>(d, c, s);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                v[i] = __fmul_rn(v[i], rs);
                const float y = __fmaf_rn(d[i], v[i], lo[i]), x = __fadd_rn(hi[i], y);
                lo[i] = __fadd_rn(__fsub_rn(hi[i], x), y);
                hi[i] = x;
                d[i] = __fmul_rn(d[i], w[i]);
                sum = __fmaf_rn(d[i], v[i], sum);
            }
            const float mean = __fmul_rn(lanes_sum<LANES>(sum), p.inv_d);
            if (row) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    d[i] = __fmul_rn(rs, __fmaf_rn(-v[i], mean, d[i]));
                store_row(const_cast<uint16_t *>(L.out.base) + head_off(L.out, t, h), m, d);
            }
        }
    }
    // the warp's lane groups in order, then the CTA's warps
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int o = LANES; o < 32; o <<= 1) {
            const float h2 = __shfl_xor_sync(0xffffffffu, hi[i], o), l2 = __shfl_xor_sync(0xffffffffu, lo[i], o);
            // the lower group's sum first, on both sides
            const bool up = threadIdx.x & o;
            float a = up ? h2 : hi[i], b = up ? l2 : lo[i];
            comp_add(a, b, up ? hi[i] : h2);
            lo[i] = __fadd_rn(b, up ? lo[i] : l2);
            hi[i] = a;
        }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane < LANES && m.live)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            part[warp * p.D + (i < 8 ? m.a : m.b - 8) + i] = make_float2(hi[i], lo[i]);
    __syncthreads();
    for (int j = threadIdx.x; j < p.D; j += kRotThreads) {
        float2 a = part[j];
        for (int k = 1; k < kRotWarps; ++k) {
            const float2 b = part[k * p.D + j];
            comp_add(a.x, a.y, b.x);
            a.y = __fadd_rn(a.y, b.y);
        }
        L.partials[(size_t)cta * p.D + j] = a;
    }
    pdl_launch_dependents();
}

// ------------------------------------------------------------------- launch

static int rotary_lanes(int D)
{
    int lanes = 2;
    while (lanes * 16 < D)
        lanes *= 2;
    return lanes;
}

// A token's heads stay with one lane group where there are tokens enough for
// all, so that its angles are computed once; fewer tokens split them.
void rotary_plan(RotaryParams &p, bool sums)
{
    const int groups = kRotThreads / rotary_lanes(p.D); // a power of two
    const uint32_t resident = (uint32_t)kSMsBlock * 4;  // CTAs
    for (RotaryList &l : p.l) {
        if (l.heads == 0 || p.tokens == 0) {
            l.ctas = 0;
            l.splits = 1;
            l.tokens_per_cta = 1;
            continue;
        }
        l.splits = 1;
        while (l.splits < groups && (uint32_t)l.splits < l.heads &&
               (uint64_t)p.tokens * l.splits < (uint64_t)resident * groups)
            l.splits *= 2;
        const uint32_t slots = groups / l.splits;
        uint64_t turns = ((uint64_t)p.tokens + slots - 1) / slots; // of a single CTA
        // sums: no more CTAs than what runs at a time, each leaves a partial
        const uint64_t most = sums ? resident : resident * 8;
        const uint64_t per = (turns + most - 1) / most;
        l.tokens_per_cta = (uint32_t)(per * slots);
        l.ctas = (int)(((uint64_t)p.tokens + l.tokens_per_cta - 1) / l.tokens_per_cta);
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
    return launch_after(kern, grid, kRotThreads, 0, stream, p, sign);
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
    const size_t smem = (size_t)kRotWarps * p.D * sizeof(float2); // at most 32 KB
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
