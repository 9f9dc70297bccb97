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
// so that one pass and one reduction over the row give every scalar.
#include "../csrc/cake_device.cuh"
#include "cake_step_launch.h"

namespace cake {

constexpr int kSwThreads = 256;
constexpr int kSwWarps = kSwThreads / 32;
constexpr int kSMsStep = 152;

__device__ __forceinline__ void load_w8(const void *w, int f32, int v, float (&f)[8])
{
    if (f32) {
        const float4 a = __ldg(static_cast<const float4 *>(w) + 2 * v), b = __ldg(static_cast<const float4 *>(w) + 2 * v + 1);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
        unpack8(__ldg(static_cast<const uint4 *>(w) + v), f);
    }
}

__device__ __forceinline__ const uint4 *row_ptr(const RowView &v, uint32_t r, uint32_t nh)
{
    return reinterpret_cast<const uint4 *>(v.base + row_off(v, r, nh));
}
__device__ __forceinline__ uint4 *out_ptr(const RowView &v, uint32_t r, uint32_t nh)
{
    return reinterpret_cast<uint4 *>(const_cast<uint16_t *>(v.base) + row_off(v, r, nh));
}

// Sums of N values over the CTA, in every thread.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (*red)[kSwWarps])
{
#pragma unroll
    for (int n = 0; n < N; ++n)
        v[n] = warp_sum(v[n]);
    __syncthreads(); // the previous row's sums are read
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int n = 0; n < N; ++n)
            red[n][threadIdx.x >> 5] = v[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
        float s = red[n][0];
        for (int w = 1; w < kSwWarps; ++w)
            s += red[n][w];
        v[n] = s;
    }
}

template <int VPT>
__global__ void __launch_bounds__(kSwThreads) sandwich_fwd_kernel(const __grid_constant__ SandwichFwdParams p)
{
    __shared__ float red[1][kSwWarps];
    for (uint32_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        float z[VPT][8], h[VPT][8];
        float ss[1] = {0.f};
        const float g_row = p.gate_rows ? p.gate_rows[r] : 1.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = k * kSwThreads + threadIdx.x;
            if (v < p.nvec) {
                unpack8(row_ptr(p.z, r, p.nh)[v], z[k]);
                unpack8(row_ptr(p.x, r, p.nh)[v], h[k]);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    ss[0] = __fmaf_rn(z[k][q], z[k][q], ss[0]);
            }
        }
        block_sum(ss, red);
        const float r1 = 1.0f / sqrtf(__fadd_rn(__fmul_rn(ss[0], p.inv_h), p.eps));
        const float sg = p.scale * g_row;
        ss[0] = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = k * kSwThreads + threadIdx.x;
            if (v < p.nvec) {
                float w[8], g[8];
                load_w8(p.w_post, p.post_f32, v, w);
                if (p.gate.base)
                    unpack8(row_ptr(p.gate, r, p.nh)[v], g);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float n = __fmul_rn(__fmul_rn(z[k][q], r1), w[q]);
                    h[k][q] = __fmaf_rn(p.gate.base ? __fmul_rn(sg, g[q]) : sg, n, h[k][q]);
                }
                const uint4 raw = pack8(h[k]);
                unpack8(raw, h[k]);
                out_ptr(p.h_new, r, p.nh)[v] = raw;
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    ss[0] = __fmaf_rn(h[k][q], h[k][q], ss[0]);
            }
        }
        block_sum(ss, red);
        const float r2 = 1.0f / sqrtf(__fadd_rn(__fmul_rn(ss[0], p.inv_h), p.eps));
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = k * kSwThreads + threadIdx.x;
            if (v < p.nvec) {
                float w[8], y[8];
                load_w8(p.w_pre, p.pre_f32, v, w);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    y[q] = __fmul_rn(__fmul_rn(h[k][q], r2), w[q]);
                out_ptr(p.y, r, p.nh)[v] = pack8(y);
            }
        }
        if (threadIdx.x == 0) {
            p.rstd_post[r] = r1;
            p.rstd_pre[r] = r2;
        }
    }
}

template <int VPT>
__global__ void __launch_bounds__(kSwThreads) sandwich_bwd_kernel(const __grid_constant__ SandwichBwdParams p)
{
    extern __shared__ float2 acc[]; // [2][H] compensated (hi, lo)
    __shared__ float red[3][kSwWarps];
    float2 *acc_post = acc, *acc_pre = acc + p.H;
    for (int j = threadIdx.x; j < 2 * p.H; j += kSwThreads)
        acc[j] = make_float2(0.f, 0.f);
    __syncthreads();
    const uint32_t r0 = blockIdx.x * p.rows_per_cta, r1 = min(p.rows, r0 + p.rows_per_cta);
    for (uint32_t r = r0; r < r1; ++r) {
        const float rp = p.rstd_post[r], rn = p.rstd_pre[r];
        const float sg = p.gate_rows ? p.scale * p.gate_rows[r] : p.scale;
        float s[3] = {0.f, 0.f, 0.f};
        uint4 rh[VPT], rz[VPT], rd[VPT], re[VPT], rg[VPT];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = k * kSwThreads + threadIdx.x;
            if (v < p.nvec) {
                rh[k] = row_ptr(p.h, r, p.nh)[v];
                rz[k] = row_ptr(p.z, r, p.nh)[v];
                rd[k] = row_ptr(p.dy, r, p.nh)[v];
                re[k] = p.dh.base ? row_ptr(p.dh, r, p.nh)[v] : make_uint4(0, 0, 0, 0);
                if (p.gate.base)
                    rg[k] = row_ptr(p.gate, r, p.nh)[v];
                float h[8], z[8], d[8], e[8], g[8], w1[8], w2[8];
                unpack8(rh[k], h);
                unpack8(rz[k], z);
                unpack8(rd[k], d);
                unpack8(re[k], e);
                load_w8(p.w_post, p.post_f32, v, w1);
                load_w8(p.w_pre, p.pre_f32, v, w2);
                if (p.gate.base)
                    unpack8(rg[k], g);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float a = __fmul_rn(d[q], w2[q]);
                    const float b = p.gate.base ? __fmul_rn(w1[q], g[q]) : w1[q];
                    const float bz = __fmul_rn(b, z[q]);
                    s[0] = __fmaf_rn(a, h[q], s[0]);
                    s[1] = __fmaf_rn(__fmaf_rn(rn, a, e[q]), bz, s[1]);
                    s[2] = __fmaf_rn(bz, h[q], s[2]);
                }
            }
        }
        block_sum(s, red);
        const float c2 = __fmul_rn(__fmul_rn(s[0], p.inv_h), rn);
        const float k2 = __fmul_rn(__fmul_rn(c2, rn), rn);
        const float dot = __fmaf_rn(-k2, s[2], s[1]);
        const float k1 = __fmul_rn(__fmul_rn(__fmul_rn(dot, p.inv_h), rp), rp);
        const float sr = __fmul_rn(sg, rp);
        if (threadIdx.x == 0 && p.dgate_rows)
            p.dgate_rows[r] = __fmul_rn(__fmul_rn(p.scale, rp), dot);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = k * kSwThreads + threadIdx.x;
            if (v < p.nvec) {
                float h[8], z[8], d[8], e[8], g[8], w1[8], w2[8], dx[8], dz[8], dg[8];
                unpack8(rh[k], h);
                unpack8(rz[k], z);
                unpack8(rd[k], d);
                unpack8(re[k], e);
                load_w8(p.w_post, p.post_f32, v, w1);
                load_w8(p.w_pre, p.pre_f32, v, w2);
                if (p.gate.base)
                    unpack8(rg[k], g);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float a = __fmul_rn(d[q], w2[q]);
                    const float t = __fmaf_rn(-k2, h[q], __fmaf_rn(rn, a, e[q]));
                    const float gq = p.gate.base ? g[q] : 1.f;
                    dx[q] = t;
                    const float tg = __fmul_rn(t, gq);
                    dz[q] = __fmul_rn(sr, __fmaf_rn(tg, w1[q], -__fmul_rn(k1, z[q])));
                    const float tz = __fmul_rn(sr, z[q]);
                    dg[q] = __fmul_rn(__fmul_rn(t, tz), w1[q]);
                    float2 m = acc_post[8 * v + q];
                    comp_add(m.x, m.y, __fmul_rn(tg, tz));
                    acc_post[8 * v + q] = m;
                    m = acc_pre[8 * v + q];
                    comp_add(m.x, m.y, __fmul_rn(__fmul_rn(d[q], h[q]), rn));
                    acc_pre[8 * v + q] = m;
                }
                out_ptr(p.dx, r, p.nh)[v] = pack8(dx);
                out_ptr(p.dz, r, p.nh)[v] = pack8(dz);
                if (p.dgate.base)
                    out_ptr(p.dgate, r, p.nh)[v] = pack8(dg);
            }
        }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < p.H; j += kSwThreads) {
        p.partials[(size_t)blockIdx.x * p.H + j] = acc_post[j];
        p.partials[((size_t)gridDim.x + blockIdx.x) * p.H + j] = acc_pre[j];
    }
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

cudaError_t ensure_smem_attr(const void *kernel, size_t smem);

int sandwich_bwd_ctas(int H, uint32_t rows)
{
    (void)H;
    const uint32_t most = kSMsStep;
    if (rows == 0)
        return 0;
    const uint32_t per = (rows + most - 1) / most;
    return (int)((rows + per - 1) / per);
}

template <int VPT>
static cudaError_t fwd_vpt(const SandwichFwdParams &p, cudaStream_t stream)
{
    const int ctas = (int)(p.rows < (uint32_t)kSMsStep * 8 ? p.rows : (uint32_t)kSMsStep * 8);
    sandwich_fwd_kernel<VPT><<<ctas, kSwThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_sandwich_fwd(const SandwichFwdParams &p, cudaStream_t stream)
{
    switch ((p.nvec + kSwThreads - 1) / kSwThreads) {
    case 1: return fwd_vpt<1>(p, stream);
    case 2: return fwd_vpt<2>(p, stream);
    case 3: return fwd_vpt<3>(p, stream);
    default: return fwd_vpt<4>(p, stream);
    }
}

template <int VPT>
static cudaError_t bwd_vpt(const SandwichBwdParams &p, int ctas, cudaStream_t stream)
{
    const size_t smem = (size_t)16 * p.H;
    cudaError_t e = ensure_smem_attr((const void *)sandwich_bwd_kernel<VPT>, smem);
    if (e != cudaSuccess)
        return e;
    sandwich_bwd_kernel<VPT><<<ctas, kSwThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_sandwich_bwd(const SandwichBwdParams &p, int ctas, cudaStream_t stream)
{
    switch ((p.nvec + kSwThreads - 1) / kSwThreads) {
    case 1: return bwd_vpt<1>(p, ctas, stream);
    case 2: return bwd_vpt<2>(p, ctas, stream);
    case 3: return bwd_vpt<3>(p, ctas, stream);
    default: return bwd_vpt<4>(p, ctas, stream);
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
