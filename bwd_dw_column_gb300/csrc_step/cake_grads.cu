// cake_grads.cu -- the global L2 norm of many gradient tensors, and clipping
// by it, for sm_103a.
//
//   norm = sqrt(sum g^2),  coef = min(1, max_norm / (norm + eps)),  out = round(g * coef)
//
// The tensors' addresses travel in the launch parameters, so a call uses no
// device memory but one FP64 partial per CTA.  All tensors are cut into chunks
// of kGradChunk values; CTA b takes chunks b, b + ctas, ...  Two kernels: the
// first leaves a partial sum of squares per CTA, the second adds the partials
// up (every CTA does, in the same order, so that no third launch and no wait
// between CTAs is needed) and scales.  Short lists of small tensors take one
// CTA and one launch.  All orders depend on the shapes alone.
//
// Sums: a thread adds the squares of the 32 values that it has of a chunk in
// FP32, and the sum to its FP64 accumulator.  An FP32 sum outside
// [2^-60, 2^80] of values that are not all zero may have lost terms to
// underflow or overflowed: those 32 values are summed again in FP64, which
// holds every square of the types.  Inside it, a term lost to underflow is
// below 2^-149 against a sum of 2^-60 or more.
//
// HBM bounds both kernels: a norm reads once, clipping reads twice beyond L2
// and writes once (GB300: the norm of 3.1 G FP32 values 1.69 ms, 7.4 TB/s; 0.65 G
// BF16 values clipped into FP32 0.78 ms, 6.7 TB/s with the second read).
#include "../csrc/cake_device.cuh"
#include "cake_step_launch.h"

namespace cake {

constexpr int kGradWarps = kGradThreads / 32;
constexpr int kPerThread = kGradChunk / kGradThreads; // 32 values

// The last of tensors [lo, hi] whose first chunk is <= chunk.
template <int N>
__device__ __forceinline__ int find_tensor(const GradParams<N> &p, uint32_t chunk, int lo, int hi)
{
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.t[mid].chunk0 <= chunk)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ float load_one(const void *src, int64_t i, bool f32)
{
    return f32 ? static_cast<const float *>(src)[i]
               : __uint_as_float((uint32_t)static_cast<const uint16_t *>(src)[i] << 16);
}

// This thread's values of a chunk; missing ones are zero.  A whole aligned
// chunk comes in 16-byte loads: 4 groups of 8 BF16 values, group u at value
// 8 (u * kGradThreads + thread), or 8 groups of 4 FP32 values, group u at
// 4 (u * kGradThreads + thread).  QUADS: BF16 values in 8 groups of 4 as well,
// so that FP32 outputs are written in whole lines.
// (Plain loads: clipping in place writes what it has read.)
template <bool QUADS>
__device__ __forceinline__ void load_chunk(const GradDesc &d, int64_t first, float (&v)[kPerThread])
{
    const bool f32 = d.flags & kGradSrcF32;
    const int64_t left = d.count - first;
    if ((d.flags & kGradVector) && left >= kGradChunk) {
        if (QUADS && !f32 && (d.flags & kGradDstF32)) {
            const uint2 *s = reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(d.src) + first);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const uint2 a = s[u * kGradThreads + threadIdx.x];
                v[u * 4] = bf16lo(a.x);
                v[u * 4 + 1] = bf16hi(a.x);
                v[u * 4 + 2] = bf16lo(a.y);
                v[u * 4 + 3] = bf16hi(a.y);
            }
        } else if (f32) {
            const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(d.src) + first);
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float4 a = s[(u * 2 + k) * kGradThreads + threadIdx.x];
                    v[u * 8 + k * 4 + 0] = a.x;
                    v[u * 8 + k * 4 + 1] = a.y;
                    v[u * 8 + k * 4 + 2] = a.z;
                    v[u * 8 + k * 4 + 3] = a.w;
                }
        } else {
            const uint4 *s = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(d.src) + first);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float f[8];
                unpack8(s[u * kGradThreads + threadIdx.x], f);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[u * 8 + k] = f[k];
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < kPerThread; ++k) {
            const int64_t i = first + k * kGradThreads + threadIdx.x;
            v[k] = i < d.count ? load_one(d.src, i, f32) : 0.f;
        }
    }
}

__device__ __forceinline__ void store_one(const GradDesc &d, int64_t i, float v)
{
    if (d.flags & kGradDstF32)
        static_cast<float *>(d.dst)[i] = v;
    else
        static_cast<uint16_t *>(d.dst)[i] = (uint16_t)pack_bf16(v, 0.f);
}

// min(1, max_norm / (norm + eps)) that keeps a NaN; 1 where norm + eps is 0
// (there is nothing to scale)
__device__ __forceinline__ float clip_coef(float max_norm, double norm, float eps)
{
    const double by = norm + (double)eps;
    if (by == 0.0)
        return 1.0f;
    const double q = (double)max_norm / by;
    return q >= 1.0 ? 1.0f : (float)q;
}

template <int K>
__device__ __forceinline__ double values_sumsq(const float (&v)[K])
{
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < K; ++k)
        s[k & 3] = __fmaf_rn(v[k], v[k], s[k & 3]);
    const float t = __fadd_rn(__fadd_rn(s[0], s[1]), __fadd_rn(s[2], s[3]));
    if (t >= 0x1p-60f && t <= 0x1p80f)
        return (double)t;
    uint32_t any = 0; // zero, tiny, huge or not finite
#pragma unroll
    for (int k = 0; k < K; ++k)
        any |= __float_as_uint(v[k]) & 0x7fffffffu;
    if (any == 0)
        return 0.0;
    double e[2] = {0.0, 0.0};
#pragma unroll
    for (int k = 0; k < K; ++k)
        e[k & 1] = fma((double)v[k], (double)v[k], e[k & 1]);
    return e[0] + e[1];
}

// A whole aligned chunk of BF16 values, and its values as they come (in the order of load_chunk).
__device__ __forceinline__ bool whole_bf16(const GradDesc &d, uint32_t chunk)
{
    return (d.flags & (kGradVector | kGradSrcF32)) == kGradVector &&
           d.count - (int64_t)(chunk - d.chunk0) * kGradChunk >= kGradChunk;
}

__device__ __forceinline__ void load_bf16(const GradDesc &d, uint32_t chunk, uint4 (&v)[kPerThread / 8])
{
    const uint4 *s = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(d.src) +
                                                     (int64_t)(chunk - d.chunk0) * kGradChunk);
#pragma unroll
    for (int u = 0; u < kPerThread / 8; ++u)
        v[u] = s[u * kGradThreads + threadIdx.x];
}

__device__ __forceinline__ double values_sumsq(const uint4 (&v)[kPerThread / 8])
{
    float f[kPerThread];
#pragma unroll
    for (int u = 0; u < kPerThread / 8; ++u) {
        float g[8];
        unpack8(v[u], g);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            f[8 * u + k] = g[k];
    }
    return values_sumsq(f);
}

// The sum over the CTA in a fixed order, in thread 0.
__device__ __forceinline__ double cta_sum(double v)
{
    __shared__ double part[kGradWarps];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        v = part[0];
        for (int w = 1; w < kGradWarps; ++w)
            v += part[w];
    }
    return v;
}

template <int N>
__global__ void __launch_bounds__(kGradThreads) grad_sumsq_kernel(const __grid_constant__ GradParams<N> p)
{
    pdl_wait();
    double acc = 0.0;
    int i = 0;
    for (uint32_t c = blockIdx.x; c < p.chunks; c += gridDim.x) {
        i = find_tensor(p, c, i, p.n - 1);
        const GradDesc &d = p.t[i];
        // two whole chunks of BF16 values at once, as many bytes on their way as of
        // FP32 values (GB300: 0.4 G values 123 us against 131)
        const uint32_t c2 = c + gridDim.x;
        if (whole_bf16(d, c) && c2 < p.chunks) {
            const int i2 = find_tensor(p, c2, i, p.n - 1);
            if (whole_bf16(p.t[i2], c2)) {
                uint4 a[kPerThread / 8], b[kPerThread / 8];
                load_bf16(d, c, a);
                load_bf16(p.t[i2], c2, b);
                acc += values_sumsq(a);
                acc += values_sumsq(b);
                c = c2;
                i = i2;
                continue;
            }
        }
        float v[kPerThread];
        load_chunk<false>(d, (int64_t)(c - d.chunk0) * kGradChunk, v);
        acc += values_sumsq(v);
    }
    acc = cta_sum(acc);
    if (threadIdx.x == 0)
        p.partials[blockIdx.x] = acc;
    pdl_launch_dependents();
}

// The sum of all partials in thread 0, in an order that is the same in every CTA.
__device__ __forceinline__ double all_partials(const double *partials, int n)
{
    double v = 0.0;
    for (int i = threadIdx.x; i < n; i += kGradThreads)
        v += __ldcg(partials + i);
    return cta_sum(v);
}

__global__ void __launch_bounds__(kGradThreads) grad_final_kernel(const double *partials, int n, float *norm)
{
    pdl_wait();
    const double v = all_partials(partials, n);
    if (threadIdx.x == 0)
        *norm = (float)sqrt(v);
}

template <int N>
__global__ void __launch_bounds__(kGradThreads) grad_clip_kernel(const __grid_constant__ GradParams<N> p)
{
    pdl_wait();
    // one thread takes the root and the quotient: FP64 is slow
    __shared__ float shared_coef;
    const double sum = all_partials(p.partials, p.npartials);
    if (threadIdx.x == 0) {
        const double norm = sqrt(sum);
        if (p.norm && blockIdx.x == 0)
            *p.norm = (float)norm;
        shared_coef = clip_coef(p.max_norm, norm, p.eps);
    }
    __syncthreads();
    const float coef = shared_coef;
    if (p.in_place && coef == 1.0f)
        return;
    // last chunks first: L2 still holds what the sum has read last
    int i = p.n - 1;
    for (uint32_t k = blockIdx.x; k < p.chunks; k += gridDim.x) {
        const uint32_t c = p.chunks - 1 - k;
        i = find_tensor(p, c, 0, i);
        const GradDesc &d = p.t[i];
        const int64_t first = (int64_t)(c - d.chunk0) * kGradChunk;
        float v[kPerThread];
        load_chunk<true>(d, first, v);
        const bool f32 = d.flags & kGradSrcF32, o32 = d.flags & kGradDstF32;
        if ((d.flags & kGradVector) && d.count - first >= kGradChunk) {
            if (o32) { // 8 groups of 4, from either type
                float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(d.dst) + first);
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    o[u * kGradThreads + threadIdx.x] =
                        make_float4(__fmul_rn(v[4 * u], coef), __fmul_rn(v[4 * u + 1], coef),
                                    __fmul_rn(v[4 * u + 2], coef), __fmul_rn(v[4 * u + 3], coef));
            } else if (f32) {
                uint2 *o = reinterpret_cast<uint2 *>(static_cast<uint16_t *>(d.dst) + first);
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    o[u * kGradThreads + threadIdx.x] =
                        make_uint2(pack_bf16(__fmul_rn(v[4 * u], coef), __fmul_rn(v[4 * u + 1], coef)),
                                   pack_bf16(__fmul_rn(v[4 * u + 2], coef), __fmul_rn(v[4 * u + 3], coef)));
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    float w[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        w[k] = __fmul_rn(v[u * 8 + k], coef);
                    reinterpret_cast<uint4 *>(static_cast<uint16_t *>(d.dst) + first)[u * kGradThreads + threadIdx.x] =
                        pack8(w);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < kPerThread; ++k) {
                const int64_t at = first + k * kGradThreads + threadIdx.x;
                if (at < d.count)
                    store_one(d, at, __fmul_rn(v[k], coef));
            }
        }
    }
}

// All of a short list in one CTA and one launch: a warp takes pieces of
// kGradPiece values, first for the sum, then (clip) again for the scaling.
__global__ void __launch_bounds__(kGradOneThreads)
    grad_one_kernel(const __grid_constant__ GradParams<kGradFewTensors> p, int clip)
{
    constexpr int kWarps = kGradOneThreads / 32, kPer = kGradPiece / 32;
    __shared__ double part[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    double acc = 0.0;
    for (uint32_t c = warp; c < p.chunks; c += kWarps) {
        const GradDesc &d = p.t[find_tensor(p, c, 0, p.n - 1)];
        const int64_t first = (int64_t)(c - d.chunk0) * kGradPiece;
        float v[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int64_t i = first + 32 * k + lane;
            v[k] = i < d.count ? load_one(d.src, i, d.flags & kGradSrcF32) : 0.f;
        }
        acc += values_sumsq(v);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (lane == 0)
        part[warp] = acc;
    __syncthreads();
    // the rest of FP64 is one warp's: an SM does two such operations a cycle
    __shared__ float shared_coef;
    if (warp == 0) {
        acc = part[lane];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            acc += __shfl_xor_sync(0xffffffffu, acc, o);
        if (lane == 0) {
            const double norm = sqrt(acc);
            *p.norm = (float)norm;
            shared_coef = clip ? clip_coef(p.max_norm, norm, p.eps) : 1.0f;
        }
    }
    if (!clip)
        return;
    __syncthreads();
    const float coef = shared_coef;
    if (p.in_place && coef == 1.0f)
        return;
    for (uint32_t c = warp; c < p.chunks; c += kWarps) {
        const GradDesc &d = p.t[find_tensor(p, c, 0, p.n - 1)];
        const int64_t first = (int64_t)(c - d.chunk0) * kGradPiece;
        float v[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int64_t i = first + 32 * k + lane;
            v[k] = i < d.count ? load_one(d.src, i, d.flags & kGradSrcF32) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int64_t i = first + 32 * k + lane;
            if (i < d.count)
                store_one(d, i, __fmul_rn(v[k], coef));
        }
    }
}

// ------------------------------------------------------------------ launch

// A launch that may start while the one before it in the stream drains.
static cudaLaunchConfig_t dependent_config(int ctas, int threads, cudaLaunchAttribute *attr, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

template <int N>
cudaError_t launch_grad_sumsq(const GradParams<N> &p, int ctas, cudaStream_t stream)
{
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = dependent_config(ctas, kGradThreads, &attr, stream);
    cudaError_t e = cudaLaunchKernelEx(&cfg, grad_sumsq_kernel<N>, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

template <int N>
cudaError_t launch_grad_clip(const GradParams<N> &p, int ctas, cudaStream_t stream)
{
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = dependent_config(ctas, kGradThreads, &attr, stream);
    cudaError_t e = cudaLaunchKernelEx(&cfg, grad_clip_kernel<N>, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_grad_final(const double *partials, int n, float *norm, cudaStream_t stream)
{
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = dependent_config(1, kGradThreads, &attr, stream);
    cudaError_t e = cudaLaunchKernelEx(&cfg, grad_final_kernel, partials, n, norm);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_grad_one(const GradParams<kGradFewTensors> &p, bool clip, cudaStream_t stream)
{
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = dependent_config(1, kGradOneThreads, &attr, stream);
    cudaError_t e = cudaLaunchKernelEx(&cfg, grad_one_kernel, p, (int)clip);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

template cudaError_t launch_grad_sumsq<kGradFewTensors>(const GradParams<kGradFewTensors> &, int, cudaStream_t);
template cudaError_t launch_grad_sumsq<kGradSomeTensors>(const GradParams<kGradSomeTensors> &, int, cudaStream_t);
template cudaError_t launch_grad_sumsq<kGradMaxTensors>(const GradParams<kGradMaxTensors> &, int, cudaStream_t);
template cudaError_t launch_grad_clip<kGradFewTensors>(const GradParams<kGradFewTensors> &, int, cudaStream_t);
template cudaError_t launch_grad_clip<kGradSomeTensors>(const GradParams<kGradSomeTensors> &, int, cudaStream_t);
template cudaError_t launch_grad_clip<kGradMaxTensors>(const GradParams<kGradMaxTensors> &, int, cudaStream_t);

} // namespace cake
