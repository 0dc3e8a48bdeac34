// norm.hip -- gfx950 (CDNA4) kernels of the gradient norms (the sum of squares of
// a tensor list, over all its elements and per tensor) and of clipping by them.
//
//   S_i = sum over tensor i of g^2,  S = sum_i S_i,  norm = sqrt(S)
//
// Every element is widened to binary64, squared (exactly, for 16-bit and fp32
// inputs) and summed in binary64: no square overflows or underflows, whatever
// the inputs' range, and the result is within n * 2^-53 of the sum.  S is not
// finite exactly if an element is inf or NaN, so the overflow test of fp16
// training comes with the norm.
//
// Each workgroup sums one chunk into one partial; a second launch joins the
// partials in a fixed order (no floating-point atomics), so a list gives the
// same bits at every call.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "adamw.h"
#include "device.hpp"
#include "layout.hpp"

namespace adamw {
namespace {

constexpr int kF32 = ADAMW_F32, kBf16 = ADAMW_BF16, kF16 = ADAMW_F16;

template <int DT>
struct Elem {
    static constexpr bool f32 = DT == kF32;
    static constexpr int size = f32 ? 4 : 2;
    static constexpr int pack = 16 / size;   // elements of a 16-byte word
};

template <int DT>
__device__ __forceinline__ double square1(uint64_t addr)
{
    float x;
    if constexpr (DT == kF32) x = *gptr<const float>(addr, 0);
    else x = widen1<DT == kF16>(*gptr<const uint16_t>(addr, 0));
    return (double)x * (double)x;
}

template <int DT>
__device__ __forceinline__ void add_squares(u32x4 q, double& a, double& b)
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (DT == kF32) {
            const double x = (double)__uint_as_float(w[j]);
            if (j & 1) b = __builtin_fma(x, x, b);
            else a = __builtin_fma(x, x, a);
        } else {
            const f32x2 x = widen2<DT == kF16>(w[j]);
            a = __builtin_fma((double)x.x, (double)x.x, a);
            b = __builtin_fma((double)x.y, (double)x.y, b);
        }
    }
}

// The elements of a sweep chunk: `head` before its first 16-byte edge, `words`
// whole 16-byte words from `body` on, `tail` after them.
template <int DT>
struct Span {
    uint64_t body;
    uint32_t head, words, tail;

    __device__ __forceinline__ Span(uint64_t addr, uint32_t n)
    {
        const uint32_t h = (uint32_t)((16u - (uint32_t)(addr & 15u)) & 15u) / Elem<DT>::size;
        head = h < n ? h : n;
        words = (n - head) / Elem<DT>::pack;
        tail = n - head - words * Elem<DT>::pack;
        body = addr + (uint64_t)head * Elem<DT>::size;
    }
    __device__ __forceinline__ uint64_t head_addr(uint32_t i) const { return body - (uint64_t)(head - i) * Elem<DT>::size; }
    __device__ __forceinline__ uint64_t tail_addr(uint32_t i) const
    {
        return body + (uint64_t)words * 16u + (uint64_t)i * Elem<DT>::size;
    }
};

// Sum over the workgroup, in lane 0 of wave 0: a butterfly in each wave, then the
// waves in order.
template <int BLOCK>
__device__ __forceinline__ double block_sum(double x)
{
    constexpr int kWaves = BLOCK / 64;
    __shared__ double wave_sum[kWaves];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d);
    if (threadIdx.x % 64 == 0) wave_sum[threadIdx.x / 64] = x;
    __syncthreads();
    double s = wave_sum[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) s += wave_sum[w];
    return s;
}

template <int DT>
__global__ __launch_bounds__(kBlockSweep) void sumsq_kernel(const DevSeg* __restrict__ segs,
                                                        const DevChunk* __restrict__ chunks,
                                                        double* __restrict__ partials)
{
    const uint32_t ci = xcd_chunk(blockIdx.x, gridDim.x);
    const DevChunk ch = chunks[ci];
    const Span<DT> sp(segs[ch.seg].ptr[ADAMW_STREAM_GRAD] + ch.off * Elem<DT>::size, ch.n_kind & kCountMask);
    const GLOBAL u32x4* __restrict__ g4 = gptr<const u32x4>(sp.body, 0);
    const uint32_t tid = threadIdx.x;
    double a = 0.0, b = 0.0;
    for (uint32_t k0 = tid; k0 < sp.words; k0 += kBlockSweep * kSweepUnroll) {
        u32x4 q[kSweepUnroll];
#pragma unroll
        for (int u = 0; u < kSweepUnroll; ++u) {
            const uint32_t k = k0 + u * kBlockSweep;
            q[u] = k < sp.words ? ld<1>(g4 + k) : u32x4{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int u = 0; u < kSweepUnroll; ++u) add_squares<DT>(q[u], a, b);
    }
    if (tid < sp.head) a += square1<DT>(sp.head_addr(tid));
    if (tid < sp.tail) b += square1<DT>(sp.tail_addr(tid));
    const double s = block_sum<kBlockSweep>(a + b);
    if (tid == 0) partials[ci] = s;
}

// One workgroup per tensor: its chunks' partials (consecutive) to its sum.
__global__ __launch_bounds__(256) void tensor_sum_kernel(const double* __restrict__ partials,
                                                     const uint32_t* __restrict__ tensor_first, NormOut out)
{
    const uint32_t i = blockIdx.x;
    const uint32_t first = tensor_first[i], last = tensor_first[i + 1];
    double x = 0.0;
    for (uint32_t k = first + threadIdx.x; k < last; k += 256) x += partials[k];
    x = block_sum<256>(x);
    if (threadIdx.x == 0) {
        if (out.tensor_sumsq) out.tensor_sumsq[i] = x;
        if (out.tensor_norm) out.tensor_norm[i] = (float)__builtin_sqrt(x);
    }
}

// One workgroup: all partials to the list's sum.
constexpr int kBlockTotal = 1024;
__global__ __launch_bounds__(kBlockTotal) void total_kernel(const double* __restrict__ partials, uint32_t n, NormOut out)
{
    double x = 0.0;
    for (uint32_t k = threadIdx.x; k < n; k += kBlockTotal) x += partials[k];
    x = block_sum<kBlockTotal>(x);
    if (threadIdx.x == 0) {
        if (out.accumulate) x += *out.sumsq;
        *out.sumsq = x;
        if (out.norm) *out.norm = (float)__builtin_sqrt(x);
        if (out.found_inf) *out.found_inf = __builtin_isfinite(x) ? 0 : 1;
    }
}

// Clipping in place: g = round(g * f), f the clipping factor rounded to binary32,
// one binary32 product and one rounding to the gradient's type per element.  A
// factor of 1 changes no element and a sum that is not finite clips nothing:
// nothing is written.
template <int DT>
__device__ __forceinline__ u32x4 scale_word(u32x4 q, float f)
{
    if constexpr (DT == kF32) {
        return u32x4{__float_as_uint(__uint_as_float(q.x) * f), __float_as_uint(__uint_as_float(q.y) * f),
                     __float_as_uint(__uint_as_float(q.z) * f), __float_as_uint(__uint_as_float(q.w) * f)};
    } else {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f32x2 x = widen2<DT == kF16>(w[j]);
            o[j] = narrow2<DT == kF16>(x.x * f, x.y * f);
        }
        return u32x4{o[0], o[1], o[2], o[3]};
    }
}

template <int DT>
__device__ __forceinline__ void scale1(uint64_t addr, float f)
{
    if constexpr (DT == kF32) {
        GLOBAL float* p = gptr<float>(addr, 0);
        *p = *p * f;
    } else {
        GLOBAL uint16_t* p = gptr<uint16_t>(addr, 0);
        *p = narrow1<DT == kF16>(widen1<DT == kF16>(*p) * f);
    }
}

template <int DT>
__global__ __launch_bounds__(kBlockSweep) void clip_kernel(const DevSeg* __restrict__ segs,
                                                       const DevChunk* __restrict__ chunks, ClipRule rule,
                                                       float inv_scale, const adamw_loss_scale_state* __restrict__ amp)
{
    if (amp) inv_scale = (float)(1.0 / (double)amp->scale);
    double factor;
    if (!clip_factor(rule, *rule.sumsq, inv_scale, factor)) return;
    const float f = (float)factor;
    if (f == 1.0f) return;
    const DevChunk ch = chunks[xcd_chunk(blockIdx.x, gridDim.x)];
    const Span<DT> sp(segs[ch.seg].ptr[ADAMW_STREAM_GRAD] + ch.off * Elem<DT>::size, ch.n_kind & kCountMask);
    GLOBAL u32x4* __restrict__ g4 = gptr<u32x4>(sp.body, 0);
    const uint32_t tid = threadIdx.x;
    for (uint32_t k = tid; k < sp.words; k += kBlockSweep) st<2>(g4 + k, scale_word<DT>(ld<0>(g4 + k), f));
    if (tid < sp.head) scale1<DT>(sp.head_addr(tid), f);
    if (tid < sp.tail) scale1<DT>(sp.tail_addr(tid), f);
}

}  // namespace

hipError_t launch_clip(adamw_dtype g_dtype, const DevSeg* segs, const DevChunk* chunks, int64_t n_chunks,
                       const ClipRule& rule, float inv_scale, const adamw_loss_scale_state* d_amp, hipStream_t stream)
{
    if (n_chunks <= 0) return hipSuccess;
    const dim3 grid((unsigned)n_chunks), block(kBlockSweep);
    if (g_dtype == ADAMW_F16)
        hipLaunchKernelGGL((clip_kernel<kF16>), grid, block, 0, stream, segs, chunks, rule, inv_scale, d_amp);
    else if (g_dtype == ADAMW_BF16)
        hipLaunchKernelGGL((clip_kernel<kBf16>), grid, block, 0, stream, segs, chunks, rule, inv_scale, d_amp);
    else
        hipLaunchKernelGGL((clip_kernel<kF32>), grid, block, 0, stream, segs, chunks, rule, inv_scale, d_amp);
    return hipGetLastError();
}

hipError_t launch_sumsq(adamw_dtype g_dtype, const DevSeg* segs, const DevChunk* chunks, int64_t n_chunks,
                        const uint32_t* tensor_first, int64_t n_tensors, double* partials, const NormOut& out,
                        hipStream_t stream)
{
    hipError_t e = hipSuccess;
    if (n_chunks > 0) {
        const dim3 grid((unsigned)n_chunks), block(kBlockSweep);
        if (g_dtype == ADAMW_F16)
            hipLaunchKernelGGL((sumsq_kernel<kF16>), grid, block, 0, stream, segs, chunks, partials);
        else if (g_dtype == ADAMW_BF16)
            hipLaunchKernelGGL((sumsq_kernel<kBf16>), grid, block, 0, stream, segs, chunks, partials);
        else
            hipLaunchKernelGGL((sumsq_kernel<kF32>), grid, block, 0, stream, segs, chunks, partials);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if ((out.tensor_norm || out.tensor_sumsq) && n_tensors > 0) {
        hipLaunchKernelGGL(tensor_sum_kernel, dim3((unsigned)n_tensors), dim3(256), 0, stream, partials, tensor_first, out);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (out.sumsq) {
        hipLaunchKernelGGL(total_kernel, dim3(1), dim3(kBlockTotal), 0, stream, partials, (uint32_t)n_chunks, out);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace adamw
