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
// Each workgroup sums one chunk into one partial; the partials are joined in a fixed
// order (no floating-point atomics), so a list gives the same bits at every call: by
// a second launch, or for small lists by the last workgroup of the first.
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

// x plus the x of another lane (0 from outside the row or mask), by data-parallel
// moves of its two halves.
template <int CTRL, int ROWS>
__device__ __forceinline__ double add_lane(double x)
{
    const uint64_t v = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROWS, 0xf, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, ROWS, 0xf, true);
    return x + __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Sum over the wave, in lane 63: rows of 16 by shifts of 1, 2, 4 and 8 lanes, then
// lane 15 of a row to the next and lane 31 to the upper half.  Lane exchanges through
// the LDS unit instead kept a workgroup's last microsecond busy: at 8 waves per CU the
// 2.7 GB sum took 595 us with them and 371 without.
constexpr uint32_t kSumLane = 63;
__device__ __forceinline__ double wave_sum(double x)
{
    x = add_lane<0x111, 0xf>(x);
    x = add_lane<0x112, 0xf>(x);
    x = add_lane<0x114, 0xf>(x);
    x = add_lane<0x118, 0xf>(x);
    x = add_lane<0x142, 0xa>(x);
    return add_lane<0x143, 0xc>(x);
}

// Sum over the workgroup, in every lane: each wave, then the waves in order.  A second
// call needs a barrier after the first.
template <int BLOCK>
__device__ __forceinline__ double block_sum(double x)
{
    constexpr int kWaves = BLOCK / 64;
    __shared__ double sums[kWaves];
    x = wave_sum(x);
    if (threadIdx.x % 64 == kSumLane) sums[threadIdx.x / 64] = x;
    __syncthreads();
    double s = sums[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) s += sums[w];
    return s;
}

// A value that another workgroup of the same launch reads: stored and loaded past
// the XCDs' L2s (agent scope).  handed_over() waits until the stores before it have
// reached memory; the relaxed count that follows then tells the reader that they
// have.  A release fence would write back the whole L2 of the XCD instead: with one
// per workgroup a 2.7 GB sum took 4,050 us instead of 390.
__device__ __forceinline__ void hand_over(double* p, double x)
{
    __hip_atomic_store(p, x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ void handed_over() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// The sum of n <= kJoin values by one workgroup, lane l taking l, l + 256, ... in
// order: however the values come (SHARED: from workgroups of this launch), the same
// bits.
template <bool SHARED>
__device__ __forceinline__ double join(const double* p, uint32_t n)
{
    constexpr int kUnroll = 8;
    double x = 0.0;
    for (uint32_t k0 = threadIdx.x; k0 < n; k0 += kBlockJoin * kUnroll) {
        double v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint32_t k = k0 + u * kBlockJoin;
            if constexpr (SHARED)
                v[u] = k < n ? __hip_atomic_load(p + k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0;
            else
                v[u] = k < n ? p[k] : 0.0;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) x += v[u];
    }
    return block_sum<kBlockJoin>(x);
}

__device__ __forceinline__ void write_total(const NormOut& out, double x)
{
    if (out.accumulate) x += *out.sumsq;
    *out.sumsq = x;
    if (out.norm) *out.norm = (float)__builtin_sqrt(x);
    if (out.found_inf) *out.found_inf = __builtin_isfinite(x) ? 0 : 1;
}

// Whether this workgroup is the last of nb to hand a value over (uniform).
__device__ __forceinline__ bool last_of(double* slot, double x, uint32_t* done, uint32_t b, uint32_t nb)
{
    __shared__ int last;
    if (threadIdx.x == 0) {
        hand_over(slot, x);
        handed_over();
        last = grid_done(done, b, nb);
    }
    __syncthreads();
    return last != 0;
}

// Non-temporal loads: 376 us for the OPT-1.3B bf16 gradients in two lists on
// MI355X, against 402 without.
constexpr int kNtNorm = 1;
// FUSED: the only launch of a small sum, whose last workgroup joins the partials.
template <int DT, bool FUSED>
__global__ __launch_bounds__(kBlockSweep) void sumsq_kernel(const DevSweep* __restrict__ groups,
                                                        double* __restrict__ partials, uint32_t* __restrict__ done,
                                                        NormOut out)
{
    const uint32_t ci = xcd_chunk(blockIdx.x, gridDim.x);
    const DevSweep gr = groups[ci];
    const Span<DT> sp(gr.addr, gr.n);
    const GLOBAL u32x4* __restrict__ g4 = gptr<const u32x4>(sp.body, 0);
    const uint32_t tid = threadIdx.x;
    constexpr uint32_t kPass = kBlockSweep * kNormUnroll;
    double a = 0.0, b = 0.0;
    uint32_t k = tid;
    for (; k - tid + kPass <= sp.words; k += kPass) {
        u32x4 q[kNormUnroll];
#pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) q[u] = ld<kNtNorm>(g4 + k + u * kBlockSweep);
#pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) add_squares<DT>(q[u], a, b);
    }
    if (k - tid < sp.words) {
        u32x4 q[kNormUnroll];
#pragma unroll
        for (int u = 0; u < kNormUnroll; ++u)
            q[u] = k + u * kBlockSweep < sp.words ? ld<kNtNorm>(g4 + k + u * kBlockSweep) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) add_squares<DT>(q[u], a, b);
    }
    if (tid < sp.head) a += square1<DT>(sp.head_addr(tid));
    if (tid < sp.tail) b += square1<DT>(sp.tail_addr(tid));
    const double s = block_sum<kBlockSweep>(a + b);
    if constexpr (FUSED) {
        if (!last_of(partials + ci, s, done, blockIdx.x, gridDim.x)) return;
        const double x = join<true>(partials, gridDim.x);
        if (tid == 0) write_total(out, x);
    } else {
        if (tid == 0) partials[ci] = s;
    }
}

// Joins the partials of a sum.  Workgroups [0, n_blocks): kJoin partials each; the
// last of them to finish joins their sums.  The others: 4 tensors each (per-tensor
// norms), one per wave, or by all waves one after the other for tensors of many
// chunks.
constexpr int kTensorsPerGroup = kBlockJoin / 64;
constexpr uint32_t kWaveChunks = 256;   // chunks of a tensor that one wave sums
__global__ __launch_bounds__(kBlockJoin) void join_kernel(double* __restrict__ partials, uint32_t n, uint32_t n_blocks,
                                                      const uint32_t* __restrict__ tensor_first, uint32_t n_tensors,
                                                      uint32_t* __restrict__ done, NormOut out)
{
    const uint32_t b = blockIdx.x, tid = threadIdx.x;
    if (b < n_blocks) {
        const uint32_t at = b * (uint32_t)kJoin;
        double x = join<false>(partials + at, n - at < (uint32_t)kJoin ? n - at : (uint32_t)kJoin);
        if (n_blocks > 1) {
            double* sums = partials + n;
            if (!last_of(sums + b, x, done, b, n_blocks)) return;
            x = join<true>(sums, n_blocks);
        }
        if (tid == 0) write_total(out, x);
        return;
    }
    const uint32_t t0 = (b - n_blocks) * kTensorsPerGroup, lane = tid % 64, wave = tid / 64;
    for (uint32_t w = 0; w < kTensorsPerGroup; ++w) {
        const uint32_t i = t0 + w;
        if (i >= n_tensors) return;
        const uint32_t first = tensor_first[i], last = tensor_first[i + 1];
        double x = 0.0;
        if (last - first > kWaveChunks) {
            for (uint32_t k = first + tid; k < last; k += kBlockJoin) x += partials[k];
            x = block_sum<kBlockJoin>(x);
            __syncthreads();
            if (tid != 0) continue;
        } else {
            if (wave != w) continue;
            for (uint32_t k = first + lane; k < last; k += 64) x += partials[k];
            x = wave_sum(x);
            if (lane != kSumLane) continue;
        }
        if (out.tensor_sumsq) out.tensor_sumsq[i] = x;
        if (out.tensor_norm) out.tensor_norm[i] = (float)__builtin_sqrt(x);
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

// Each element is touched once: non-temporal loads and stores.  MI355X, OPT-1.3B
// bf16 gradients: 787 us, against 861 with non-temporal stores only and 863 without;
// 52 MB of fp32 whose three copies take turns in the last-level cache: 17.7 against
// 16.9 us, one copy alone 15.4 against 17.0.
constexpr int kNtClip = 3;
template <int DT>
__global__ __launch_bounds__(kBlockSweep) void clip_kernel(const DevSweep* __restrict__ groups, ClipRule rule,
                                                       float inv_scale, const adamw_loss_scale_state* __restrict__ amp)
{
    if (amp) inv_scale = (float)(1.0 / (double)amp->scale);
    double factor;
    if (!clip_factor(rule, *rule.sumsq, inv_scale, factor)) return;
    const float f = (float)factor;
    if (f == 1.0f) return;
    const DevSweep gr = groups[blockIdx.x];
    const Span<DT> sp(gr.addr, gr.n);
    GLOBAL u32x4* __restrict__ g4 = gptr<u32x4>(sp.body, 0);
    const uint32_t tid = threadIdx.x;
    const uint32_t parts = gr.part == kWholeChunk ? 1 : kXcdParts, part = gr.part == kWholeChunk ? 0 : gr.part;
    // tile t of kTileWords words goes to part t % parts
    const uint32_t first = (tid / kTileWords * parts + part) * kTileWords + tid % kTileWords;
    const uint32_t stride = kBlockSweep * parts;
    uint32_t at = 0;
    for (; at + kClipUnroll * stride <= sp.words; at += kClipUnroll * stride) {
        u32x4 q[kClipUnroll];
#pragma unroll
        for (int u = 0; u < kClipUnroll; ++u) q[u] = ld<kNtClip>(g4 + at + first + u * stride);
#pragma unroll
        for (int u = 0; u < kClipUnroll; ++u) st<kNtClip>(g4 + at + first + u * stride, scale_word<DT>(q[u], f));
    }
    for (uint32_t k = at + first; k < sp.words; k += stride) st<kNtClip>(g4 + k, scale_word<DT>(ld<kNtClip>(g4 + k), f));
    if (part != 0) return;
    if (tid < sp.head) scale1<DT>(sp.head_addr(tid), f);
    if (tid < sp.tail) scale1<DT>(sp.tail_addr(tid), f);
}

}  // namespace

// Occupancy caps by reserved LDS, as for the update kernels: four 256-lane workgroups
// per CU.  MI355X, clipping the OPT-1.3B bf16 gradients: 788 us with four, 789 with
// three, 804 with eight, 831 with two; norms of 26 MB of fp16: 8.0 us with four, 8.1 with
// five, 8.8 with three; of 2,000 fp32 tensors (580 MB): 86.7 with four, 87.4 with three, 88.4
// with eight, 96.0 with two; of 10,000 fp16 tensors: 765 with four, 771 with three, 769 with
// five.  Three gain on lists of long tensors among other passes (OPT-1.3B bf16 377 -> 365
// us, 4.3 GB of fp32 609 -> 601) and lose on a pass by itself (the sum's kernel 357 -> 370).
// (The sum's own 32 bytes of LDS count too.)
#ifndef ADAMW_LDS_CLIP
#define ADAMW_LDS_CLIP 40960
#endif
#ifndef ADAMW_LDS_NORM
#define ADAMW_LDS_NORM 40000
#endif

hipError_t launch_clip(adamw_dtype g_dtype, const DevSweep* groups, int64_t n_groups, const ClipRule& rule,
                       float inv_scale, const adamw_loss_scale_state* d_amp, hipStream_t stream)
{
    if (n_groups <= 0) return hipSuccess;
    const dim3 grid((unsigned)n_groups), block(kBlockSweep);
    if (g_dtype == ADAMW_F16)
        hipLaunchKernelGGL((clip_kernel<kF16>), grid, block, ADAMW_LDS_CLIP, stream, groups, rule, inv_scale, d_amp);
    else if (g_dtype == ADAMW_BF16)
        hipLaunchKernelGGL((clip_kernel<kBf16>), grid, block, ADAMW_LDS_CLIP, stream, groups, rule, inv_scale, d_amp);
    else
        hipLaunchKernelGGL((clip_kernel<kF32>), grid, block, ADAMW_LDS_CLIP, stream, groups, rule, inv_scale, d_amp);
    return hipGetLastError();
}

int64_t partial_count(int64_t n_chunks) { return n_chunks + (n_chunks + kJoin - 1) / kJoin; }
static_assert(kMaxSweepChunks <= (int64_t)kJoin * kJoin, "one workgroup joins the block sums");

template <bool FUSED>
static void launch_sums(adamw_dtype g_dtype, const DevSweep* groups, int64_t n_chunks,
                        double* partials, uint32_t* done, const NormOut& out, hipStream_t stream)
{
    const dim3 grid((unsigned)n_chunks), block(kBlockSweep);
    if (g_dtype == ADAMW_F16)
        hipLaunchKernelGGL((sumsq_kernel<kF16, FUSED>), grid, block, ADAMW_LDS_NORM, stream, groups, partials, done, out);
    else if (g_dtype == ADAMW_BF16)
        hipLaunchKernelGGL((sumsq_kernel<kBf16, FUSED>), grid, block, ADAMW_LDS_NORM, stream, groups, partials, done, out);
    else
        hipLaunchKernelGGL((sumsq_kernel<kF32, FUSED>), grid, block, ADAMW_LDS_NORM, stream, groups, partials, done, out);
}

hipError_t launch_sumsq(adamw_dtype g_dtype, const DevSweep* groups, int64_t n_chunks,
                        const uint32_t* tensor_first, int64_t n_tensors, double* partials, uint32_t* done, bool single,
                        const NormOut& out, hipStream_t stream)
{
    const bool per_tensor = (out.tensor_norm || out.tensor_sumsq) && n_tensors > 0;
    if (single && !per_tensor) {
        launch_sums<true>(g_dtype, groups, n_chunks, partials, done, out, stream);
        return hipGetLastError();
    }
    if (n_chunks > 0) {
        launch_sums<false>(g_dtype, groups, n_chunks, partials, done, out, stream);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    // an empty list's total is written by one workgroup all the same
    const int64_t blocks = !out.sumsq ? 0 : n_chunks > 0 ? (n_chunks + kJoin - 1) / kJoin : 1;
    const int64_t joins = blocks + (per_tensor ? (n_tensors + kTensorsPerGroup - 1) / kTensorsPerGroup : 0);
    if (joins == 0) return hipSuccess;
    hipLaunchKernelGGL(join_kernel, dim3((unsigned)joins), dim3(kBlockJoin), 0, stream, partials, (uint32_t)n_chunks,
                       (uint32_t)blocks, tensor_first, (uint32_t)n_tensors, done, out);
    return hipGetLastError();
}

}  // namespace adamw
