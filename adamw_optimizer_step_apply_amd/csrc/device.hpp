// device.hpp -- what the gfx950 kernels share: 16-byte vector types, global-memory
// accesses with a chosen cache policy, 16-bit <-> fp32 conversions, and the
// completion count by which a launch finds its last workgroup.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "adamw.h"
#include "layout.hpp"

namespace adamw {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <int N>
using words_t = uint32_t __attribute__((ext_vector_type(N)));

// Device addresses taken from the segment table are plain integers; casting them
// to the global address space lets the compiler emit global_load/global_store
// (rather than flat accesses, which also test the LDS aperture).
#define GLOBAL __attribute__((address_space(1)))
template <typename T>
__device__ __forceinline__ GLOBAL T* gptr(uint64_t addr, uint64_t elem_off)
{
    return reinterpret_cast<GLOBAL T*>(addr) + elem_off;
}
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------------------
// 16-bit <-> fp32.  A 32-bit word holds two 16-bit elements, the lower-addressed
// one in the low half.
// ---------------------------------------------------------------------------

template <bool F16>
__device__ __forceinline__ f32x2 widen2(uint32_t w)
{
    if constexpr (F16) {
        return __builtin_convertvector(__builtin_bit_cast(f16x2, w), f32x2);   // v_cvt_f32_f16 (exact)
    } else {
        f32x2 r;
        r.x = __uint_as_float(w << 16);            // bf16 is the top half of an fp32
        r.y = __uint_as_float(w & 0xffff0000u);
        return r;
    }
}

// Round two fp32 values to nearest-even 16-bit and pack them (v_cvt_pk_bf16_f32 /
// v_cvt_pk_f16_f32 under the default round-to-nearest-even mode).
template <bool F16>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi)
{
    f32x2 x = {lo, hi};
    if constexpr (F16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, f16x2));
    else return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2));
}

template <bool F16>
__device__ __forceinline__ float widen1(uint16_t h)
{
    if constexpr (F16) return (float)__builtin_bit_cast(_Float16, h);
    else return __uint_as_float((uint32_t)h << 16);
}

template <bool F16>
__device__ __forceinline__ uint16_t narrow1(float x)
{
    if constexpr (F16) return __builtin_bit_cast(uint16_t, (_Float16)x);
    else return __builtin_bit_cast(uint16_t, (__bf16)x);
}

// The cache policy of a streaming access: bit 0 of NT = non-temporal loads, bit 1 =
// non-temporal stores.
template <int NT, typename T>
__device__ __forceinline__ T ld(const GLOBAL T* p)
{
    if constexpr (NT & 1) return __builtin_nontemporal_load(p);
    else return *p;
}

template <int NT, typename T>
__device__ __forceinline__ void st(GLOBAL T* p, T v)
{
    if constexpr (NT & 2) __builtin_nontemporal_store(v, p);
    else *p = v;
}

// The grid's completion count, shared by the single-launch kernels.  Each
// workgroup counts itself in a first-level counter (b % kDoneLanes); the
// workgroup completing a first-level count rearms it and counts once in the
// second level, and the one completing that rearms it and returns true.
// Spreading the count over separate 256-byte lines keeps the same-address
// atomics, which the memory side serialises, to about nb / kDoneLanes +
// kDoneLanes per launch.  The atomics are relaxed: acquire-release ones at device scope
// would write back and invalidate the XCD's L2 in every workgroup.  So a count by
// itself orders only reads that every wave has consumed before the workgroup's barrier (an update's
// counter and loss scale).  A workgroup that hands a value over stores it at agent scope
// from the lane that counts, and that lane waits for the store (vmcnt 0) before it
// counts; the last workgroup loads such values at agent scope after its barrier
// (last_of and join in norm.hip).
struct DoneLane {
    uint32_t lanes, j, in_lane;
};

__device__ __forceinline__ DoneLane done_lane(uint32_t b, uint32_t nb)
{
    const uint32_t lanes = nb < (uint32_t)kDoneLanes ? nb : (uint32_t)kDoneLanes;
    const uint32_t j = b % lanes;
    return DoneLane{lanes, j, nb / lanes + (j < nb % lanes ? 1u : 0u)};
}

// The count alone, on 32-bit words (the low words of the counter lines), of
// workgroup b of nb that count themselves.
__device__ __forceinline__ bool grid_done(uint32_t* done, uint32_t b, uint32_t nb)
{
    const DoneLane d = done_lane(b, nb);
    uint32_t* first = done + (size_t)d.j * kDoneStrideWords;
    uint32_t* second = done + (size_t)kDoneLanes * kDoneStrideWords;
    if (__hip_atomic_fetch_add(first, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != d.in_lane - 1) return false;
    __hip_atomic_store(first, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (__hip_atomic_fetch_add(second, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != d.lanes - 1) return false;
    __hip_atomic_store(second, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return true;
}

// The count with a 0/1 verdict per workgroup, on 64-bit words: the count in the
// low half and the number of raised verdicts in the high half, so the verdicts
// travel in the atomics' own values.  The completer gets the number of lanes
// with a raised verdict in *lanes_hit.  Both forms leave every counter word at
// zero, so the update and check kernels of one stream share the lines.
__device__ __forceinline__ bool grid_done_verdict(uint32_t* done, uint32_t verdict, uint32_t* lanes_hit)
{
    const DoneLane d = done_lane(blockIdx.x, gridDim.x);
    uint64_t* first = reinterpret_cast<uint64_t*>(done + (size_t)d.j * kDoneStrideWords);
    uint64_t* second = reinterpret_cast<uint64_t*>(done + (size_t)kDoneLanes * kDoneStrideWords);
    const uint64_t prev = __hip_atomic_fetch_add(first, 1ull + ((uint64_t)verdict << 32), __ATOMIC_RELAXED,
                                                 __HIP_MEMORY_SCOPE_AGENT);
    if ((uint32_t)prev != d.in_lane - 1) return false;
    __hip_atomic_store(first, 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const uint64_t hit = ((prev >> 32) + verdict) != 0 ? 1ull : 0ull;
    const uint64_t prev2 = __hip_atomic_fetch_add(second, 1ull + (hit << 32), __ATOMIC_RELAXED,
                                                  __HIP_MEMORY_SCOPE_AGENT);
    if ((uint32_t)prev2 != d.lanes - 1) return false;
    __hip_atomic_store(second, 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *lanes_hit = (uint32_t)(prev2 >> 32) + (uint32_t)hit;
    return true;
}

__device__ __forceinline__ bool is_sum_of_squares(double s) { return s >= 0.0 && __builtin_isfinite(s); }

// The clipping factor of a sum of squares S, in binary64.  Returns false if S is no
// finite sum of squares (an inf or NaN gradient).  A factor of 0/0 (no gradient, no
// eps) clips nothing.
__device__ __forceinline__ bool clip_factor(const ClipRule& rule, double s, float inv_scale, double& factor)
{
    if (!is_sum_of_squares(s)) return false;
    const double c = (double)rule.max_norm / (__builtin_sqrt(s) * (double)inv_scale + (double)rule.eps);
    factor = c < 1.0 ? c : 1.0;
    return true;
}

}  // namespace adamw
