// muon.hip -- gfx950 (CDNA4) kernels of the Newton-Schulz products and the Muon step.
//
// The mathematics (adamw.h): from X = u / (|u| + eps), per step A = X X^T on the
// shorter side, B = b A + c A A, X <- a X + B X.  On a wide matrix (rows <= columns)
// A = X X^T and B X, on a tall one A = X^T X and X B, so A and B are squares of the
// shorter side; both are symmetric, and only the tiles on and below the diagonal are
// computed and written to both places.
//
// All three products are sums over the last index of both factors, C[i][j] = sum_k
// P[i][k] Q[j][k], the form in which every lane's operand of a matrix instruction
// is 16 bytes of a row:
//   gram   P = Q = X in the order whose rows are the shorter side
//   poly   P = Q = A
//   apply  wide: P = B, Q = X^T;  tall: P = X, Q = B
// X is therefore kept in both orders (hi and t); the tile leaves the accumulators through
// LDS, from where it is read once by rows and once by columns.
//
// Numerics.  A step multiplies a small singular value by a, five of them by 485, and with
// it the rounding of X.  So X is the pair hi + lo of fp16 (22 bits) under the power of two
// sx, the products take hi (11 bits), and the epilogue of apply forms
//   X' = (a + B_ii - fp16(B_ii)) hi + sum_k fp16(B)_ik hi_k + (a + B_ii) lo :
// the linear term, all there is of a small singular value, is exact to 22 bits; the diagonal of B, whose
// rounding would be the same for a whole row, is fp32; and lo takes part with the
// diagonal of B, nearly all of B once the singular values are near 1.  A's diagonal
// is treated alike in poly.  On matrices with a decaying spectrum (500 to 1000 rows,
// simulated in binary64 with these roundings) the result is 2.5e-4 from the exact one in
// the Frobenius norm, on normal random ones 3.6e-4 to 1.1e-3; fp16 X alone 3.7e-3 and
// bf16 throughout 3e-2.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "adamw.h"
#include "device.hpp"
#include "layout.hpp"
#include "muon_launch.hpp"

namespace adamw {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kLoScale = 2048.0f;   // lo is held as lo * 2^11, of the size of hi

__device__ __forceinline__ float pow2(int e) { return __builtin_ldexpf(1.0f, e); }

template <typename T>
__device__ __forceinline__ GLOBAL T* at(char* ws, uint64_t off)
{
    return gptr<T>((uint64_t)(uintptr_t)ws + off, 0);
}

// ---------------------------------------------------------------------------
// Prologue of a step: one lane.
// ---------------------------------------------------------------------------

__global__ void ns_prologue_kernel(float inv_loss_scale, ClipRule clip, int32_t* __restrict__ step,
                                   const int32_t* __restrict__ found_inf, const adamw_loss_scale_state* __restrict__ amp,
                                   NsScalars* __restrict__ out)
{
    if (threadIdx.x != 0 || blockIdx.x != 0) return;
    NsScalars s{1, 0.0f};
    const int32_t step0 = *step;
    bool take = step0 >= 0 && step0 != INT32_MAX && !(found_inf && *found_inf != 0);
    float mult = amp ? (float)(1.0 / (double)amp->scale) : inv_loss_scale;
    if (clip.sumsq) {
        double factor = 1.0;
        if (clip_factor(clip, *clip.sumsq, mult, factor)) mult = (float)((double)mult * factor);
        else take = false;
    }
    if (take) {
        s = NsScalars{0, mult};
        *step = step0 + 1;
    }
    *out = s;
}

// ---------------------------------------------------------------------------
// Moments: the sum of squares of each matrix, as a partial sum for each run of elements; in a
// step m = beta m + (1 - beta) g first, and u to the workspace.
// ---------------------------------------------------------------------------

enum { kInF32 = 0, kInBf16 = 1, kInF16 = 2 };

template <int IN>
__device__ __forceinline__ float load1(uint64_t base, uint64_t i)
{
    if constexpr (IN == kInF32) return *gptr<const float>(base, i);
    else return widen1<IN == kInF16>(*gptr<const uint16_t>(base, i));
}

// 8 elements from a 16-byte aligned address
template <int IN>
__device__ __forceinline__ void load8(uint64_t base, uint64_t i, float (&x)[8])
{
    if constexpr (IN == kInF32) {
        const GLOBAL f32x4* p = reinterpret_cast<const GLOBAL f32x4*>(gptr<const float>(base, i));
        const f32x4 a = p[0], b = p[1];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[k] = a[k];
            x[k + 4] = b[k];
        }
    } else {
        const u32x4 w = *reinterpret_cast<const GLOBAL u32x4*>(gptr<const uint16_t>(base, i));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const f32x2 v = widen2<IN == kInF16>(w[k]);
            x[2 * k] = v.x;
            x[2 * k + 1] = v.y;
        }
    }
}

__device__ __forceinline__ void store8_f32(GLOBAL float* p, const float (&x)[8])
{
    GLOBAL f32x4* q = reinterpret_cast<GLOBAL f32x4*>(p);
    q[0] = f32x4{x[0], x[1], x[2], x[3]};
    q[1] = f32x4{x[4], x[5], x[6], x[7]};
}

template <bool F16>
__device__ __forceinline__ u32x4 pack8(const float (&x)[8])
{
    return u32x4{narrow2<F16>(x[0], x[1]), narrow2<F16>(x[2], x[3]), narrow2<F16>(x[4], x[5]), narrow2<F16>(x[6], x[7])};
}

struct MomentCoef {
    float beta, omb;
    int nesterov;
};

__device__ __forceinline__ float moment(float g, float mult, float& m, const MomentCoef& c)
{
    const float og = c.omb * (g * mult);
    m = c.beta * m + og;
    return c.nesterov ? c.beta * m + og : m;
}

template <int IN, bool STEP, bool M16>
__global__ __launch_bounds__(kBlockMoments) void ns_moments_kernel(const DevMatrix* __restrict__ mats,
                                                                    const DevTile* __restrict__ tiles, char* ws,
                                                                    MomentCoef c)
{
    const NsScalars* sc = reinterpret_cast<const NsScalars*>(ws);
    float mult = 1.0f;
    if constexpr (STEP) {
        if (sc->skip) return;
        mult = sc->mult;
    }
    const DevTile t = tiles[blockIdx.x];
    const DevMatrix& mx = mats[t.mat];
    const uint64_t n = (uint64_t)mx.rows * (uint64_t)mx.cols, first = (uint64_t)t.row * kMomentElems;
    const uint32_t count = (uint32_t)(n - first < (uint64_t)kMomentElems ? n - first : (uint64_t)kMomentElems);
    const uint32_t packs = mx.flat16 ? count / 8 : 0, tid = threadIdx.x;
    const uint64_t in = mx.ptr[1];
    GLOBAL float* u = at<float>(ws, mx.u) + first;
    double sum = 0.0;
    for (uint32_t k = tid; k < packs; k += kBlockMoments) {
        const uint64_t i = first + (uint64_t)k * 8;
        float x[8];
        load8<IN>(in, i, x);
        if constexpr (STEP) {
            float m[8], v[8];
            load8<M16 ? kInBf16 : kInF32>(mx.ptr[2], i, m);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] = moment(x[e], mult, m[e], c);
                x[e] = v[e];
            }
            if constexpr (M16) *reinterpret_cast<GLOBAL u32x4*>(gptr<uint16_t>(mx.ptr[2], i)) = pack8<false>(m);
            else store8_f32(gptr<float>(mx.ptr[2], i), m);
            store8_f32(u + (size_t)k * 8, v);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += (double)x[e] * (double)x[e];
    }
    for (uint32_t k = packs * 8 + tid; k < count; k += kBlockMoments) {
        const uint64_t i = first + k;
        float x = load1<IN>(in, i);
        if constexpr (STEP) {
            float m = load1<M16 ? kInBf16 : kInF32>(mx.ptr[2], i);
            x = moment(x, mult, m, c);
            if constexpr (M16) *gptr<uint16_t>(mx.ptr[2], i) = narrow1<false>(m);
            else *gptr<float>(mx.ptr[2], i) = m;
            u[k] = x;
        }
        sum += (double)x * (double)x;
    }
    // in a fixed order: lanes of a wave by halves, then the waves
#pragma unroll
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
    __shared__ double part[kBlockMoments / 64];
    if (tid % 64 == 0) part[tid / 64] = sum;
    __syncthreads();
    if (tid == 0) {
        double s = 0.0;
#pragma unroll
        for (int w = 0; w < kBlockMoments / 64; ++w) s += part[w];
        at<double>(ws, mx.partials)[t.row] = s;
    }
}

// ---------------------------------------------------------------------------
// Normalisation: X = u / (|u| + eps) into hi, lo and t, zeros in the padding.
// ---------------------------------------------------------------------------

// x * 2^sx as hi + lo * 2^-11
__device__ __forceinline__ void split_pair(float x, _Float16& hi, _Float16& lo)
{
    hi = (_Float16)x;
    lo = (_Float16)((x - (float)hi) * kLoScale);
}

template <int IN>
__global__ __launch_bounds__(256) void ns_normalise_kernel(const DevMatrix* __restrict__ mats,
                                                           const DevTile* __restrict__ tiles, char* ws, float eps,
                                                           int sx, int step)
{
    if (step && reinterpret_cast<const NsScalars*>(ws)->skip) return;
    const DevTile t = tiles[blockIdx.x];
    const DevMatrix& mx = mats[t.mat];
    const uint32_t tid = threadIdx.x;
    // the sum of the partial sums, by every workgroup alike
    __shared__ double part[4];
    const GLOBAL double* partials = at<const double>(ws, mx.partials);
    double sum = 0.0;
    for (uint32_t k = tid; k < mx.n_partials; k += 256) sum += partials[k];
#pragma unroll
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
    if (tid % 64 == 0) part[tid / 64] = sum;
    __syncthreads();
    sum = ((part[0] + part[1]) + part[2]) + part[3];
    const double len = __builtin_sqrt(sum) + (double)eps;
    // a zero matrix without eps is zero
    const double scale = len == 0.0 ? 0.0 : __builtin_ldexp(1.0, sx) / len;

    constexpr int kLd = 72;   // 144-byte rows: 16-byte reads stay aligned
    __shared__ alignas(16) _Float16 hi[kPad * kLd];
    __shared__ alignas(16) _Float16 lo[kPad * kLd];
    const uint32_t r0 = t.row * kPad, c0 = t.col * kPad;
    const uint64_t in = step ? (uint64_t)(uintptr_t)ws + mx.u : mx.ptr[1];
    for (uint32_t k = 0; k < kPad / 4; ++k) {
        const uint32_t r = k * 4 + tid / 64, c = tid % 64;
        float x = 0.0f;
        if (r0 + r < (uint32_t)mx.rows && c0 + c < (uint32_t)mx.cols)
            x = (float)((double)load1<IN>(in, (uint64_t)(r0 + r) * (uint64_t)mx.cols + c0 + c) * scale);
        split_pair(x, hi[r * kLd + c], lo[r * kLd + c]);
    }
    __syncthreads();
    for (uint32_t k = tid; k < kPad * 8; k += 256) {
        const uint32_t r = k / 8, c = k % 8 * 8;
        const uint64_t o = (uint64_t)(r0 + r) * (uint64_t)mx.cp + c0 + c;
        *reinterpret_cast<GLOBAL f16x8*>(at<_Float16>(ws, mx.hi) + o) = *reinterpret_cast<const f16x8*>(hi + r * kLd + c);
        *reinterpret_cast<GLOBAL f16x8*>(at<_Float16>(ws, mx.lo) + o) = *reinterpret_cast<const f16x8*>(lo + r * kLd + c);
        f16x8 v;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = hi[(c + e) * kLd + r];
        *reinterpret_cast<GLOBAL f16x8*>(at<_Float16>(ws, mx.t) + (uint64_t)(c0 + r) * (uint64_t)mx.rp + r0 + c) = v;
    }
}

// ---------------------------------------------------------------------------
// Products
// ---------------------------------------------------------------------------

enum NsOp { kGram, kPoly, kApply, kLast };

struct ProductArgs {
    float a, b, c;
    int sx, sa, sb;
    int parity;      // of the product step: which of the two buffers X is in
    int step;        // a Muon step: its skip mark is looked at
    float lr, decay, lrwd;   // a step's last epilogue
};

__device__ __forceinline__ f32x16 mfma(f16x8 a, f16x8 b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// 16 bytes for every lane of the wave from its own address to LDS, lane after lane from `to` on
__device__ __forceinline__ void load_to_lds(const GLOBAL char* from, char* to)
{
    __builtin_amdgcn_global_load_lds(from, (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}

template <int KIND>
struct TileShape;
template <>
struct TileShape<0> {
    static constexpr int side = 256, wy = 2, wx = 4;
};
template <>
struct TileShape<1> {
    static constexpr int side = 128, wy = 2, wx = 2;
};
template <>
struct TileShape<2> {
    static constexpr int side = 64, wy = 2, wx = 2;
};

// Loads `side` rows of one summing step (kPad elements, 128 bytes a row) of a factor into
// LDS without passing registers.  A wave's access fills 8 rows (1 KiB) in order; the 16-byte words of row r
// are exchanged, word c in place c ^ (r & 7), by the addresses that the lanes read from,
// so that the reads of a matrix instruction's operand, one word of 32 rows each, spread
// over all banks.  Rows past the matrix read its last row again; what they give is not stored.
template <int SIDE, int WAVES>
struct Stage {
    static constexpr int kLoads = SIDE / 8 / WAVES;
    const GLOBAL char* src[kLoads];
    uint32_t lds[kLoads];

    __device__ __forceinline__ void init(const GLOBAL _Float16* p, uint32_t row0, uint32_t rows, uint32_t ld, uint32_t wave,
                                         uint32_t lane)
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t r = (wave * kLoads + (uint32_t)i) * 8 + lane / 8;
            const uint32_t row = row0 + r < rows ? row0 + r : rows - 1;
            src[i] = reinterpret_cast<const GLOBAL char*>(p + (uint64_t)row * ld) + ((lane ^ (lane >> 3)) & 7u) * 16;
            lds[i] = (wave * kLoads + (uint32_t)i) * 1024;
        }
    }
    __device__ __forceinline__ void load(char* buf, uint32_t k)
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            load_to_lds(src[i] + (uint64_t)k * (kPad * 2), buf + lds[i]);
    }
};

__device__ __forceinline__ f16x8 operand(const char* buf, uint32_t row, uint32_t word)
{
    return *reinterpret_cast<const f16x8*>(buf + row * 128 + ((word ^ (row & 7u)) << 4));
}

__device__ __forceinline__ uint32_t join_master(uint32_t p16, uint32_t r16)
{
    return (p16 << 16) + (uint32_t)(int32_t)(int16_t)(uint16_t)r16;
}

// the nearest bf16, ties away from zero; a NaN keeps its high half, quiet
__device__ __forceinline__ uint32_t split_master(uint32_t w, uint32_t& r16)
{
    const bool nan = (w & 0x7fffffffu) > 0x7f800000u;
    const uint32_t hi = nan ? (w >> 16) | 0x0040u : (w >> 16) + ((w >> 15) & 1u);
    r16 = (w - (hi << 16)) & 0xffffu;
    return hi & 0xffffu;
}

// The end of the list's work: o = 8 neighbouring elements of the result, from element i.
// V: 16-byte accesses; else the first n of the 8 one by one.
template <int END>
__device__ __forceinline__ void end_elem(const DevMatrix& mx, uint64_t i, float o, float stepf, const ProductArgs& q)
{
    if constexpr (END == kEndOrtho) {
        *gptr<uint16_t>(mx.ptr[0], i) = narrow1<false>(o);
    } else if constexpr (END == kEndMixedBf16 || END == kEndMixedF16) {
        GLOBAL float* w = gptr<float>(mx.ptr[3], i);
        const float x = *w * q.decay - stepf * o;
        *w = x;
        *gptr<uint16_t>(mx.ptr[0], i) = narrow1<END == kEndMixedF16>(x);
    } else if constexpr (END == kEndSplit) {
        GLOBAL uint16_t* p = gptr<uint16_t>(mx.ptr[0], i);
        GLOBAL uint16_t* r = gptr<uint16_t>(mx.ptr[3], i);
        const float x = __uint_as_float(join_master(*p, *r)) * q.decay - stepf * o;
        uint32_t r16;
        *p = (uint16_t)split_master(__float_as_uint(x), r16);
        *r = (uint16_t)r16;
    } else {
        GLOBAL uint16_t* p = gptr<uint16_t>(mx.ptr[0], i);
        const float pf = widen1<false>(*p);
        if constexpr (END == kEndPure) {
            *p = narrow1<false>(pf * q.decay - stepf * o);
        } else {
            const float cf = END == kEndKahan ? widen1<false>(*gptr<uint16_t>(mx.ptr[3], i)) : *gptr<float>(mx.ptr[3], i);
            const float s = cf + (-(q.lrwd * pf) - stepf * o);
            const uint16_t pn = narrow1<false>(pf + s);
            const float rest = s - (widen1<false>(pn) - pf);
            *p = pn;
            if constexpr (END == kEndKahan) *gptr<uint16_t>(mx.ptr[3], i) = narrow1<false>(rest);
            else *gptr<float>(mx.ptr[3], i) = rest;
        }
    }
}

template <int END>
__device__ __forceinline__ void end_eight(const DevMatrix& mx, uint64_t i, const float (&o)[8], float stepf,
                                          const ProductArgs& q)
{
    GLOBAL u32x4* p16 = reinterpret_cast<GLOBAL u32x4*>(gptr<uint16_t>(mx.ptr[0], i));
    float x[8];
    if constexpr (END == kEndOrtho) {
        *p16 = pack8<false>(o);
    } else if constexpr (END == kEndMixedBf16 || END == kEndMixedF16) {
        load8<kInF32>(mx.ptr[3], i, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * q.decay - stepf * o[e];
        store8_f32(gptr<float>(mx.ptr[3], i), x);
        *p16 = pack8<END == kEndMixedF16>(x);
    } else if constexpr (END == kEndSplit) {
        GLOBAL u32x4* r16 = reinterpret_cast<GLOBAL u32x4*>(gptr<uint16_t>(mx.ptr[3], i));
        const u32x4 pw = *p16, rw = *r16;
        u32x4 pn, rn;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t r0, r1;
            const float a = __uint_as_float(join_master(pw[e] & 0xffffu, rw[e] & 0xffffu)) * q.decay - stepf * o[2 * e];
            const float b = __uint_as_float(join_master(pw[e] >> 16, rw[e] >> 16)) * q.decay - stepf * o[2 * e + 1];
            const uint32_t h0 = split_master(__float_as_uint(a), r0), h1 = split_master(__float_as_uint(b), r1);
            pn[e] = h0 | h1 << 16;
            rn[e] = r0 | r1 << 16;
        }
        *p16 = pn;
        *r16 = rn;
    } else {
        load8<kInBf16>((uint64_t)mx.ptr[0], i, x);
        if constexpr (END == kEndPure) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = x[e] * q.decay - stepf * o[e];
            *p16 = pack8<false>(x);
        } else {
            float c[8], s[8];
            load8<END == kEndKahan ? kInBf16 : kInF32>(mx.ptr[3], i, c);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = c[e] + (-(q.lrwd * x[e]) - stepf * o[e]);
            float sum[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] = x[e] + s[e];
            const u32x4 pn = pack8<false>(sum);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f32x2 v = widen2<false>(pn[e]);
                c[2 * e] = s[2 * e] - (v.x - x[2 * e]);
                c[2 * e + 1] = s[2 * e + 1] - (v.y - x[2 * e + 1]);
            }
            *p16 = pn;
            if constexpr (END == kEndKahan) *reinterpret_cast<GLOBAL u32x4*>(gptr<uint16_t>(mx.ptr[3], i)) = pack8<false>(c);
            else store8_f32(gptr<float>(mx.ptr[3], i), c);
        }
    }
}

// The element of row r among 8 from column c on, if the diagonal passes there.
__device__ __forceinline__ void store_diagonal(GLOBAL float* d, uint32_t r, uint32_t c, const float (&v)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (r == c + e) d[r] = v[e];
}

template <int KIND, int OP, int END>
__global__ __launch_bounds__(TileShape<KIND>::wy * TileShape<KIND>::wx * 64) void ns_product_kernel(
    const DevMatrix* __restrict__ mats, const DevTile* __restrict__ tiles, char* ws, ProductArgs q)
{
    using S = TileShape<KIND>;
    constexpr int WAVES = S::wy * S::wx, WR = S::side / S::wy, WC = S::side / S::wx;   // a wave's part of the tile
    constexpr int MI = WR / 32, NI = WC / 32;
    constexpr int kStageBytes = S::side * kPad * 2;
    constexpr int kEpiLd = WC + 8;                      // floats: rows 4 apart fall on the other half of the banks
    constexpr int kEpiBytes = 32 * kEpiLd * 4;          // one wave's 32 rows on their way out
    static_assert(WAVES * kEpiBytes <= 4 * kStageBytes, "the epilogue takes the place of the operands");
    __shared__ alignas(16) char lds[4 * kStageBytes];
    if (q.step && reinterpret_cast<const NsScalars*>(ws)->skip) return;

    const DevTile t = tiles[blockIdx.x];
    const DevMatrix& mx = mats[t.mat];
    const uint32_t tid = threadIdx.x, lane = tid & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t rp = (uint32_t)mx.rp, cp = (uint32_t)mx.cp, sp = (uint32_t)mx.sp;
    const bool tall = mx.tall != 0;
    // X in its own order and transposed: the one that apply reads changes its buffer with every step
    const uint64_t hi_now = tall && q.parity ? mx.y : mx.hi, t_now = !tall && q.parity ? mx.y : mx.t;
    const uint64_t hi_next = tall && !q.parity ? mx.y : mx.hi, t_next = !tall && !q.parity ? mx.y : mx.t;

    const GLOBAL _Float16 *P, *Q;
    uint32_t rows_p, rows_q, ld;   // ld: elements summed
    if constexpr (OP == kGram) {
        P = Q = at<const _Float16>(ws, tall ? t_now : hi_now);
        rows_p = rows_q = sp;
        ld = tall ? rp : cp;
    } else if constexpr (OP == kPoly) {
        P = Q = at<const _Float16>(ws, mx.a);
        rows_p = rows_q = ld = sp;
    } else {
        P = at<const _Float16>(ws, tall ? hi_now : mx.b);
        Q = at<const _Float16>(ws, tall ? mx.b : t_now);
        rows_p = rp;
        rows_q = cp;
        ld = sp;
    }
    const uint32_t r0 = t.row * S::side, c0 = t.col * S::side;

    Stage<S::side, WAVES> sp_, sq_;
    sp_.init(P, r0, rows_p, ld, wave, lane);
    sq_.init(Q, c0, rows_q, ld, wave, lane);
    const uint32_t wr = wave / S::wx * WR, wc = wave % S::wx * WC;   // the wave's place in the tile

    f32x16 acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

    const uint32_t nk = ld / kPad;
    sp_.load(lds, 0);
    sq_.load(lds + kStageBytes, 0);
    for (uint32_t k = 0; k < nk; ++k) {
        // the loads of this summing step have arrived, and every wave is past its reads of the last
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        const char* bp = lds + (k & 1u) * 2 * kStageBytes;
        const char* bq = bp + kStageBytes;
        if (k + 1 < nk) {
            char* nb = lds + ((k + 1) & 1u) * 2 * kStageBytes;
            sp_.load(nb, k + 1);
            sq_.load(nb + kStageBytes, k + 1);
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            f16x8 a[MI], b[NI];
            const uint32_t word = (uint32_t)kk * 2 + (lane >> 5);
#pragma unroll
            for (int i = 0; i < MI; ++i) a[i] = operand(bp, wr + i * 32 + (lane & 31u), word);
#pragma unroll
            for (int j = 0; j < NI; ++j) b[j] = operand(bq, wc + j * 32 + (lane & 31u), word);
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j) acc[i][j] = mfma(a[i], b[j], acc[i][j]);
        }
    }
    __syncthreads();   // the operands' room is free

    // Epilogue, 32 rows of the wave's part at a time through LDS of its own: 8 neighbours of a row
    // to a lane, and for what is kept in both orders then 8 of a column.
    float* out = reinterpret_cast<float*>(lds + wave * kEpiBytes);
    constexpr int kRowPacks = WC / 8;
    const float stepf = OP == kLast ? (float)((double)q.lr * mx.factor) : 0.0f;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                out[((e & 3) + 8 * (e >> 2) + 4 * (lane >> 5)) * kEpiLd + j * 32 + (lane & 31u)] = acc[i][j][e];
        __builtin_amdgcn_wave_barrier();
        const uint32_t row0 = r0 + wr + (uint32_t)i * 32, col0 = c0 + wc;
#pragma unroll
        for (int h = 0; h < 32 * kRowPacks / 64; ++h) {
            const uint32_t k = (uint32_t)h * 64 + lane, lr = k / kRowPacks, lc = k % kRowPacks * 8;
            const uint32_t r = row0 + lr, c = col0 + lc;
            float* cell = out + lr * kEpiLd + lc;
            float v[8];
            {
                const f32x4 x = *reinterpret_cast<const f32x4*>(cell), y = *reinterpret_cast<const f32x4*>(cell + 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] = x[e];
                    v[e + 4] = y[e];
                }
            }
            const bool inside = OP == kGram || OP == kPoly ? r < sp && c < sp : r < rp && c < cp;
            if (inside) {
                if constexpr (OP == kGram || OP == kPoly) {
                    if constexpr (OP == kGram) {
                        const float f = pow2(q.sa - 2 * q.sx);
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] *= f;
                        store_diagonal(at<float>(ws, mx.da), r, c, v);
                    } else {
                        // b A + c A A, with A's diagonal in fp32: (A + E)(A + E) = A A + (e_r + e_c) A + E E
                        const f16x8 ah = *reinterpret_cast<const GLOBAL f16x8*>(at<const _Float16>(ws, mx.a) +
                                                                                (uint64_t)r * sp + c);
                        const GLOBAL float* da = at<const float>(ws, mx.da);
                        const float f = pow2(-q.sa);
                        const float dr = da[r], er = (dr - (float)(_Float16)dr) * f;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float dc = da[c + e], ec = (dc - (float)(_Float16)dc) * f;
                            float x = (float)ah[e] * f, sq = v[e] * (f * f) + (er + ec) * x;
                            if (r == c + e) {
                                sq += er * er;
                                x += er;
                            }
                            v[e] = (q.b * x + q.c * sq) * pow2(q.sb);
                        }
                        store_diagonal(at<float>(ws, mx.db), r, c, v);
                    }
                    f16x8 w;
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = (_Float16)v[e];
                    *reinterpret_cast<GLOBAL f16x8*>(at<_Float16>(ws, OP == kGram ? mx.a : mx.b) + (uint64_t)r * sp + c) = w;
                } else {
                    const uint64_t o = (uint64_t)r * cp + c;
                    const f16x8 hi = *reinterpret_cast<const GLOBAL f16x8*>(at<const _Float16>(ws, hi_now) + o);
                    const f16x8 lo = *reinterpret_cast<const GLOBAL f16x8*>(at<const _Float16>(ws, mx.lo) + o);
                    const GLOBAL float* db = at<const float>(ws, mx.db);
                    const float f = pow2(-q.sb);
                    // X' * 2^sx
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float d = db[tall ? c + e : r], rest = (d - (float)(_Float16)d) * f;
                        v[e] = (q.a + rest) * (float)hi[e] + v[e] * f + (q.a + d * f) * ((float)lo[e] * (1.0f / kLoScale));
                    }
                    if constexpr (OP == kApply) {
                        f16x8 h8, l8;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            _Float16 x, y;
                            split_pair(v[e], x, y);
                            h8[e] = x;
                            l8[e] = y;
                        }
                        *reinterpret_cast<GLOBAL f16x8*>(at<_Float16>(ws, hi_next) + o) = h8;
                        *reinterpret_cast<GLOBAL f16x8*>(at<_Float16>(ws, mx.lo) + o) = l8;
                    } else if (r < (uint32_t)mx.rows && c < (uint32_t)mx.cols) {
                        const float g = pow2(-q.sx);
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] *= g;
                        const uint64_t i0 = (uint64_t)r * (uint64_t)mx.cols + c;
                        if (mx.row16) {
                            end_eight<END>(mx, i0, v, stepf, q);
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (c + e < (uint32_t)mx.cols) end_elem<END>(mx, i0 + e, v[e], stepf, q);
                        }
                    }
                }
                if constexpr (OP != kLast) {
                    *reinterpret_cast<f32x4*>(cell) = f32x4{v[0], v[1], v[2], v[3]};
                    *reinterpret_cast<f32x4*>(cell + 4) = f32x4{v[4], v[5], v[6], v[7]};
                }
            }
        }
        __builtin_amdgcn_wave_barrier();
        if constexpr (OP != kLast) {
            // by columns: 8 of a column to a lane, 4 lanes to a column of the 32 rows
            const bool both = OP == kApply || t.row != t.col;   // a tile on the diagonal is its own mirror
            GLOBAL _Float16* dst = at<_Float16>(ws, OP == kGram ? mx.a : OP == kPoly ? mx.b : t_next);
            const uint32_t lim_r = OP == kApply ? rp : sp, lim_c = OP == kApply ? cp : sp;
#pragma unroll
            for (int h = 0; h < WC * 4 / 64; ++h) {
                const uint32_t k = (uint32_t)h * 64 + lane, lc = k / 4, lr = k % 4 * 8;
                const uint32_t r = row0 + lr, c = col0 + lc;
                f16x8 w;
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = (_Float16)out[(lr + e) * kEpiLd + lc];
                if (both && r < lim_r && c < lim_c)
                    *reinterpret_cast<GLOBAL f16x8*>(dst + (uint64_t)c * lim_r + r) = w;
            }
            __builtin_amdgcn_wave_barrier();
        }
    }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------

hipError_t launch_ns_prologue(const adamw_muon_hparams& hp, const ClipRule& clip, int32_t* d_step,
                              const int32_t* d_found_inf, const adamw_loss_scale_state* d_amp, char* ws,
                              hipStream_t stream)
{
    ns_prologue_kernel<<<1, 64, 0, stream>>>(hp.inv_loss_scale, clip, d_step, d_found_inf, d_amp,
                                             reinterpret_cast<NsScalars*>(ws));
    return hipGetLastError();
}

namespace {

template <int KIND, int OP, int END>
hipError_t launch_product(const NsCall& call, const NsLaunch& l, const ProductArgs& q, hipStream_t stream)
{
    ns_product_kernel<KIND, OP, END><<<(uint32_t)l.count, TileShape<KIND>::wy * TileShape<KIND>::wx * 64, 0, stream>>>(
        call.mats, call.tiles + l.first, call.ws, q);
    return hipGetLastError();
}

template <int OP, int END = 0>
hipError_t product(const NsCall& call, const NsLaunch& l, const ProductArgs& q, hipStream_t stream)
{
    return l.kind == 0 ? launch_product<0, OP, END>(call, l, q, stream)
         : l.kind == 1 ? launch_product<1, OP, END>(call, l, q, stream)
                       : launch_product<2, OP, END>(call, l, q, stream);
}

hipError_t last_product(const NsCall& call, const NsLaunch& l, const ProductArgs& q, hipStream_t stream)
{
    switch (call.kind.end) {
    case kEndOrtho: return product<kLast, kEndOrtho>(call, l, q, stream);
    case kEndMixedBf16: return product<kLast, kEndMixedBf16>(call, l, q, stream);
    case kEndMixedF16: return product<kLast, kEndMixedF16>(call, l, q, stream);
    case kEndSplit: return product<kLast, kEndSplit>(call, l, q, stream);
    case kEndPure: return product<kLast, kEndPure>(call, l, q, stream);
    case kEndKahan: return product<kLast, kEndKahan>(call, l, q, stream);
    default: return product<kLast, kEndKahan32>(call, l, q, stream);
    }
}

template <int IN>
hipError_t moments(const NsCall& call, const NsLaunch& l, bool step, const MomentCoef& c, hipStream_t stream)
{
    const DevTile* tiles = call.tiles + l.first;
    const dim3 grid((uint32_t)l.count), block(kBlockMoments);
    if (!step) ns_moments_kernel<IN, false, false><<<grid, block, 0, stream>>>(call.mats, tiles, call.ws, c);
    else if (call.kind.m16) ns_moments_kernel<IN, true, true><<<grid, block, 0, stream>>>(call.mats, tiles, call.ws, c);
    else ns_moments_kernel<IN, true, false><<<grid, block, 0, stream>>>(call.mats, tiles, call.ws, c);
    return hipGetLastError();
}

template <int IN>
hipError_t normalise(const NsCall& call, const NsLaunch& l, bool step, hipStream_t stream)
{
    ns_normalise_kernel<IN><<<(uint32_t)l.count, 256, 0, stream>>>(call.mats, call.tiles + l.first, call.ws, call.ns.eps,
                                                                   call.scales.sx, step);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ns_batch(const NsCall& call, const NsBatch& batch, hipStream_t stream)
{
    const bool step = call.kind.end != kEndOrtho;
    const int in = call.kind.in == ADAMW_F32 ? kInF32 : call.kind.in == ADAMW_BF16 ? kInBf16 : kInF16;
    MomentCoef mc{};
    ProductArgs q{};
    q.a = call.ns.a;
    q.b = call.ns.b;
    q.c = call.ns.c;
    q.sx = call.scales.sx;
    q.sa = call.scales.sa;
    q.sb = call.scales.sb;
    q.step = step;
    if (step) {
        mc = MomentCoef{call.hp.momentum, 1.0f - call.hp.momentum, call.hp.nesterov};
        const double lr = (double)call.hp.lr, wd = (double)call.hp.weight_decay;
        q.lr = call.hp.lr;
        q.decay = (float)(1.0 - lr * wd);
        q.lrwd = (float)(lr * wd);
    }
    hipError_t e = in == kInF32 ? moments<kInF32>(call, batch.moments, step, mc, stream)
                 : in == kInBf16 ? moments<kInBf16>(call, batch.moments, step, mc, stream)
                                 : moments<kInF16>(call, batch.moments, step, mc, stream);
    if (e != hipSuccess) return e;
    e = step || in == kInF32 ? normalise<kInF32>(call, batch.normalise, step, stream)
      : in == kInBf16 ? normalise<kInBf16>(call, batch.normalise, step, stream)
                      : normalise<kInF16>(call, batch.normalise, step, stream);
    if (e != hipSuccess) return e;
    for (int k = 0; k < call.ns.steps; ++k) {
        q.parity = k & 1;
        if ((e = product<kGram>(call, batch.square, q, stream)) != hipSuccess) return e;
        if ((e = product<kPoly>(call, batch.square, q, stream)) != hipSuccess) return e;
        e = k + 1 < call.ns.steps ? product<kApply>(call, batch.apply, q, stream) : last_product(call, batch.apply, q, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace adamw
