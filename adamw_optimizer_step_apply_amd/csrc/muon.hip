// muon.hip -- gfx950 (CDNA4) kernels of the Newton-Schulz products and the Muon step.
//
// The mathematics (adamw.h): from X = u / (|u| + eps), per step A = X X^T on the
// shorter side, B = b A + c A A, X <- a X + B X.  On a wide matrix (rows <= columns)
// A = X X^T and B X, on a tall one A = X^T X and X B, so A and B are squares of the
// shorter side; both are symmetric, and only the tiles on and below the diagonal are
// computed and written to both places.
//
// X is held wide, transposed where the matrix is tall, so that A and B belong to its rows.  A tile of a product
// C[i][j] = sum_k P[i][k] Q[k][j] takes P by rows, 16 bytes of a row for a lane's operand of a matrix
// instruction; A and B are symmetric, so Q is by rows too in gram (Q = P = X, transposed) and
// poly (Q = P = A), while in apply (P = B, Q = X) its operands are columns, which LDS
// returns transposed (ds_read_b64_tr_b16).
//
// Numerics.  A step multiplies a small singular value by a, five of them by 485, and with
// it the rounding of X.  So X is the pair hi + lo of fp16 (22 bits) under the power of two
// sx, the products take hi (11 bits), and the epilogue of apply forms
//   X' = (a + B_ii - fp16(B_ii)) hi + sum_k fp16(B)_ik hi_k + (a + B_ii) lo :
// the linear term, all there is of a small singular value, is exact to 22 bits; the diagonal of B, whose
// rounding would be the same for a whole row, is fp32; and in the last steps lo takes part with the
// diagonal of B, nearly all of B once the singular values are near 1.  In the steps before those its factor is a alone:
// where X has no singular value lo has to go the way of a hi, whose rounding it undoes, and B_ii lo would be left over and be
// multiplied by a in every step that follows (a 65 x 65 matrix of rank one after eight steps: 0.2 off with B_ii in all of
// them, 1.2e-3 with it in three; normal random matrices of full rank the other way round, 1.4e-3 and 2e-3).  A's diagonal
// is treated like B's in poly.  Simulated in binary64 with these roundings (65 to 768 rows), five steps: 3.5e-4 to 8e-4 from
// the definition in the Frobenius norm on full rank, 2e-4 to 1.2e-3 on rank 1 to 60, with noise of 1e-3 and without;
// fp16 X alone 3.7e-3 and bf16 throughout 3e-2 on full rank.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "adamw.h"
#include "device.hpp"
#include "layout.hpp"
#include "muon_launch.hpp"

namespace adamw {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr float kLoScale = 2048.0f;   // lo is held as lo * 2^11, of the size of hi

__device__ __forceinline__ float pow2(int e) { return __builtin_ldexpf(1.0f, e); }

template <typename T>
__device__ __forceinline__ GLOBAL T* at(char* ws, uint64_t off)
{
    return gptr<T>((uint64_t)(uintptr_t)ws + off, 0);
}

// ---------------------------------------------------------------------------
// Whether a step is taken, and its gradients' multiplier.
// ---------------------------------------------------------------------------

struct StepRule {
    float inv_loss_scale;
    ClipRule clip;
    const int32_t* step;
    const int32_t* found_inf;
    const adamw_loss_scale_state* amp;
};

__device__ __forceinline__ bool begin_step(const StepRule& rule, float& mult)
{
    const int32_t step = *rule.step, flag = rule.found_inf ? *rule.found_inf : 0;
    const float scale = rule.amp ? rule.amp->scale : 1.0f;
    const double sumsq = rule.clip.sumsq ? *rule.clip.sumsq : 0.0;
    mult = rule.amp ? (float)(1.0 / (double)scale) : rule.inv_loss_scale;
    if (step < 0 || step == INT32_MAX || flag != 0) return false;
    if (rule.clip.sumsq) {
        double factor;
        if (!clip_factor(rule.clip, sumsq, mult, factor)) return false;
        mult = (float)((double)mult * factor);
    }
    return true;
}

__global__ void ns_count_kernel(StepRule rule, int32_t* step)
{
    float mult;
    if (threadIdx.x == 0 && begin_step(rule, mult)) *step += 1;
}

// ---------------------------------------------------------------------------
// Moments: the sum of squares of each matrix, as a partial sum for each run of elements; in a
// step m = beta m + (1 - beta) g first, and u to the workspace.
//
// Bound by HBM: a step reads g and m and writes m and u, 14 bytes an element with fp32 m, at 4.7 TB/s (302 M elements
// in 904 us on MI355X), the rate of a large copy.  Each workgroup sums one run of 4,096 elements or more into one
// binary64 partial, so that no atomic orders the sum and the readers add at most 256 of them.
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
                                                                    MomentCoef c, StepRule rule)
{
    float mult = 1.0f;
    if constexpr (STEP) {
        const bool take = begin_step(rule, mult);
        if (blockIdx.x == 0 && threadIdx.x == 0) *reinterpret_cast<NsScalars*>(ws) = NsScalars{take ? 0 : 1};
        if (!take) return;
    }
    constexpr int IN_M = M16 ? kInBf16 : kInF32;
    const DevTile t = tiles[blockIdx.x];
    const DevMatrix& mx = mats[t.mat];
    const uint64_t n = (uint64_t)mx.rows * (uint64_t)mx.cols, first = (uint64_t)t.row * mx.chunk;
    const uint32_t count = (uint32_t)(n - first < mx.chunk ? n - first : mx.chunk);
    const uint32_t packs = mx.flat16 ? count / 8 : 0, tid = threadIdx.x;
    const uint64_t in = mx.ptr[1];
    GLOBAL float* u = at<float>(ws, t.parts.u()) + first;
    double sum = 0.0;
    constexpr int U = 2;   // packs of a lane under way together
    for (uint32_t k0 = tid; k0 < packs; k0 += kBlockMoments * U) {
        float x[U][8], m[U][8];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            // past the end the lane's first pack again, which is not used
            const uint32_t k = k0 + j * kBlockMoments < packs ? k0 + j * kBlockMoments : k0;
            load8<IN>(in, first + (uint64_t)k * 8, x[j]);
            if constexpr (STEP) load8<IN_M>(mx.ptr[2], first + (uint64_t)k * 8, m[j]);
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const uint32_t k = k0 + j * kBlockMoments;
            if (k >= packs) break;
            if constexpr (STEP) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[j][e] = moment(x[j][e], mult, m[j][e], c);
                const uint64_t i = first + (uint64_t)k * 8;
                if constexpr (M16) *reinterpret_cast<GLOBAL u32x4*>(gptr<uint16_t>(mx.ptr[2], i)) = pack8<false>(m[j]);
                else store8_f32(gptr<float>(mx.ptr[2], i), m[j]);
                store8_f32(u + (size_t)k * 8, x[j]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += (double)x[j][e] * (double)x[j][e];
        }
    }
    constexpr int V = 8;   // elements of a lane under way together
    for (uint32_t k0 = packs * 8 + tid; k0 < count; k0 += kBlockMoments * V) {
        float x[V], m[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint32_t k = k0 + j * kBlockMoments < count ? k0 + j * kBlockMoments : k0;
            x[j] = load1<IN>(in, first + k);
            if constexpr (STEP) m[j] = load1<IN_M>(mx.ptr[2], first + k);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint32_t k = k0 + j * kBlockMoments;
            if (k >= count) break;
            if constexpr (STEP) {
                x[j] = moment(x[j], mult, m[j], c);
                if constexpr (M16) *gptr<uint16_t>(mx.ptr[2], first + k) = narrow1<false>(m[j]);
                else *gptr<float>(mx.ptr[2], first + k) = m[j];
                u[k] = x[j];
            }
            sum += (double)x[j] * (double)x[j];
        }
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
// Normalisation: X = u / (|u| + eps) into hi and lo, zeros in the padding.
//
// Bound by HBM: 8 bytes an element of an fp32 u, at 5.1 TB/s (302 M elements in 471 us on MI355X).  Tiles of 64 x 64 go
// through LDS, since a tall matrix is transposed on the way and a wide one shares the path; every workgroup adds the
// partial sums by itself, which costs one load a lane and saves a launch.
// ---------------------------------------------------------------------------

// x * 2^sx as hi + lo * 2^-11
__device__ __forceinline__ void split_pair(float x, _Float16& hi, _Float16& lo)
{
    hi = (_Float16)x;
    lo = (_Float16)((x - (float)hi) * kLoScale);
}

// 4 neighbouring elements, from an address aligned to their size
template <int IN>
__device__ __forceinline__ f32x4 load4(uint64_t base, uint64_t i)
{
    if constexpr (IN == kInF32) {
        return *reinterpret_cast<const GLOBAL f32x4*>(gptr<const float>(base, i));
    } else {
        const u32x2 w = *reinterpret_cast<const GLOBAL u32x2*>(gptr<const uint16_t>(base, i));
        const f32x2 a = widen2<IN == kInF16>(w.x), b = widen2<IN == kInF16>(w.y);
        return f32x4{a.x, a.y, b.x, b.y};
    }
}

// |u| + eps from the partial sums, by every workgroup alike; its barrier is the workgroup's.
__device__ __forceinline__ double norm_of(const DevMatrix& mx, const char* ws, float eps)
{
    static_assert(kMaxPartials == 256, "four waves add the partial sums");
    __shared__ double part[4];
    const uint32_t tid = threadIdx.x;
    double sum = tid < mx.n_partials ? *at<const double>(const_cast<char*>(ws), mx.partials + (uint64_t)tid * 8) : 0.0;
#pragma unroll
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
    if (tid % 64 == 0 && tid < 256) part[tid / 64] = sum;
    __syncthreads();
    sum = ((part[0] + part[1]) + part[2]) + part[3];
    return __builtin_sqrt(sum) + (double)eps;
}

// 2^sx / (|u| + eps)
__device__ __forceinline__ double norm_scale(const DevMatrix& mx, const char* ws, float eps, int sx)
{
    const double len = norm_of(mx, ws, eps);
    // a zero matrix without eps is zero
    return len == 0.0 ? 0.0 : __builtin_ldexp(1.0, sx) / len;
}

// A 64 x 64 tile of u as it lies in the matrix, from row r0 and column c0 on: 4 neighbours of row 16 k + tid / 16 in x[k]
// of a lane, zeros outside.
template <int IN>
__device__ __forceinline__ void load_tile(uint64_t in, bool by4, uint32_t rows, uint32_t cols, uint32_t r0, uint32_t c0,
                                          f32x4 (&x)[4])
{
    const uint32_t tid = threadIdx.x;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t r = r0 + (uint32_t)k * 16 + tid / 16, c = c0 + tid % 16 * 4;
        x[k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (r >= rows) continue;
        const uint64_t i = (uint64_t)r * cols + c;
        if (by4) {
            if (c < cols) x[k] = load4<IN>(in, i);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < cols) x[k][e] = load1<IN>(in, i + e);
        }
    }
}

// The tile's pairs to LDS, in rows of kTileLd elements (144 bytes: 16-byte reads stay aligned), or transposed.
constexpr int kTileLd = 72;
__device__ __forceinline__ void store_tile(const f32x4 (&x)[4], double scale, bool transposed, _Float16* hi, _Float16* lo)
{
    const uint32_t tid = threadIdx.x;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t r = (uint32_t)k * 16 + tid / 16, c = tid % 16 * 4;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t o = transposed ? (c + e) * kTileLd + r : r * kTileLd + c + e;
            split_pair((float)((double)x[k][e] * scale), hi[o], lo[o]);
        }
    }
}

// Rows start at a multiple of 4 elements
__device__ __forceinline__ bool rows_by4(uint32_t cols, uint64_t in) { return cols % 4 == 0 && in % 16 == 0; }

template <int IN>
__global__ __launch_bounds__(256) void ns_normalise_kernel(const DevMatrix* __restrict__ mats,
                                                           const DevTile* __restrict__ tiles, char* ws, float eps,
                                                           int sx, int step)
{
    if (step && reinterpret_cast<const NsScalars*>(ws)->skip) return;
    const DevTile t = tiles[blockIdx.x];
    const DevMatrix& mx = mats[t.mat];
    const bool tall = mx.tall != 0;
    const uint32_t cols = (uint32_t)mx.cols;
    const uint64_t in = step ? (uint64_t)(uintptr_t)ws + t.parts.u() : mx.ptr[1];
    f32x4 x[4];
    load_tile<IN>(in, rows_by4(cols, in), (uint32_t)mx.rows, cols, (tall ? t.col : t.row) * kPad, (tall ? t.row : t.col) * kPad, x);
    const double scale = norm_scale(mx, ws, eps, sx);
    __shared__ alignas(16) _Float16 hi[kPad * kTileLd];
    __shared__ alignas(16) _Float16 lo[kPad * kTileLd];
    store_tile(x, scale, tall, hi, lo);
    __syncthreads();
    for (uint32_t k = threadIdx.x; k < kPad * 8; k += 256) {
        const uint32_t r = k / 8, c = k % 8 * 8;
        const uint64_t o = (uint64_t)(t.row * kPad + r) * (uint64_t)t.parts.lp + t.col * kPad + c;
        *reinterpret_cast<GLOBAL f16x8*>(at<_Float16>(ws, t.parts.hi(0)) + o) = *reinterpret_cast<const f16x8*>(hi + r * kTileLd + c);
        *reinterpret_cast<GLOBAL f16x8*>(at<_Float16>(ws, t.parts.lo()) + o) = *reinterpret_cast<const f16x8*>(lo + r * kTileLd + c);
    }
}

// ---------------------------------------------------------------------------
// Products: A = X X^T, B = b A + c A A and X' = a X + B X, tile by tile.
//
// A tile's two factors come in runs of 64 summed elements straight to LDS, in two stages (four of the small tiles) that
// turn about: while the matrix instructions of one run go on, the next one is under way, and one wait and one
// barrier stand between two runs.  Sums stay in registers; the epilogue takes them through LDS, 32 rows of a wave
// at a time, so that global memory sees 16-byte words of rows (of columns where a square is mirrored).
//
// 256 x 256 tiles on 8 waves read 1 byte for 128 operations, 128 x 128 and 64 x 64 half and a quarter as many
// operations, and are for launches that would leave CUs idle.  On MI355X, 24 matrices of 2048 x 2048 and 12 of
// 2048 x 8192 (tiles of 256): gram 733 us (949 TFLOP/s over the tiles on and below the diagonal), poly 409 us (851),
// apply 1,662 us (744), with a step's epilogue 2,028 us (610); a library product of 8192 x 8192 in fp16, which writes
// little and sums long, reaches 1,402.  What bounds them: the matrix instructions, at 2.0 to 2.2 GHz, take 44, 39, 33 and
// 26 % of the cycles; the largest part of the rest is each tile's epilogue, which no other workgroup of
// the CU covers (one fits): of apply 2 bytes an element read and 4 written, of the squares 2 written, of a mixed step 6 read
// and 6 written.  An earlier build without epilogues took 667 us for gram (of 735), 346 for poly (448), and 1,070 for
// either apply (1,770 and 1,844): two fifths of apply are its epilogue.
// Tiles of 64 in launches of 78 to 144 (768 x 768) are latencies, 7 to 11 us each.
// ---------------------------------------------------------------------------

enum NsOp { kGram, kGramLong, kPoly, kApply, kLast };

struct ProductArgs {
    float a, b, c;
    int sx, sa, sb;
    int parity;      // of the product step: which of the two buffers X is in
    int diagonal_lo; // B's diagonal takes part in the product with lo (NsScales::lo_steps)
    int step;        // a Muon step: its skip mark is looked at
    float lr, decay, lrwd;   // a step's last epilogue
    int32_t* count;          // the counter that the launch advances, or null
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

__device__ __forceinline__ f16x4 read_transposed(const char* p)
{
    return __builtin_bit_cast(f16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                         (__attribute__((address_space(3))) s16x4*)const_cast<char*>(p)));
}

// A workgroup's waves take 2 x wx parts of its tile.  `stages` runs of kPad summed elements of both
// factors are in LDS at once, all but one of them on their way.
template <int KIND>
struct TileShape {
    static constexpr int rows = kTileRows[KIND], cols = kTileCols[KIND], lanes = kTileLanes[KIND], waves = lanes / 64;
    static constexpr int wx = waves / 2, stages = KIND == 2 ? 4 : 2;
};

// Loads of one summing step of a factor into LDS that do not pass registers.  A wave's access fills 1 KiB in order;
// 16-byte words are exchanged by the addresses that the lanes read from.

// ROWS rows of 128 bytes.  Word w of row r lies in place w ^ (r / 2 % 8): the operand of a matrix
// instruction takes one word of 32 rows, 16 rows at a time ({0-3, 12-15, 20-23, 24-27} and the
// others), which with this exchange lie in 16 different words of 256 bytes, all the banks
// there are.  Rows past the factor read its last row again; what they give is not stored.
template <int ROWS, int WAVES>
struct RowStage {
    static constexpr int kLoads = ROWS / 8 / WAVES;
    const GLOBAL char* src[kLoads];

    __device__ __forceinline__ void init(const GLOBAL _Float16* p, uint32_t row0, uint32_t rows, uint32_t pitch, uint32_t wave,
                                         uint32_t lane)
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t r = (wave * kLoads + (uint32_t)i) * 8 + lane / 8;
            const uint32_t row = row0 + r < rows ? row0 + r : rows - 1;
            src[i] = reinterpret_cast<const GLOBAL char*>(p + (uint64_t)row * pitch) + ((lane ^ (r >> 1)) & 7u) * 16;
        }
    }
    __device__ __forceinline__ void load(char* buf, uint32_t k, uint32_t wave) const
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            load_to_lds(src[i] + (uint64_t)k * (kPad * 2), buf + (wave * kLoads + (uint32_t)i) * 1024);
    }
    // word 2 kk + lane / 32 of row lane % 32 of the 32 rows from `row` on
    static __device__ __forceinline__ f16x8 operand(const char* buf, uint32_t row, uint32_t kk, uint32_t lane)
    {
        const uint32_t r = row + (lane & 31u), w = (kk * 2 + (lane >> 5)) ^ ((r >> 1) & 7u);
        return *reinterpret_cast<const f16x8*>(buf + r * (kPad * 2) + w * 16);
    }
};

// 64 rows of COLS elements, whose columns are the operands.  A transposing read takes 4 rows by 32 columns
// (64 bytes) for each half wave; 64 bytes number c of row r lie in place c ^ (r % 4) (two
// rows to 256 bytes: c ^ (r / 2 % 2)), so that the four rows fall on all the banks.  Columns
// past the factor read its last ones again.
template <int COLS, int WAVES>
struct ColumnStage {
    static constexpr int kLoads = COLS / 8 / WAVES, kRowBytes = COLS * 2, kWords = COLS / 8;
    const GLOBAL char* src[kLoads];
    uint64_t step;

    static __device__ __forceinline__ uint32_t exchange(uint32_t row)
    {
        return (COLS == 64 ? row >> 1 & 1u : row & 3u) * 4;
    }
    __device__ __forceinline__ void init(const GLOBAL _Float16* p, uint32_t col0, uint32_t cols, uint32_t pitch, uint32_t wave,
                                         uint32_t lane)
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t w = (wave * kLoads + (uint32_t)i) * 64 + lane, r = w / kWords;
            const uint32_t c = col0 + ((w % kWords) ^ exchange(r)) * 8;
            src[i] = reinterpret_cast<const GLOBAL char*>(p + (uint64_t)r * pitch + (c < cols ? c : cols - 8));
        }
        step = (uint64_t)pitch * (kPad * 2);
    }
    __device__ __forceinline__ void load(char* buf, uint32_t k, uint32_t wave) const
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) load_to_lds(src[i] + k * step, buf + (wave * kLoads + (uint32_t)i) * 1024);
    }
    // rows 16 kk + lane / 32 * 8 .. + 7 of column lane % 32 of the 32 from `col` on: two reads of 4 rows each, for
    // which lane i of 16 gives the address of 4 columns of row i / 4 and gets column i
    static __device__ __forceinline__ f16x8 operand(const char* buf, uint32_t col, uint32_t kk, uint32_t lane)
    {
        const uint32_t r = kk * 16 + (lane >> 5) * 8 + (lane >> 2 & 3u), c = col + (lane & 16u) + (lane & 3u) * 4;
        const char* p = buf + r * kRowBytes + ((c / 8) ^ exchange(r)) * 16 + (c & 4u) * 2;
        const f16x4 a = read_transposed(p), b = read_transposed(p + 4 * kRowBytes);
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};

// Waits until at most N of the wave's loads are under way and its reads of LDS have arrived, then for the
// other waves.
template <int N>
__device__ __forceinline__ void wait_and_meet()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// 8 neighbouring floats
__device__ __forceinline__ void read8(const GLOBAL float* p, float (&x)[8])
{
    const GLOBAL f32x4* q = reinterpret_cast<const GLOBAL f32x4*>(p);
    const f32x4 a = q[0], b = q[1];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        x[k] = a[k];
        x[k + 4] = b[k];
    }
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

// The end of the list's work for element i of a matrix: what it reads, and what it writes given the result o.
struct EndScalar {
    uint32_t p, aux;   // as stored
};

template <int END>
__device__ __forceinline__ EndScalar end_read(const DevMatrix& mx, uint64_t i)
{
    EndScalar in{};
    if constexpr (END == kEndSplit || END == kEndPure || END == kEndKahan || END == kEndKahan32)
        in.p = *gptr<const uint16_t>(mx.ptr[0], i);
    if constexpr (END == kEndMixedBf16 || END == kEndMixedF16 || END == kEndKahan32) in.aux = *gptr<const uint32_t>(mx.ptr[3], i);
    if constexpr (END == kEndSplit || END == kEndKahan) in.aux = *gptr<const uint16_t>(mx.ptr[3], i);
    return in;
}

template <int END>
__device__ __forceinline__ void end_write(const DevMatrix& mx, uint64_t i, const EndScalar& in, float o, float stepf,
                                          const ProductArgs& q)
{
    GLOBAL uint16_t* p = gptr<uint16_t>(mx.ptr[0], i);
    if constexpr (END == kEndOrtho) {
        *p = narrow1<false>(o);
    } else if constexpr (END == kEndMixedBf16 || END == kEndMixedF16) {
        const float x = __uint_as_float(in.aux) * q.decay - stepf * o;
        *gptr<float>(mx.ptr[3], i) = x;
        *p = narrow1<END == kEndMixedF16>(x);
    } else if constexpr (END == kEndSplit) {
        const float x = __uint_as_float(join_master(in.p, in.aux)) * q.decay - stepf * o;
        uint32_t r16;
        *p = (uint16_t)split_master(__float_as_uint(x), r16);
        *gptr<uint16_t>(mx.ptr[3], i) = (uint16_t)r16;
    } else {
        const float pf = widen1<false>((uint16_t)in.p);
        if constexpr (END == kEndPure) {
            *p = narrow1<false>(pf * q.decay - stepf * o);
        } else {
            const float cf = END == kEndKahan ? widen1<false>((uint16_t)in.aux) : __uint_as_float(in.aux);
            const float s = cf + (-(q.lrwd * pf) - stepf * o);
            const uint16_t pn = narrow1<false>(pf + s);
            const float rest = s - (widen1<false>(pn) - pf);
            *p = pn;
            if constexpr (END == kEndKahan) *gptr<uint16_t>(mx.ptr[3], i) = narrow1<false>(rest);
            else *gptr<float>(mx.ptr[3], i) = rest;
        }
    }
}

// What the end reads of 8 neighbouring elements: master; param and remainder; param and compensation.
template <int END>
struct EndInput {
    u32x4 p, aux0, aux1;
};

template <int END>
__device__ __forceinline__ EndInput<END> end_input(const DevMatrix& mx, uint64_t i)
{
    constexpr bool kParam = END == kEndSplit || END == kEndPure || END == kEndKahan || END == kEndKahan32;
    constexpr bool kAux32 = END == kEndMixedBf16 || END == kEndMixedF16 || END == kEndKahan32;
    EndInput<END> in{};
    if constexpr (kParam) in.p = *reinterpret_cast<const GLOBAL u32x4*>(gptr<const uint16_t>(mx.ptr[0], i));
    if constexpr (kAux32) {
        const GLOBAL u32x4* w = reinterpret_cast<const GLOBAL u32x4*>(gptr<const float>(mx.ptr[3], i));
        in.aux0 = w[0];
        in.aux1 = w[1];
    } else if constexpr (END == kEndSplit || END == kEndKahan) {
        in.aux0 = *reinterpret_cast<const GLOBAL u32x4*>(gptr<const uint16_t>(mx.ptr[3], i));
    }
    return in;
}

// 8 values of two words of four fp32, or of one of eight bf16
__device__ __forceinline__ void as_floats(const u32x4& a, const u32x4& b, float (&x)[8])
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[e] = __uint_as_float(a[e]);
        x[e + 4] = __uint_as_float(b[e]);
    }
}
__device__ __forceinline__ void as_floats(const u32x4& a, float (&x)[8])
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const f32x2 v = widen2<false>(a[e]);
        x[2 * e] = v.x;
        x[2 * e + 1] = v.y;
    }
}

template <int END>
__device__ __forceinline__ void end_eight(const DevMatrix& mx, uint64_t i, const EndInput<END>& in, const float (&o)[8],
                                          float stepf, const ProductArgs& q)
{
    GLOBAL u32x4* p16 = reinterpret_cast<GLOBAL u32x4*>(gptr<uint16_t>(mx.ptr[0], i));
    float x[8];
    if constexpr (END == kEndOrtho) {
        *p16 = pack8<false>(o);
    } else if constexpr (END == kEndMixedBf16 || END == kEndMixedF16) {
        as_floats(in.aux0, in.aux1, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * q.decay - stepf * o[e];
        store8_f32(gptr<float>(mx.ptr[3], i), x);
        *p16 = pack8<END == kEndMixedF16>(x);
    } else if constexpr (END == kEndSplit) {
        u32x4 pn, rn;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t r0, r1;
            const float a = __uint_as_float(join_master(in.p[e] & 0xffffu, in.aux0[e] & 0xffffu)) * q.decay - stepf * o[2 * e];
            const float b = __uint_as_float(join_master(in.p[e] >> 16, in.aux0[e] >> 16)) * q.decay - stepf * o[2 * e + 1];
            const uint32_t h0 = split_master(__float_as_uint(a), r0), h1 = split_master(__float_as_uint(b), r1);
            pn[e] = h0 | h1 << 16;
            rn[e] = r0 | r1 << 16;
        }
        *p16 = pn;
        *reinterpret_cast<GLOBAL u32x4*>(gptr<uint16_t>(mx.ptr[3], i)) = rn;
    } else {
        as_floats(in.p, x);
        if constexpr (END == kEndPure) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = x[e] * q.decay - stepf * o[e];
            *p16 = pack8<false>(x);
        } else {
            float c[8], s[8], sum[8];
            if constexpr (END == kEndKahan) as_floats(in.aux0, c);
            else as_floats(in.aux0, in.aux1, c);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[e] = c[e] + (-(q.lrwd * x[e]) - stepf * o[e]);
                sum[e] = x[e] + s[e];
            }
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
__global__ __launch_bounds__(kTileLanes[KIND], 2) void ns_product_kernel(const DevMatrix* __restrict__ mats,
                                                                        const DevTile* __restrict__ tiles, char* ws,
                                                                        ProductArgs q)
{
    using S = TileShape<KIND>;
    constexpr bool kGramOp = OP == kGram || OP == kGramLong, kSquare = kGramOp || OP == kPoly;
    using StageP = RowStage<S::rows, S::waves>;
    using StageQ = std::conditional_t<kSquare, RowStage<S::cols, S::waves>, ColumnStage<S::cols, S::waves>>;
    constexpr int WR = S::rows / 2, WC = S::cols / S::wx;   // a wave's part of the tile
    constexpr int MI = WR / 32, NI = WC / 32;
    constexpr int kBytesP = S::rows * kPad * 2, kStageBytes = kBytesP + S::cols * kPad * 2;
    constexpr int kLoads = StageP::kLoads + StageQ::kLoads;   // of a wave, for one stage
    constexpr int kEpiLd = WC + 8;                      // floats: rows 4 apart fall on the other half of the banks
    constexpr int kEpiBytes = 32 * kEpiLd * 4;          // one wave's 32 rows on their way out
    static_assert(S::waves * kEpiBytes <= S::stages * kStageBytes, "the epilogue takes the place of the operands");
    __shared__ alignas(16) char lds[S::stages * kStageBytes];
    if (q.step && reinterpret_cast<const NsScalars*>(ws)->skip) return;

    const DevTile tile = tiles[blockIdx.x];
    const NsParts& parts = tile.parts;
    const uint32_t tid = threadIdx.x, lane = tid & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t sp = parts.sp, lp = parts.lp;
    const uint32_t r0 = tile.row * S::rows, c0 = tile.col * S::cols;
    const GLOBAL _Float16* x_now = at<const _Float16>(ws, parts.hi(q.parity));

    StageP stage_p;
    StageQ stage_q;
    if constexpr (kGramOp) {
        stage_p.init(x_now, r0, sp, lp, wave, lane);
        stage_q.init(x_now, c0, sp, lp, wave, lane);
    } else if constexpr (OP == kPoly) {
        stage_p.init(at<const _Float16>(ws, parts.a()), r0, sp, sp, wave, lane);
        stage_q.init(at<const _Float16>(ws, parts.a()), c0, sp, sp, wave, lane);
    } else {
        stage_p.init(at<const _Float16>(ws, parts.b()), r0, sp, sp, wave, lane);
        stage_q.init(x_now, c0, lp, lp, wave, lane);
    }
    const auto load = [&](uint32_t k, uint32_t buf) {
        stage_p.load(lds + buf * kStageBytes, k, wave);
        stage_q.load(lds + buf * kStageBytes + kBytesP, k, wave);
    };
    const uint32_t wr = wave / S::wx * WR, wc = wave % S::wx * WC;   // the wave's place in the tile

    // What the epilogue reads.  A wait for a load waits for every store before it too, so each round's is asked for
    // one round ahead, the first round's of the small tiles, which have registers to spare, before the
    // summing; and inside the matrix wherever the lane lies, so that all are under way together.
    constexpr int kRowPacks = WC / 8, kPacks = 32 * kRowPacks / 64;
    const uint32_t lim_c = kSquare ? sp : lp, col0 = c0 + wc;
    struct Input {
        f16x8 x[kPacks];    // A, or lo
        float dr[kPacks];   // the diagonal of A or B at the rows
    };
    const auto read_ahead = [&](int i, Input& in) {
        if constexpr (OP == kPoly || !kSquare) {
#pragma unroll
            for (int h = 0; h < kPacks; ++h) {
                const uint32_t k = (uint32_t)h * 64 + lane;
                uint32_t r = r0 + wr + (uint32_t)i * 32 + k / kRowPacks, c = col0 + k % kRowPacks * 8;
                r = r < sp ? r : sp - 1;
                c = c < lim_c ? c : lim_c - 8;
                in.dr[h] = at<const float>(ws, OP == kPoly ? parts.da() : parts.db())[r];
                in.x[h] = *reinterpret_cast<const GLOBAL f16x8*>(at<const _Float16>(ws, OP == kPoly ? parts.a() : parts.lo()) +
                                                                 (uint64_t)r * lim_c + c);
            }
        }
    };
    float dc[8];   // the diagonal of A at the columns, the same in every round
    if constexpr (OP == kPoly) {
        const uint32_t c = col0 + lane % kRowPacks * 8;
        read8(at<const float>(ws, parts.da()) + (c < sp ? c : sp - 8), dc);
    }
    Input in[2];
    if constexpr (KIND != 0 && OP != kLast) read_ahead(0, in[0]);
    // the matrix as the caller has it, for the last product
    const DevMatrix& mx = mats[OP == kLast ? tile.mat : 0];
    const bool tall = OP == kLast && mx.tall != 0, row16 = OP == kLast && mx.row16 != 0;
    const uint32_t rows = OP == kLast ? (uint32_t)mx.rows : 0, cols = OP == kLast ? (uint32_t)mx.cols : 0;
    const float stepf = OP == kLast ? (float)((double)q.lr * mx.factor) : 0.0f;
    // The place in the matrix of pack k of round row0: of a tall one, 8 of a column of X.
    const auto place = [&](uint32_t row0, uint32_t k, uint32_t& r, uint32_t& c) {
        r = tall ? col0 + k / 4 : row0 + k / kRowPacks;
        c = tall ? row0 + k % 4 * 8 : col0 + k % kRowPacks * 8;
    };
    if constexpr (OP == kLast)
        if (q.count && blockIdx.x == 0 && tid == 0) *q.count += 1;   // the step is taken

    f32x16 acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

    const uint32_t nk = (kGramOp ? lp : sp) / kPad;
    struct Operands {
        f16x8 a[MI], b[NI];
    };
    const auto read = [&](uint32_t buf, int kk, Operands& o) __attribute__((always_inline)) {
        const char* bp = lds + buf * kStageBytes;
#pragma unroll
        for (int i = 0; i < MI; ++i) o.a[i] = StageP::operand(bp, wr + i * 32, kk, lane);
#pragma unroll
        for (int j = 0; j < NI; ++j) o.b[j] = StageQ::operand(bp + kBytesP, wc + j * 32, kk, lane);
    };
    // acc += (a + B_rr - fp16(B_rr)) X, for the 16 rows of X in `o` if they are the wave's; acc is under 2^(sb + sx)
    const auto linear = [&](const Operands& o, uint32_t k, int kk) __attribute__((always_inline)) {
        const uint32_t first = r0 + wr;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            if ((k * kPad + (uint32_t)kk * 16) / 32 != first / 32 + i) continue;
            const uint32_t r = k * kPad + (uint32_t)kk * 16 + (lane >> 5) * 4;
            const GLOBAL float* db = at<const float>(ws, parts.db()) + r;
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = db[e < 4 ? e : e + 4];
                f[e] = q.a * pow2(q.sb) + (d - (float)(_Float16)d);
            }
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                // a lane has 8 rows of its column; of 16 the results want rows 0-3 and 8-11 in the lower half wave, 4-7 and
                // 12-15 in the upper
                const u32x4 x = __builtin_bit_cast(u32x4, o.b[j]);
                const auto s0 = __builtin_amdgcn_permlane32_swap(x[0], x[2], false, false);
                const auto s1 = __builtin_amdgcn_permlane32_swap(x[1], x[3], false, false);
                const u32x4 y = {s0[0], s1[0], s0[1], s1[1]};
                const f16x8 v = __builtin_bit_cast(f16x8, y);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int c = (kk & 1) * 8 + e;
                    acc[i][j][c] = __builtin_fmaf(f[e], (float)v[e], acc[i][j][c]);
                }
            }
        }
    };

#pragma unroll
    for (uint32_t t = 0; t + 1 < S::stages; ++t)
        if (t < nk) load(t, t);
    // stage 0 has arrived: all but the loads behind it
    if (nk >= S::stages - 1) wait_and_meet<(S::stages - 2) * kLoads>();
    else wait_and_meet<0>();
    uint32_t buf = 0, fill = S::stages - 1;
    const auto multiply = [&](const Operands& o) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) acc[i][j] = mfma(o.a[i], o.b[j], acc[i][j]);
    };
    // Waits until the stage behind `buf` has arrived, and every wave has its last operands of this one, whose room is
    // loaded next.
    const auto next_stage = [&](uint32_t t) __attribute__((always_inline)) {
        if (S::stages > 2 && t + S::stages - 1 < nk) wait_and_meet<(S::stages - 2) * kLoads>();
        else wait_and_meet<0>();
        fill = buf;
        buf = buf + 1 == S::stages ? 0 : buf + 1;
    };
    // A long sum in two levels.  An fp32 sum of l / 16 like terms, as of equal columns, is off by l / 16 2^-25 of it at worst,
    // each element by its own share: 65 x 4 M of rank one came out 6.4e-3 off after five steps, 1.9e-3 this way, as 65 x 64 K is.
    f32x16 total[MI][NI];
    const bool in_two = OP == kGramLong && lp > kLongSum;
    if constexpr (OP == kGramLong) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) total[i][j] = acc[i][j];
    }
    const auto carry = [&](uint32_t done) __attribute__((always_inline)) {
        if constexpr (OP == kGramLong) {
            if (!in_two || done % kLongRun) return;
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        total[i][j][e] += acc[i][j][e];
                        acc[i][j][e] = 0.0f;
                    }
        }
    };
    using Yes = std::true_type;
    using No = std::false_type;
    uint32_t t = 0;
    if constexpr (KIND == 2) {
        // One matrix instruction a wave for each 16 summed elements: the reads of a whole stage lie between its
        // arrival and the instructions of the one before.
        Operands o[2][kPad / 16];
        const auto read_stage = [&](Operands(&to)[kPad / 16]) __attribute__((always_inline)) {
#pragma unroll
            for (int kk = 0; kk < kPad / 16; ++kk) read(buf, kk, to[kk]);
        };
        const auto summing_step = [&](uint32_t t, auto odd, auto last) __attribute__((always_inline)) {
            constexpr int now = decltype(odd)::value ? 1 : 0;
            if (t + S::stages - 1 < nk) load(t + S::stages - 1, fill);
            if constexpr (!decltype(last)::value) {
                next_stage(t);
                read_stage(o[now ^ 1]);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int kk = 0; kk < kPad / 16; ++kk) {
                multiply(o[now][kk]);
                if constexpr (!kSquare) linear(o[now][kk], t, kk);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        read_stage(o[0]);
        for (; t + 2 < nk; t += 2) {
            summing_step(t, No{}, No{});
            summing_step(t + 1, Yes{}, No{});
            carry(t + 2);
        }
        if (t + 1 < nk) {
            summing_step(t, No{}, No{});
            summing_step(t + 1, Yes{}, Yes{});
        } else {
            summing_step(t, No{}, Yes{});
        }
    } else {
        Operands o[2];
        read(0, 0, o[0]);
        // One summing step.  The next operands are asked for before the matrix instructions of the present ones; left to
        // itself the compiler moves the reads behind them and waits for each.
        const auto summing_step = [&](uint32_t t, auto with_linear, auto last) __attribute__((always_inline)) {
            if (S::stages == 2 ? !decltype(last)::value : t + S::stages - 1 < nk) load(t + S::stages - 1, fill);
#pragma unroll
            for (int kk = 0; kk < kPad / 16; ++kk) {
                if (kk + 1 < kPad / 16) {
                    read(buf, kk + 1, o[(kk + 1) & 1]);
                } else if (!decltype(last)::value) {
                    next_stage(t);
                    read(buf, 0, o[0]);   // covered by the matrix instructions below
                }
                __builtin_amdgcn_sched_barrier(0);
                multiply(o[kk & 1]);
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (decltype(with_linear)::value) linear(o[kk & 1], t, kk);
            }
        };
        if constexpr (!kSquare) {
            // the steps whose rows of X are the tile's own: apply meets there the elements that its linear term needs, in
            // the registers that hold them as an operand
            for (; t < r0 / kPad; ++t) summing_step(t, No{}, No{});
            for (; t < (r0 + S::rows) / kPad && t + 1 < nk; ++t) summing_step(t, Yes{}, No{});
        }
        for (; t + 1 < nk; ++t) {
            summing_step(t, No{}, No{});
            carry(t + 1);
        }
        summing_step(t, std::bool_constant<!kSquare>{}, Yes{});
    }
    if constexpr (OP == kGramLong) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] += total[i][j][e];
    }
    wait_and_meet<0>();   // the operands' room is free

    // Epilogue, 32 rows of the wave's part at a time through LDS of its own: 8 neighbours of a row to a
    // lane, and for what is needed by columns then 8 of a column.
    float* out = reinterpret_cast<float*>(lds + wave * kEpiBytes);
    if constexpr (KIND == 0 && OP != kLast) read_ahead(0, in[0]);
    // of lo in X': a, and where it takes part B's diagonal
    const float diagonal = q.diagonal_lo ? pow2(-q.sb) : 0.0f;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const uint32_t row0 = r0 + wr + (uint32_t)i * 32;
        // the last product's epilogue has no registers for a round ahead
        const Input& now = in[OP == kLast ? 0 : i & 1];
        if constexpr (OP == kLast) read_ahead(i, in[0]);
        else if (i + 1 < MI) read_ahead(i + 1, in[(i + 1) & 1]);
        const float scale = OP == kLast ? pow2(-q.sb - q.sx) : 1.0f;
        EndInput<END> end[kPacks];
        if constexpr (OP == kLast) {
            if (row16) {
#pragma unroll
                for (int h = 0; h < kPacks; ++h) {
                    // aligned rows are of a multiple of 8: the 8 elements lie inside
                    uint32_t r, c;
                    place(row0, (uint32_t)h * 64 + lane, r, c);
                    r = r < rows ? r : rows - 1;
                    c = c < cols ? c : cols - 8;
                    end[h] = end_input<END>(mx, (uint64_t)r * cols + c);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                out[((e & 3) + 8 * (e >> 2) + 4 * (lane >> 5)) * kEpiLd + j * 32 + (lane & 31u)] = acc[i][j][e] * scale;
        __builtin_amdgcn_wave_barrier();
        if constexpr (OP == kLast) {
            // lo's part, by rows of X as lo lies
#pragma unroll
            for (int h = 0; h < kPacks; ++h) {
                const uint32_t k = (uint32_t)h * 64 + lane;
                f32x4* cell = reinterpret_cast<f32x4*>(out + k / kRowPacks * kEpiLd + k % kRowPacks * 8);
                const float of_lo = __builtin_fmaf(now.dr[h], diagonal, q.a) * (1.0f / kLoScale) * pow2(-q.sx);
                f32x4 x = cell[0], y = cell[1];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = __builtin_fmaf(of_lo, (float)now.x[h][e], x[e]);
                    y[e] = __builtin_fmaf(of_lo, (float)now.x[h][e + 4], y[e]);
                }
                cell[0] = x;
                cell[1] = y;
            }
            __builtin_amdgcn_wave_barrier();
            if (row16) {
#pragma unroll
                for (int h = 0; h < kPacks; ++h) {
                    const uint32_t k = (uint32_t)h * 64 + lane;
                    uint32_t r, c;
                    place(row0, k, r, c);
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] = tall ? out[(k % 4 * 8 + e) * kEpiLd + k / 4] : out[k / kRowPacks * kEpiLd + k % kRowPacks * 8 + e];
                    if (r < rows && c < cols) end_eight<END>(mx, (uint64_t)r * cols + c, end[h], v, stepf, q);
                }
            } else {
                // element by element along the matrix's rows, kSome of a lane under way together
                constexpr uint32_t kSome = 8;
                for (uint32_t k0 = lane; k0 < 32 * WC; k0 += 64 * kSome) {
                    EndScalar some[kSome];
                    float v[kSome];
                    uint64_t at_rc[kSome];
                    bool inside[kSome];
#pragma unroll
                    for (uint32_t h = 0; h < kSome; ++h) {
                        const uint32_t k = k0 + h * 64, lr = tall ? k % 32 : k / WC, lc = tall ? k / 32 : k % WC;
                        const uint32_t r = tall ? col0 + lc : row0 + lr, c = tall ? row0 + lr : col0 + lc;
                        inside[h] = r < rows && c < cols;
                        at_rc[h] = inside[h] ? (uint64_t)r * cols + c : 0;
                        v[h] = out[lr * kEpiLd + lc];
                        some[h] = end_read<END>(mx, at_rc[h]);
                    }
#pragma unroll
                    for (uint32_t h = 0; h < kSome; ++h)
                        if (inside[h]) end_write<END>(mx, at_rc[h], some[h], v[h], stepf, q);
                }
            }
            __builtin_amdgcn_wave_barrier();
            continue;
        }
#pragma unroll
        for (int h = 0; h < kPacks; ++h) {
            const uint32_t k = (uint32_t)h * 64 + lane, lr = k / kRowPacks, lc = k % kRowPacks * 8;
            const uint32_t r = row0 + lr, c = col0 + lc;
            float* cell = out + lr * kEpiLd + lc;
            const uint64_t at_rc = (uint64_t)r * lim_c + c;
            const bool inside = r < sp && c < lim_c;
            float v[8];
            {
                const f32x4 x = *reinterpret_cast<const f32x4*>(cell), y = *reinterpret_cast<const f32x4*>(cell + 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] = x[e];
                    v[e + 4] = y[e];
                }
            }
            if constexpr (kSquare) {
                if constexpr (kGramOp) {
                    const float f = pow2(q.sa - 2 * q.sx);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= f;
                } else {
                    // b A + c A A, with A's diagonal in fp32: (A + E)(A + E) = A A + (e_r + e_c) A + E E; all under 2^sb
                    const float f = pow2(-q.sa), g = pow2(q.sb), er = (now.dr[h] - (float)(_Float16)now.dr[h]) * f;
                    const float c2 = q.c * f * f * g, c1 = q.b * f * g, ce = q.c * f * g;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float ec = (dc[e] - (float)(_Float16)dc[e]) * f;
                        v[e] = __builtin_fmaf(c2, v[e], __builtin_fmaf(ce, er + ec, c1) * (float)now.x[h][e]);
                        if (r == c + e) v[e] += (q.b * er + q.c * er * er) * g;
                    }
                }
                if (inside) {
                    store_diagonal(at<float>(ws, kGramOp ? parts.da() : parts.db()), r, c, v);
                    f16x8 w;
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = (_Float16)v[e];
                    *reinterpret_cast<GLOBAL f16x8*>(at<_Float16>(ws, kGramOp ? parts.a() : parts.b()) + at_rc) = w;
                }
                *reinterpret_cast<f32x4*>(cell) = f32x4{v[0], v[1], v[2], v[3]};
                *reinterpret_cast<f32x4*>(cell + 4) = f32x4{v[4], v[5], v[6], v[7]};
            } else {
                // X' * 2^sx
                const float f = pow2(-q.sb), of_lo = __builtin_fmaf(now.dr[h], diagonal, q.a) * (1.0f / kLoScale);
                f16x8 h8, l8;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    _Float16 x, y;
                    split_pair(__builtin_fmaf(of_lo, (float)now.x[h][e], v[e] * f), x, y);
                    h8[e] = x;
                    l8[e] = y;
                }
                if (inside) {
                    *reinterpret_cast<GLOBAL f16x8*>(at<_Float16>(ws, parts.hi(q.parity ^ 1)) + at_rc) = h8;
                    *reinterpret_cast<GLOBAL f16x8*>(at<_Float16>(ws, parts.lo()) + at_rc) = l8;
                }
            }
        }
        __builtin_amdgcn_wave_barrier();
        if constexpr (kSquare) {
            if (tile_mirrored(KIND, tile.row, tile.col)) {
                // by columns: 8 of a column to a lane, 4 lanes to a column of the 32 rows
#pragma unroll
                for (int h = 0; h < kPacks; ++h) {
                    const uint32_t k = (uint32_t)h * 64 + lane, lc = k / 4, lr = k % 4 * 8;
                    const uint32_t r = row0 + lr, c = col0 + lc;
                    f16x8 w;
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = (_Float16)out[(lr + e) * kEpiLd + lc];
                    if (r < sp && c < sp)
                        *reinterpret_cast<GLOBAL f16x8*>(at<_Float16>(ws, kGramOp ? parts.a() : parts.b()) + (uint64_t)c * sp + r) = w;
                }
            }
            __builtin_amdgcn_wave_barrier();
        }
    }
}

// ---------------------------------------------------------------------------
// Matrices whose shorter side is at most 64: everything between the two passes over u in one workgroup, in binary64.
//
// With A = X X^T and p(A) = a I + b A + c A A, a step is X <- p(A) X and A <- p(A) A p(A), all polynomials of the first
// A, so Q = p_k(A_k) ... p_1(A_1) is found from 64 x 64 matrices alone and the result is Q X = (Q / (|u| + eps)) u:
// 4 steps - 3 products of at most 64 x 64 that never leave LDS instead of three launches a step.
//
// Where X has no singular value nothing in those polynomials brings a rounding of A back, which step-by-step products with
// X do: it grows by a^2 a step.  With A, Q and X as fp16 pairs (22 bits) a 64 x 2048 matrix of one direction and 0.3 % of noise
// came out 5e-2 off after seven steps, where the definition in fp32 is 3e-5 off.  So all of it is binary64, on its
// matrix instructions: the 2^-53 of a run of steps (NsScales::run) grows to 2^-31 at most, the result is rounded once, to
// fp32, and X is fp32 between runs.
//
// On MI355X, five steps, in us: one 16 x 768 moments 2.5, small gram 4.8, small chain 10, small apply 4.5; one
// 64 x 768 4.5, 8.4, 35 and 7.5; 64 x 1,048,576 67, 199, 125 and 245.  Short ones are latencies but for
// chain, which the matrix instructions bound where s is over 32: a 16 x 16 x 4 product takes a SIMD 64 cycles, so the
// 17 products of ten blocks take 18 us on one CU at least, and 22 with three blocks on two of its SIMDs.  As fp16 pairs chain took
// 18.6 us whatever s was, and a pass of either matrix 31, which take 20 and 55 now.
// ---------------------------------------------------------------------------

// Place of element (i, j), j <= i, of a lower triangle.
__device__ __forceinline__ uint32_t tri_at(uint32_t i, uint32_t j) { return i * (i + 1) / 2 + j; }

// The kernels that use it are compiled for two waves a SIMD or more, so that sums lie in VGPRs: in AGPRs, which the compiler
// takes where it may use 512 registers, a wave's instructions took 140 cycles each instead of 64 (MI355X).
__device__ __forceinline__ f64x4 mfma64(double a, double b, f64x4 c)
{
    return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0);
}
// Row of result e of a 16 x 16 product in binary64; the column is lane % 16.
__device__ __forceinline__ uint32_t result_row64(int e, uint32_t lane) { return (uint32_t)e * 4 + (lane >> 4); }

// A tile of u to LDS as fp32, in rows of kXLd elements, or transposed.  17 words of 16 bytes a row: the operands of a
// product in binary64, 4 neighbours of each of 16 rows, lie in all 64 banks.
constexpr int kXLd = 68;
__device__ __forceinline__ void store_tile_f32(const f32x4 (&x)[4], bool transposed, float* to)
{
    const uint32_t tid = threadIdx.x;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t r = (uint32_t)k * 16 + tid / 16, c = tid % 16 * 4;
        if (transposed) {
#pragma unroll
            for (int e = 0; e < 4; ++e) to[(c + e) * kXLd + r] = x[k][e];
        } else {
            *reinterpret_cast<f32x4*>(to + r * kXLd + c) = x[k];
        }
    }
}

// A run of columns' part of U U^T, in binary64: products of two fp32 are exact there, and the sum's rounding, 2^-53 of it
// a term at most, is nothing beside what the inputs are known to however long the run is.  Sums in fp32 are not good
// enough: like terms, as of a matrix of rank one with equal columns, are all rounded the same way (9e-5 of the sum of 4 M of
// them), and the steps multiply what is wrong by a^2 each where X has no singular value.  Each wave takes 16 of
// 64 columns and all 16 x 16 blocks on and below the diagonal that the matrix has rows for, so that a row block's operand is
// read once; the next 64 columns are under way while the last ones are multiplied.
template <int IN>
__global__ __launch_bounds__(256, 2) void ns_small_gram_kernel(const DevMatrix* __restrict__ mats,
                                                            const DevTile* __restrict__ tiles, char* ws, int step, int again)
{
    if (step && reinterpret_cast<const NsScalars*>(ws)->skip) return;
    const DevTile t = tiles[blockIdx.x];
    const DevMatrix& mx = mats[t.mat];
    const bool tall = mx.tall != 0;
    const uint32_t rows = (uint32_t)mx.rows, cols = (uint32_t)mx.cols, l = tall ? rows : cols, s = tall ? cols : rows;
    const uint64_t in = step || again ? (uint64_t)(uintptr_t)ws + t.parts.u() : mx.ptr[1];
    const bool by4 = rows_by4(cols, in);
    const uint32_t run = (uint32_t)small_gram_cols(t.parts.lp), j0 = t.col * run, j1 = j0 + run < l ? j0 + run : l;
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6, blocks = (s + 15) / 16;
    constexpr int kBlocks = kPad / 16;
    __shared__ alignas(16) float x[kPad * kXLd];
    __shared__ double join[2][kBlocks * (kBlocks + 1) / 2 * 256];
    f32x4 v[4];
    load_tile<IN>(in, by4, rows, cols, tall ? j0 : 0, tall ? 0 : j0, v);
    f64x4 acc[kBlocks][kBlocks];
#pragma unroll
    for (int i = 0; i < kBlocks; ++i)
#pragma unroll
        for (int j = 0; j <= i; ++j) acc[i][j] = f64x4{0.0, 0.0, 0.0, 0.0};
    for (uint32_t j = j0; j < j1; j += kPad) {
        store_tile_f32(v, tall, x);
        __syncthreads();
        if (j + kPad < j1) load_tile<IN>(in, by4, rows, cols, tall ? j + kPad : 0, tall ? 0 : j + kPad, v);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            const uint32_t c = wave * 16 + (uint32_t)kk * 4 + (lane >> 4);
            double o[kBlocks];
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) {
                if ((uint32_t)i >= blocks) break;
                o[i] = (double)x[((uint32_t)i * 16 + (lane & 15u)) * kXLd + c];
#pragma unroll
                for (int k = 0; k <= i; ++k) acc[i][k] = mfma64(o[i], o[k], acc[i][k]);
            }
        }
        __syncthreads();
    }
    // The waves' parts: the third and fourth's to the first and second, theirs to the first.
    const auto each = [&](auto&& f) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
            if ((uint32_t)i >= blocks) break;
#pragma unroll
            for (int j = 0; j <= i; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = f((double)acc[i][j][e], (uint32_t)((i * (i + 1) / 2 + j) * 256 + e * 64) + lane);
        }
    };
    for (uint32_t half = 2; half; half /= 2) {
        if (wave >= half && wave < 2 * half) each([&](double v, uint32_t k) { return join[wave - half][k] = v; });
        __syncthreads();
        if (wave < half) each([&](double v, uint32_t k) { return v + join[wave][k]; });
        __syncthreads();
    }
    if (wave) return;
    GLOBAL double* out = at<double>(ws, t.parts.base) + (uint64_t)t.col * kSmallTri;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
        if ((uint32_t)i >= blocks) break;
#pragma unroll
        for (int j = 0; j <= i; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t r = (uint32_t)i * 16 + result_row64(e, lane), c = (uint32_t)j * 16 + (lane & 15u);
                if (c <= r) out[tri_at(r, c)] = acc[i][j][e];
            }
    }
}

struct ChainArgs {
    float a, b, c, eps;
    int steps, step, again;
};

// A wave has one of the ten 16 x 16 blocks on and below the diagonal, of which a matrix of s rows needs those of its
// first ceil(s / 16) block rows.  All that is held is symmetric, and has to stay so to the last bit: an antisymmetric part,
// which exact products of commuting matrices have not, grows by a^2 with every step.  So the results on and below the
// diagonal count, and are stored twice.  Rows of 66 elements: the operands of a product, 4 neighbours of each of
// 16 rows, lie in all 64 banks twice.
constexpr int kBlockChain = 640;
constexpr int kChainLd = kPad + 2;

__global__ __launch_bounds__(kBlockChain) void ns_small_chain_kernel(const DevMatrix* __restrict__ mats,
                                                                       const DevTile* __restrict__ tiles, char* ws, ChainArgs g)
{
    if (g.step && reinterpret_cast<const NsScalars*>(ws)->skip) return;
    const DevTile t = tiles[blockIdx.x];
    const DevMatrix& mx = mats[t.mat];
    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t bi = wave < 1 ? 0 : wave < 3 ? 1 : wave < 6 ? 2 : 3, bj = wave - bi * (bi + 1) / 2;
    const uint32_t blocks = ((uint32_t)(mx.tall ? mx.cols : mx.rows) + 15) / 16;
    const bool active = bi < blocks;
    const uint32_t row = bi * 16 + result_row64(0, lane), col = bj * 16 + (lane & 15u);   // of result e: row + 4 e
    const uint32_t runs = (uint32_t)((t.parts.lp + small_gram_cols(t.parts.lp) - 1) / small_gram_cols(t.parts.lp));
    __shared__ double ta[kPad * kChainLd], tp[kPad * kChainLd], tq[kPad * kChainLd], tz[kPad * kChainLd];
    // NaN for a norm that is inf or NaN, so that every element of the result is; a zero matrix without eps is zero
    const double len = g.again ? 1.0 : norm_of(mx, ws, g.eps);
    const double inv = !(len < __builtin_inf()) ? __builtin_nan("") : len == 0.0 ? 0.0 : 1.0 / len;
    GLOBAL double* at_base = at<double>(ws, t.parts.base);
    f64x4 a = {0.0, 0.0, 0.0, 0.0}, p = a, q = a;
    if (active) {
#pragma unroll 8
        for (uint32_t k = 0; k < runs; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t r = row + (uint32_t)e * 4;
                a[e] += at_base[(uint64_t)k * kSmallTri + (r >= col ? tri_at(r, col) : tri_at(col, r))];
            }
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = a[e] * inv * inv;
    }
    const auto store = [&](const f64x4& v, double* to) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t r = row + (uint32_t)e * 4;
            if (active && r >= col) to[r * kChainLd + col] = to[col * kChainLd + r] = v[e];
        }
    };
    const auto product = [&](const double* x, const double* y) __attribute__((always_inline)) {
        f64x4 sum = {0.0, 0.0, 0.0, 0.0};
        if (!active) return sum;
        const double* px = x + (bi * 16 + (lane & 15u)) * kChainLd + (lane >> 4);
        const double* py = y + (bj * 16 + (lane & 15u)) * kChainLd + (lane >> 4);
        for (uint32_t k = 0; k < blocks * 16; k += 16)
#pragma unroll
            for (uint32_t kk = 0; kk < 16; kk += 4) sum = mfma64(px[k + kk], py[k + kk], sum);
        return sum;
    };
    for (int k = 0;; ++k) {
        store(a, ta);
        if (k) store(q, tq);
        __syncthreads();
        const f64x4 sq = product(ta, ta);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            p[e] = (double)g.c * sq[e] + (double)g.b * a[e];
            if (row + (uint32_t)e * 4 == col) p[e] += (double)g.a;
        }
        store(p, tp);
        __syncthreads();
        q = k ? product(tp, tq) : p;
        if (k + 1 == g.steps) break;
        store(product(tp, ta), tz);
        __syncthreads();
        a = product(tz, tp);
    }
    // Q / (|u| + eps) over the partial sums, which every wave has read
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t r = row + (uint32_t)e * 4;
        if (active && r >= col) at_base[tri_at(r, col)] = q[e] * inv;
    }
}

// The end of a run of steps that is not the last: X in fp32, as u lay.
constexpr int kEndAgain = kNumEnds;

// Q X, 64 columns at a time as small gram reads them, 16 to a wave; workgroups of 64 columns up to 4,096 and of 256
// beyond, where reading Q anew would cost as much as X.
template <int IN, int END>
__global__ __launch_bounds__(256, 2) void ns_small_apply_kernel(const DevMatrix* __restrict__ mats,
                                                             const DevTile* __restrict__ tiles, char* ws, int again,
                                                             ProductArgs g)
{
    if (g.step && reinterpret_cast<const NsScalars*>(ws)->skip) return;
    const uint32_t tid = threadIdx.x;
    if (g.count && blockIdx.x == 0 && tid == 0) *g.count += 1;   // the step is taken
    const DevTile t = tiles[blockIdx.x];
    const DevMatrix& mx = mats[t.mat];
    const bool tall = mx.tall != 0, row16 = mx.row16 != 0;
    const uint32_t rows = (uint32_t)mx.rows, cols = (uint32_t)mx.cols, l = tall ? rows : cols, s = tall ? cols : rows;
    const uint64_t in = g.step || again ? (uint64_t)(uintptr_t)ws + t.parts.u() : mx.ptr[1];
    const bool by4 = rows_by4(cols, in);
    const uint32_t run = (uint32_t)small_apply_cols(t.parts.lp), j0 = t.col * run, j1 = j0 + run < l ? j0 + run : l;
    const uint32_t lane = tid & 63u, wave = tid >> 6, blocks = (s + 15) / 16;
    const float stepf = (float)((double)g.lr * mx.factor);
    constexpr uint32_t kBlocks = kPad / 16;
    __shared__ double q[kPad * kChainLd];
    __shared__ alignas(16) float x[kPad * kXLd];
    constexpr int kOutLd = kPad + 4;
    __shared__ alignas(16) float out[kPad * kOutLd];   // as the matrix lies: rows of the caller's
    f32x4 v[4];
    load_tile<IN>(in, by4, rows, cols, tall ? j0 : 0, tall ? 0 : j0, v);
    {
        // Q, all of a lane's loads under way together
        const GLOBAL double* from = at<const double>(ws, t.parts.base);
        const uint32_t c = lane, n = blocks * 16;
        double w[kPad / 4];
#pragma unroll
        for (uint32_t i = 0; i < kPad / 4; ++i) {
            const uint32_t r = i * 4 + wave;
            w[i] = r < n && c < n ? from[r >= c ? tri_at(r, c) : tri_at(c, r)] : 0.0;
        }
#pragma unroll
        for (uint32_t i = 0; i < kPad / 4; ++i) q[(i * 4 + wave) * kChainLd + c] = w[i];
    }
    for (uint32_t j = j0; j < j1; j += kPad) {
        store_tile_f32(v, tall, x);
        __syncthreads();
        if (j + kPad < j1) load_tile<IN>(in, by4, rows, cols, tall ? j + kPad : 0, tall ? 0 : j + kPad, v);
        f64x4 acc[kBlocks];
#pragma unroll
        for (uint32_t i = 0; i < kBlocks; ++i) acc[i] = f64x4{0.0, 0.0, 0.0, 0.0};
        const uint32_t c = wave * 16 + (lane & 15u);
        for (uint32_t k4 = 0; k4 < blocks * 16; k4 += 4) {
            const uint32_t k = k4 + (lane >> 4);
            const double o = (double)x[k * kXLd + c];
#pragma unroll
            for (uint32_t i = 0; i < kBlocks; ++i) {
                if (i >= blocks) break;
                acc[i] = mfma64(q[(i * 16 + (lane & 15u)) * kChainLd + k], o, acc[i]);
            }
        }
#pragma unroll
        for (uint32_t i = 0; i < kBlocks; ++i) {
            if (i >= blocks) break;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t r = i * 16 + result_row64(e, lane);
                out[tall ? c * kOutLd + r : r * kOutLd + c] = (float)acc[i][e];
            }
        }
        __syncthreads();
        const uint32_t r0 = tall ? j : 0, c0 = tall ? 0 : j;
        if constexpr (END == kEndAgain) {
            // in u's place, of which this workgroup has read the tile and no other one reads any of its run
            GLOBAL float* to = at<float>(ws, t.parts.u());
#pragma unroll
            for (int h = 0; h < 16; ++h) {
                const uint32_t k = (uint32_t)h * 256 + tid, r = r0 + k / 64, c = c0 + k % 64;
                if (r < rows && c < cols) to[(uint64_t)r * cols + c] = out[k / 64 * kOutLd + k % 64];
            }
        } else if (row16) {
            EndInput<END> end[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t k = (uint32_t)h * 256 + tid, r = r0 + k / 8, c = c0 + k % 8 * 8;
                if (r < rows && c < cols) end[h] = end_input<END>(mx, (uint64_t)r * cols + c);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t k = (uint32_t)h * 256 + tid, r = r0 + k / 8, c = c0 + k % 8 * 8;
                const float* from = out + k / 8 * kOutLd + k % 8 * 8;
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = from[e];
                if (r < rows && c < cols) end_eight<END>(mx, (uint64_t)r * cols + c, end[h], o, stepf, g);
            }
        } else {
            EndScalar some[16];
#pragma unroll
            for (int h = 0; h < 16; ++h) {
                const uint32_t k = (uint32_t)h * 256 + tid, r = r0 + k / 64, c = c0 + k % 64;
                if (r < rows && c < cols) some[h] = end_read<END>(mx, (uint64_t)r * cols + c);
            }
#pragma unroll
            for (int h = 0; h < 16; ++h) {
                const uint32_t k = (uint32_t)h * 256 + tid, r = r0 + k / 64, c = c0 + k % 64;
                if (r < rows && c < cols)
                    end_write<END>(mx, (uint64_t)r * cols + c, some[h], out[k / 64 * kOutLd + k % 64], stepf, g);
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------

namespace {

template <int KIND, int OP, int END>
hipError_t launch_product(const NsCall& call, const NsLaunch& l, const ProductArgs& q, hipStream_t stream)
{
    ns_product_kernel<KIND, OP, END><<<(uint32_t)l.count, kTileLanes[KIND], 0, stream>>>(
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

// Tiles of 256 have no registers for a long sum's second level (planner).
hipError_t gram(const NsCall& call, const NsBatch& batch, const ProductArgs& q, hipStream_t stream)
{
    if (!batch.long_sums) return product<kGram>(call, batch.square, q, stream);
    return batch.square.kind == 1 ? launch_product<1, kGramLong, 0>(call, batch.square, q, stream)
                                  : launch_product<2, kGramLong, 0>(call, batch.square, q, stream);
}

template <int IN>
hipError_t moments(const NsCall& call, const NsLaunch& l, bool step, const MomentCoef& c, const StepRule& rule,
                   hipStream_t stream)
{
    const DevTile* tiles = call.tiles + l.first;
    const dim3 grid((uint32_t)l.count), block(kBlockMoments);
    if (!step) ns_moments_kernel<IN, false, false><<<grid, block, 0, stream>>>(call.mats, tiles, call.ws, c, rule);
    else if (call.kind.m16) ns_moments_kernel<IN, true, true><<<grid, block, 0, stream>>>(call.mats, tiles, call.ws, c, rule);
    else ns_moments_kernel<IN, true, false><<<grid, block, 0, stream>>>(call.mats, tiles, call.ws, c, rule);
    return hipGetLastError();
}

template <int IN>
hipError_t normalise(const NsCall& call, const NsLaunch& l, bool step, hipStream_t stream)
{
    ns_normalise_kernel<IN><<<(uint32_t)l.count, 256, 0, stream>>>(call.mats, call.tiles + l.first, call.ws, call.ns.eps,
                                                                   call.scales.sx, step);
    return hipGetLastError();
}

template <int IN, int END>
hipError_t launch_small_apply(const NsCall& call, const NsBatch& batch, bool again, const ProductArgs& q, hipStream_t stream)
{
    ns_small_apply_kernel<IN, END><<<(uint32_t)batch.apply.count, 256, 0, stream>>>(
        call.mats, call.tiles + batch.apply.first, call.ws, again, q);
    return hipGetLastError();
}

// `in`: the type of what is read, which is fp32 of a step and of X between two runs
template <int END>
hipError_t small_apply(const NsCall& call, const NsBatch& batch, int in, bool again, const ProductArgs& q, hipStream_t stream)
{
    if constexpr (END == kEndOrtho || END == kEndAgain) {
        if (in == kInBf16) return launch_small_apply<kInBf16, END>(call, batch, again, q, stream);
        if (in == kInF16) return launch_small_apply<kInF16, END>(call, batch, again, q, stream);
    }
    return launch_small_apply<kInF32, END>(call, batch, again, q, stream);
}

// Whatever depends on the end: the last product, or the small matrices' one.
template <int END>
hipError_t end_launch(const NsCall& call, const NsBatch& batch, int in, bool again, const ProductArgs& q, hipStream_t stream)
{
    return batch.small ? small_apply<END>(call, batch, in, again, q, stream)
                       : product<kLast, END>(call, batch.apply, q, stream);
}

template <int IN>
hipError_t small_gram(const NsCall& call, const NsLaunch& l, bool step, bool again, hipStream_t stream)
{
    ns_small_gram_kernel<IN><<<(uint32_t)l.count, 256, 0, stream>>>(call.mats, call.tiles + l.first, call.ws, step, again);
    return hipGetLastError();
}

StepRule step_rule(const NsCall& call)
{
    return StepRule{call.hp.inv_loss_scale, call.clip, call.step, call.found_inf, call.amp};
}

// `in`: the type of u, which a step has in fp32
hipError_t last_product(const NsCall& call, const NsBatch& batch, int in, bool again, const ProductArgs& q,
                        hipStream_t stream)
{
    switch (call.kind.end) {
    case kEndOrtho: return end_launch<kEndOrtho>(call, batch, in, again, q, stream);
    case kEndMixedBf16: return end_launch<kEndMixedBf16>(call, batch, in, again, q, stream);
    case kEndMixedF16: return end_launch<kEndMixedF16>(call, batch, in, again, q, stream);
    case kEndSplit: return end_launch<kEndSplit>(call, batch, in, again, q, stream);
    case kEndPure: return end_launch<kEndPure>(call, batch, in, again, q, stream);
    case kEndKahan: return end_launch<kEndKahan>(call, batch, in, again, q, stream);
    default: return end_launch<kEndKahan32>(call, batch, in, again, q, stream);
    }
}

}  // namespace

hipError_t launch_ns_count(const NsCall& call, hipStream_t stream)
{
    ns_count_kernel<<<1, 64, 0, stream>>>(step_rule(call), call.step);
    return hipGetLastError();
}

hipError_t launch_ns_batch(const NsCall& call, const NsBatch& batch, bool last, hipStream_t stream)
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
    const StepRule rule = step_rule(call);
    hipError_t e = in == kInF32 ? moments<kInF32>(call, batch.moments, step, mc, rule, stream)
                 : in == kInBf16 ? moments<kInBf16>(call, batch.moments, step, mc, rule, stream)
                                 : moments<kInF16>(call, batch.moments, step, mc, rule, stream);
    if (e != hipSuccess) return e;
    const int in_u = step ? kInF32 : in;
    if (batch.small) {
        const NsScales& s = call.scales;
        for (int left = call.ns.steps, from = in_u;; from = kInF32) {
            const bool again = left < call.ns.steps;
            e = from == kInF32 ? small_gram<kInF32>(call, batch.normalise, step, again, stream)
              : from == kInBf16 ? small_gram<kInBf16>(call, batch.normalise, step, again, stream)
                                : small_gram<kInF16>(call, batch.normalise, step, again, stream);
            if (e != hipSuccess) return e;
            const int run = left < s.run ? left : s.run;
            left -= run;
            ns_small_chain_kernel<<<(uint32_t)batch.square.count, kBlockChain, 0, stream>>>(
                call.mats, call.tiles + batch.square.first, call.ws,
                ChainArgs{call.ns.a, call.ns.b, call.ns.c, call.ns.eps, run, step, again});
            if ((e = hipGetLastError()) != hipSuccess) return e;
            if (left == 0) {
                q.count = last ? call.step : nullptr;
                return last_product(call, batch, from, again, q, stream);
            }
            e = small_apply<kEndAgain>(call, batch, from, again, q, stream);
            if (e != hipSuccess) return e;
        }
    }
    e = step || in == kInF32 ? normalise<kInF32>(call, batch.normalise, step, stream)
      : in == kInBf16 ? normalise<kInBf16>(call, batch.normalise, step, stream)
                      : normalise<kInF16>(call, batch.normalise, step, stream);
    if (e != hipSuccess) return e;
    for (int k = 0; k < call.ns.steps; ++k) {
        q.parity = k & 1;
        q.diagonal_lo = k + call.scales.lo_steps >= call.ns.steps;
        if ((e = gram(call, batch, q, stream)) != hipSuccess) return e;
        if ((e = product<kPoly>(call, batch.square, q, stream)) != hipSuccess) return e;
        if (k + 1 < call.ns.steps) {
            e = product<kApply>(call, batch.apply, q, stream);
        } else {
            q.count = last ? call.step : nullptr;
            e = last_product(call, batch, in_u, false, q, stream);
        }
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace adamw
