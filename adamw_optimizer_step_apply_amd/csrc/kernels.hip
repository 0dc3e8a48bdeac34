// kernels.hip -- gfx950 (CDNA4) kernels of the fused AdamW step.
//
// The step is a pure stream: every element is read once and written once, with
// no reuse, so there is nothing to stage in LDS and no contraction for the
// matrix cores.  The kernels are shaped for HBM: a lane moves a unit of a stream
// with one access (16 bytes, or 8 of a 16-bit stream beside fp32 ones), consecutive
// lanes touch consecutive units, and each lane issues all loads of its 8 elements
// (one or two units per stream) before it computes.  The math is fp32 in registers.
//
// Kernels:
//   prologue_kernel      one lane: reads the skip flag and the step counter,
//                        forms the step's scalars in binary64, advances the counter
//   update_kernel<MODE, FUSED> / update_pure_kernel<M32, V32, AUX, FUSED>
//                        eight workgroups per chunk, one on each XCD, the chunk
//                        interleaved between them in tiles of 256 or 512
//                        elements (a short chunk: one workgroup): the AdamW
//                        element update;
//                        FUSED: without a prologue, for small plans (each
//                        workgroup forms the scalars, the last one advances
//                        the counter)
//   zero_flag_kernel /
//   check_kernel<F16, FUSED>  the fp16-AMP overflow test (any inf/NaN gradient);
//                        FUSED: one launch that also sets the flag to 0 or 1
//   state_copy_kernel    layout only: state between per-tensor buffers and the
//                        blocked buffer
//   zero_words_kernel    clears the completion counters of a new workspace
//
// Element rule (the AdamW of Loshchilov & Hutter, Algorithm 2, with Adam's bias
// correction from Kingma & Ba, Algorithm 1; named on the pages "Distributed
// optimizer support for BERT", Usage, and "[pure bf16 training] w/
// AnyPrecisionAdamW and Kahan summation", the opt-1.3b command):
//   m = b1*m + (1-b1)*g ; v = b2*v + (1-b2)*(g*g) ; u = m / (sqrt(v*rbc2) + eps)
//   mixed: w = w*decay - step_size*u, p = round16(w)
//   Kahan: d = -(lrwd*p) - step_size*u ; s = c + d ; p' = rbf16(p + s) ; c = rbf16(s - (p' - p))
//          (with an fp32 compensation buffer c = s - (p' - p), unrounded)
// Each operation is one binary32 operation in that order; the library is
// compiled with -ffp-contract=off so no multiply-add is fused, sqrt and
// division are the correctly rounded ones, and fp32 subnormals are kept.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "adamw.h"
#include "device.hpp"
#include "layout.hpp"

namespace adamw {

// ---------------------------------------------------------------------------
// Element math
// ---------------------------------------------------------------------------

struct Coef {
    float step_size, rbc2, decay, lrwd, omb1, omb2, beta1, beta2, eps, inv_scale;
};

// Moments and the bias-corrected Adam direction u = m_hat / (sqrt(v_hat) + eps),
// with 1/(1-b1^t) carried by step_size.
__device__ __forceinline__ float adam_dir(float g, float& m, float& v, const Coef& c)
{
    m = c.beta1 * m + c.omb1 * g;
    v = c.beta2 * v + c.omb2 * (g * g);
    return m / (__builtin_sqrtf(v * c.rbc2) + c.eps);
}

// Mixed precision: fp32 master w (in place); returns the new w.
__device__ __forceinline__ float mixed_elem(float g16, float& w, float& m, float& v, const Coef& c)
{
    const float g = g16 * c.inv_scale;
    const float u = adam_dir(g, m, v, c);
    w = w * c.decay - c.step_size * u;
    return w;
}

// Kahan: returns the fp32 sum p + s to be rounded into the new bf16 p, and the
// pending increment s through `s_out`.
__device__ __forceinline__ float kahan_sum(float g16, float pf, float cf, float& m, float& v, const Coef& c,
                                           float& s_out)
{
    const float g = g16 * c.inv_scale;
    const float u = adam_dir(g, m, v, c);
    const float d = -(c.lrwd * pf) - c.step_size * u;
    const float s = cf + d;
    s_out = s;
    return pf + s;
}

// Split master: w's bits = (p << 16) + r, r an int16 (two's complement, mod 2^32).
__device__ __forceinline__ uint32_t join_bits(uint32_t p16, uint32_t r16)
{
    return (p16 << 16) + (uint32_t)(int32_t)(int16_t)(uint16_t)r16;
}

// p = nearest bf16 of w, ties away from zero (bit 15 of the dropped half rounds the
// magnitude up), so the remainder w - (p << 16) lies in [-32768, 32767]; a NaN
// keeps its high half with the quiet bit set.  Returns p; r through `r16`.
// Both candidates are formed and one is picked with a mask: written as a
// conditional, the NaN case compiled to a divergent branch per element.
__device__ __forceinline__ uint32_t split_bits(uint32_t w, uint32_t& r16)
{
    const uint32_t nan_mask = 0u - (uint32_t)((w & 0x7fffffffu) > 0x7f800000u);
    const uint32_t rounded = (w >> 16) + ((w >> 15) & 1u);
    const uint32_t quieted = (w >> 16) | 0x0040u;
    const uint32_t hi = (rounded & ~nan_mask) | (quieted & nan_mask);
    r16 = (w - (hi << 16)) & 0xffffu;
    return hi & 0xffffu;
}

// ---------------------------------------------------------------------------
// Prologue: one lane.  skip = *found_inf != 0; otherwise t = *step + 1, the
// step's scalars, and *step = t.  With a loss-scale state, the unscale factor
// is 1/scale and the state advances by the dynamic loss-scaling rule.  With a
// clipping rule, the unscale factor is multiplied by the clipping factor, and a
// sum of squares that is not finite skips the step as the flag does.
// ---------------------------------------------------------------------------

__device__ double pow_sq(double b, int64_t t)
{
    // beta^t by right-to-left binary powering: square the base every round,
    // multiply it into the result for every set bit of t.
    double r = 1.0;
    for (; t > 0; t >>= 1) {
        if (t & 1) r = r * b;
        b = b * b;
    }
    return r;
}

// Multiplies the gradients' multiplier by the clipping factor: one rounding of the
// binary64 product.  Returns false if the step has to be skipped.
// Callers test clip.sumsq first.  The empty statement keeps the square root and the
// division behind that test: without it the compiler formed them in every step, clipped or not,
// ahead of the single launch's data loads: 0.1 to 0.25 us of a plain step of up to 1 M
// elements (of 5 to 7 us) on MI355X.
__device__ __forceinline__ bool clip_scale(const ClipRule& clip, double sumsq, float& inv_scale)
{
    asm volatile("" : "+s"(sumsq));
    double factor;
    if (!clip_factor(clip, sumsq, inv_scale, factor)) return false;
    inv_scale = (float)((double)inv_scale * factor);
    return true;
}

// The scalars of step t: binary64 from +, -, *, / only, each rounded once to
// binary32.  The prologue kernel and the single-launch form share this code.
__device__ __forceinline__ Coef step_coef(const adamw_hparams& hp, int64_t t, float inv_scale)
{
    const double lr = (double)hp.lr, wd = (double)hp.weight_decay;
    const double b1t = pow_sq((double)hp.beta1, t);
    const double b2t = pow_sq((double)hp.beta2, t);
    Coef c;
    c.step_size = (float)(lr / (1.0 - b1t));
    c.rbc2 = (float)(1.0 / (1.0 - b2t));
    c.decay = (float)(1.0 - lr * wd);
    c.lrwd = (float)(lr * wd);
    c.omb1 = 1.0f - hp.beta1;
    c.omb2 = 1.0f - hp.beta2;
    c.beta1 = hp.beta1;
    c.beta2 = hp.beta2;
    c.eps = hp.eps;
    c.inv_scale = inv_scale;
    return c;
}

// The dynamic loss-scaling rule, applied once per step after the step's
// unscale factor 1/scale has been read: back off on an overflow, grow after
// growth_interval clean steps in a row (a growth that would overflow binary32
// is refused).  One lane of the grid runs it.
__device__ __forceinline__ void advance_loss_scale(adamw_loss_scale_state* amp, const adamw_loss_scaler& scaler,
                                                   float scale, bool skip)
{
    if (scaler.growth_interval < 1) return;   // a scale that this call only reads
    if (skip) {
        amp->scale = scale * scaler.backoff_factor;
        amp->growth_tracker = 0;
    } else {
        const int32_t run = amp->growth_tracker + 1;
        if (run == scaler.growth_interval) {
            const float grown = scale * scaler.growth_factor;
            if (__builtin_isfinite(grown)) amp->scale = grown;
            amp->growth_tracker = 0;
        } else {
            amp->growth_tracker = run;
        }
    }
}

// A step is taken only from a counter in [0, INT32_MAX): the step it takes,
// t = counter + 1, must be a positive int32.  From any other value the call
// writes nothing at all (no buffer, no counter, no loss scale), as on a skip.
__device__ __forceinline__ bool counter_in_range(int32_t step) { return step >= 0 && step != INT32_MAX; }

__global__ void prologue_kernel(adamw_hparams hp, int32_t* __restrict__ step, const int32_t* __restrict__ found_inf,
                                LaunchScalars* __restrict__ out, adamw_loss_scale_state* __restrict__ amp,
                                adamw_loss_scaler scaler, ClipRule clip)
{
    if (threadIdx.x != 0 || blockIdx.x != 0) return;
    LaunchScalars s{};
    const int32_t step0 = *step;
    if (!counter_in_range(step0)) {
        // no step t = step0 + 1 exists in int32: write nothing but the skip mark
        s.skip = 1;
        *out = s;
        return;
    }
    bool skip = found_inf && *found_inf != 0;
    const float scale = amp ? amp->scale : 0.0f;
    float inv_scale = amp ? (float)(1.0 / (double)scale) : hp.inv_loss_scale;
    if (clip.sumsq) skip |= !clip_scale(clip, *clip.sumsq, inv_scale);
    // this step unscales by the current scale; the scale for the next step
    // follows from the flag
    if (amp) advance_loss_scale(amp, scaler, scale, skip);
    if (skip) {
        s.skip = 1;
        *out = s;
        return;
    }
    const int64_t t = (int64_t)step0 + 1;
    const Coef c = step_coef(hp, t, inv_scale);
    s.skip = 0;
    s.t = (int32_t)t;
    s.step_size = c.step_size;
    s.rbc2 = c.rbc2;
    s.decay = c.decay;
    s.lrwd = c.lrwd;
    s.omb1 = c.omb1;
    s.omb2 = c.omb2;
    s.beta1 = c.beta1;
    s.beta2 = c.beta2;
    s.eps = c.eps;
    s.inv_scale = c.inv_scale;
    *out = s;
    *step = (int32_t)t;
}

// ---------------------------------------------------------------------------
// Update kernel
// ---------------------------------------------------------------------------

// The cache policy of the streaming accesses: every element is touched exactly once
// per step, so loads and stores are non-temporal (bit 0 = loads, bit 1 = stores).
// The mixed family's gradient, which is not written back, is loaded plainly: on
// MI355X (OPT-1.3B list) 85.7 % of peak against 83.1 with non-temporal loads on
// blocked state, 78.7 against 79.1 per tensor; plain loads of the state streams lost
// 0.7 and 2.4 points.  In the pure family, plain loads cost the Kahan step 8 %, and the
// steps with an fp32 stream 2-12 points; there too the gradient alone is loaded plainly
// where a stream is fp32.  Non-temporal / plain gradient, per tensor and blocked: split
// master, BERT 222 / 212 and 215 / 207 us, OPT-1.3B 5,528 / 5,541 and 5,369 / 5,315, 10,000
// ragged tensors 12,363 / 12,402 and 12,449 / 12,164; bf16 moments with fp32
// compensation, OPT-125m 453 / 427 and 433 / 415, ragged 10,544 / 10,510 and 10,625 /
// 10,021.
#ifndef ADAMW_NT_MIXED
#define ADAMW_NT_MIXED 3
#endif
#ifndef ADAMW_NT_MIXED_GRAD
#define ADAMW_NT_MIXED_GRAD 2
#endif
#ifndef ADAMW_NT_PURE
#define ADAMW_NT_PURE 3
#endif
#ifndef ADAMW_NT_CHECK
#define ADAMW_NT_CHECK 1
#endif
constexpr int kCheckUnroll = kCheckChunkMult;

// The overflow check's workgroup -> chunk map: xcd_chunk (layout.hpp), under
// which each XCD walks one contiguous run of chunks.
__device__ __forceinline__ uint32_t chunk_index(uint32_t b, uint32_t nb) { return xcd_chunk(b, nb); }

__device__ __forceinline__ Work work_of(const DevChunk* items, uint32_t n_shared, uint32_t n_single)
{
    const ItemPart ip = update_item(blockIdx.x, n_shared, n_single);
    return item_work(items[ip.item], ip);
}

__device__ __forceinline__ Coef load_coef(const LaunchScalars* sc)
{
    Coef c;
    c.step_size = sc->step_size;
    c.rbc2 = sc->rbc2;
    c.decay = sc->decay;
    c.lrwd = sc->lrwd;
    c.omb1 = sc->omb1;
    c.omb2 = sc->omb2;
    c.beta1 = sc->beta1;
    c.beta2 = sc->beta2;
    c.eps = sc->eps;
    c.inv_scale = sc->inv_scale;
    return c;
}

// What a single-launch workgroup reads before its data: the step it takes, the loss
// scale and the sum of squares to clip by.
struct StepIn {
    int64_t t;
    float scale;
    double sumsq;
};

// Start of a step in an update kernel.  Two-launch form: the prologue kernel
// has written the skip flag and the scalars.  Single launch: the workgroup
// reads the flag, the counter and (with a dynamic loss scale) the scale
// itself; its scalars are formed by fused_coef once its data loads are in
// flight.  Returns false on a skipped step (uniform over the grid: nothing is
// written, the counter is kept; workgroup 0 backs the loss scale off) and on a
// counter out of range (nothing is written at all).
template <bool FUSED>
__device__ __forceinline__ bool begin_step(const LaunchScalars* sc, const FusedStep& fs, Coef& c, StepIn& in)
{
    if constexpr (FUSED) {
        // All four reads come before the one store a workgroup may make here,
        // so that the compiler can issue them as scalar loads (a store ahead of
        // a load in the kernel would turn it into a vector load with a full
        // wait before the data loads start).
        const int32_t flag = fs.found_inf ? *fs.found_inf : 0;
        const int32_t step = *fs.step;
        in.scale = fs.amp ? fs.amp->scale : 0.0f;
        in.sumsq = fs.clip.sumsq ? *fs.clip.sumsq : 0.0;
        if (!counter_in_range(step)) return false;
        if (flag != 0 || !is_sum_of_squares(in.sumsq)) {
            if (fs.amp && blockIdx.x == 0 && threadIdx.x == 0) advance_loss_scale(fs.amp, fs.scaler, in.scale, true);
            return false;
        }
        in.t = (int64_t)step + 1;   // as the prologue: no int32 overflow in the scalars
    } else {
        if (sc->skip) return false;
        c = load_coef(sc);
    }
    return true;
}

template <bool FUSED>
__device__ __forceinline__ void fused_coef(const FusedStep& fs, const StepIn& in, Coef& c)
{
    if constexpr (FUSED) {
        float inv_scale = fs.amp ? (float)(1.0 / (double)in.scale) : fs.hp.inv_loss_scale;
        if (fs.clip.sumsq) clip_scale(fs.clip, in.sumsq, inv_scale);
        c = step_coef(fs.hp, in.t, inv_scale);
    }
}

// End of a single-launch step: once every wave of this workgroup is past its
// reads of the counter and the loss scale, one lane counts the workgroup; the
// last one of the grid stores the new counter and advances the loss scale.
template <bool FUSED>
__device__ __forceinline__ void end_step(const FusedStep& fs, const StepIn& in)
{
    if constexpr (FUSED) {
        __syncthreads();
        if (threadIdx.x == 0 && grid_done(fs.done, blockIdx.x, gridDim.x)) {
            __hip_atomic_store(fs.step, (int32_t)in.t, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (fs.amp) advance_loss_scale(fs.amp, fs.scaler, in.scale, false);
        }
    }
}

// MODE 0: mixed bf16, 1: mixed fp16 (the split-master step is a pure-family
// kernel below: its param is read as well as written)
template <int MODE, bool FUSED>
__global__ __launch_bounds__(kBlockMixed) void update_kernel(const DevSeg* __restrict__ segs,
                                                        const DevChunk* __restrict__ items, uint32_t n_shared,
                                                        uint32_t n_single,
                                                        const LaunchScalars* __restrict__ sc, FusedStep fs)
{
    Coef c{};
    StepIn in{};
    if (!begin_step<FUSED>(sc, fs, c, in)) return;
    constexpr bool F16 = (MODE == 1);
    constexpr int NTG = ADAMW_NT_MIXED_GRAD, NTS = ADAMW_NT_MIXED;   // gradient; state and param
    constexpr int E = 4, N = kPack / E;   // elements of a unit, units of a lane and pass
    const Work wk = work_of(items, n_shared, n_single);
    const DevSeg& sg = segs[wk.seg];
    const uint64_t off = wk.off;
    const uint32_t tid = threadIdx.x;

    GLOBAL uint16_t* __restrict__ p = gptr<uint16_t>(sg.ptr[ADAMW_STREAM_PARAM], off);
    const GLOBAL uint16_t* __restrict__ g = gptr<const uint16_t>(sg.ptr[ADAMW_STREAM_GRAD], off);
    GLOBAL float* __restrict__ m = gptr<float>(sg.ptr[ADAMW_STREAM_EXP_AVG], off);
    GLOBAL float* __restrict__ v = gptr<float>(sg.ptr[ADAMW_STREAM_EXP_AVG_SQ], off);
    GLOBAL float* __restrict__ w = gptr<float>(sg.ptr[ADAMW_STREAM_AUX], off);
    if (wk.body) {
        const uint32_t units = wk.body / E, pass = wk.parts * kBlockMixed * N;
        const GLOBAL u32x2* __restrict__ g2 = reinterpret_cast<const GLOBAL u32x2*>(g + wk.head);
        GLOBAL u32x2* __restrict__ p2 = reinterpret_cast<GLOBAL u32x2*>(p + wk.head);
        GLOBAL f32x4* __restrict__ m4 = reinterpret_cast<GLOBAL f32x4*>(m + wk.head);
        GLOBAL f32x4* __restrict__ v4 = reinterpret_cast<GLOBAL f32x4*>(v + wk.head);
        GLOBAL f32x4* __restrict__ w4 = reinterpret_cast<GLOBAL f32x4*>(w + wk.head);
        const auto update = [&](u32x2 G, f32x4& W, f32x4& M, f32x4& V) {
            float* wf = reinterpret_cast<float*>(&W);
            float* mf = reinterpret_cast<float*>(&M);
            float* vf = reinterpret_cast<float*>(&V);
            const uint32_t gw[2] = {G.x, G.y};
            uint32_t pw[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const f32x2 gg = widen2<F16>(gw[j]);
                const float a = mixed_elem(gg.x, wf[2 * j], mf[2 * j], vf[2 * j], c);
                const float b = mixed_elem(gg.y, wf[2 * j + 1], mf[2 * j + 1], vf[2 * j + 1], c);
                pw[j] = narrow2<F16>(a, b);
            }
            return u32x2{pw[0], pw[1]};
        };
        // A wave's whole passes without a test, then its last units one by one: with a test
        // before each unit's accesses the compiler waits for one unit's loads before it
        // issues the next one's (blocked state: 83.8 % of peak on MI355X at best, 77.9 with
        // some register assignments, against 86).  The scheduling barrier keeps every load
        // ahead of the arithmetic; left to itself the compiler moved one gradient load
        // behind a wait in some variants (blocked 81 %).  Whole by wave rather than by pass of the
        // workgroup: 0.2 points blocked, 0.3 to 1.1 per tensor.
        const uint32_t last = __builtin_amdgcn_readfirstlane(unit_at<kTilePacksMixed, N>(tid | 63u, wk, N - 1));
        uint32_t at = 0;
        for (; at + last < units; at += pass) {
            u32x2 G[N], P[N];
            f32x4 W[N], M[N], V[N];
#pragma unroll
            for (int h = 0; h < N; ++h) {
                const uint32_t k = at + unit_at<kTilePacksMixed, N>(tid, wk, h);
                G[h] = ld<NTG>(g2 + k);
                W[h] = ld<NTS>(w4 + k);
                M[h] = ld<NTS>(m4 + k);
                V[h] = ld<NTS>(v4 + k);
            }
            __builtin_amdgcn_sched_barrier(0);
            if (at == 0) fused_coef<FUSED>(fs, in, c);   // while the loads are in flight
#pragma unroll
            for (int h = 0; h < N; ++h) P[h] = update(G[h], W[h], M[h], V[h]);
#pragma unroll
            for (int h = 0; h < N; ++h) {
                const uint32_t k = at + unit_at<kTilePacksMixed, N>(tid, wk, h);
                st<NTS>(w4 + k, W[h]);
                st<NTS>(m4 + k, M[h]);
                st<NTS>(v4 + k, V[h]);
                st<NTS>(p2 + k, P[h]);
            }
        }
        if (at < units) {   // the last units, which do not fill a pass of the wave
            if (at == 0) fused_coef<FUSED>(fs, in, c);
#pragma unroll
            for (int h = 0; h < N; ++h) {
                const uint32_t k = at + unit_at<kTilePacksMixed, N>(tid, wk, h);
                if (k >= units) continue;
                f32x4 W = ld<NTS>(w4 + k), M = ld<NTS>(m4 + k), V = ld<NTS>(v4 + k);
                const u32x2 P = update(ld<NTG>(g2 + k), W, M, V);
                st<NTS>(w4 + k, W);
                st<NTS>(m4 + k, M);
                st<NTS>(v4 + k, V);
                st<NTS>(p2 + k, P);
            }
        }
    }
    if (wk.edge) {
        if (wk.body == 0) fused_coef<FUSED>(fs, in, c);
        for (uint32_t e = wk.part * kBlockMixed + tid; e < wk.edge; e += wk.parts * kBlockMixed) {
            const uint32_t i = edge_at(wk, e);
            float wi = w[i], mi = m[i], vi = v[i];
            const float nw = mixed_elem(widen1<F16>(g[i]), wi, mi, vi, c);
            w[i] = wi;
            m[i] = mi;
            v[i] = vi;
            p[i] = narrow1<F16>(nw);
        }
    }
    end_step<FUSED>(fs, in);
}

// The aux stream of a pure-family step.
constexpr int kAuxNone = 0;    // no aux stream: p' = round(p * decay - step_size * u)
constexpr int kAuxKahan = 1;   // bf16 Kahan compensation c
constexpr int kAuxSplit = 2;   // int16 remainder r of the split fp32 master w = join(p, r)
constexpr int kAuxKahan32 = 3; // fp32 Kahan compensation c (the residual kept unrounded)

// Steps whose param is read as well as written, over bf16 params: the pure-bf16
// family with chosen state precisions (M32 / V32 = fp32 exp_avg / exp_avg_sq,
// else bf16; aux none, bf16 or fp32 compensation; <false, false, kAuxKahan> is
// the pure-bf16 Kahan mode), and the split-master mixed step (<true, true,
// kAuxSplit>).
template <bool M32, bool V32, int AUX, bool FUSED>
__global__ __launch_bounds__(kBlockPure) void update_pure_kernel(const DevSeg* __restrict__ segs,
                                                                            const DevChunk* __restrict__ items,
                                                                            uint32_t n_shared, uint32_t n_single,
                                                                            const LaunchScalars* __restrict__ sc,
                                                                            FusedStep fs)
{
    Coef c{};
    StepIn in{};
    if (!begin_step<FUSED>(sc, fs, c, in)) return;
    constexpr bool KAHAN = AUX == kAuxKahan, SPLIT = AUX == kAuxSplit, KAHAN32 = AUX == kAuxKahan32;
    static_assert(!SPLIT || (M32 && V32), "the split master keeps fp32 moments");
    constexpr int NT = ADAMW_NT_PURE;
    // elements of a unit, 32-bit words of a 16-bit stream's unit, units of a lane and pass
    constexpr int E = M32 || V32 || KAHAN32 ? 4 : kPack, H = E / 2, N = kPack / E;
    constexpr int P = E == 4 ? kTilePacksMixed : kTilePacks;
    constexpr int NTG = E == 4 ? ADAMW_NT_MIXED_GRAD : NT;   // the gradient
    const Work wk = work_of(items, n_shared, n_single);
    const DevSeg& sg = segs[wk.seg];
    const uint64_t off = wk.off;
    const uint32_t tid = threadIdx.x;
    using MT = typename std::conditional<M32, float, uint16_t>::type;
    using VT = typename std::conditional<V32, float, uint16_t>::type;
    GLOBAL uint16_t* __restrict__ p = gptr<uint16_t>(sg.ptr[ADAMW_STREAM_PARAM], off);
    const GLOBAL uint16_t* __restrict__ g = gptr<const uint16_t>(sg.ptr[ADAMW_STREAM_GRAD], off);
    GLOBAL MT* __restrict__ m = gptr<MT>(sg.ptr[ADAMW_STREAM_EXP_AVG], off);
    GLOBAL VT* __restrict__ v = gptr<VT>(sg.ptr[ADAMW_STREAM_EXP_AVG_SQ], off);
    using CT = typename std::conditional<KAHAN32, float, uint16_t>::type;
    GLOBAL CT* __restrict__ cc = gptr<CT>(sg.ptr[ADAMW_STREAM_AUX], off);

    if (wk.body) {
        const uint32_t units = wk.body / E, pass = wk.parts * kBlockPure * N;
        using W16 = words_t<H>;   // a unit of a 16-bit stream
        using WM = words_t<M32 ? E : H>;
        using WV = words_t<V32 ? E : H>;
        using WC = words_t<KAHAN32 ? E : H>;
        const GLOBAL W16* __restrict__ gu = reinterpret_cast<const GLOBAL W16*>(g + wk.head);
        GLOBAL W16* __restrict__ pu = reinterpret_cast<GLOBAL W16*>(p + wk.head);
        GLOBAL WM* __restrict__ mu = reinterpret_cast<GLOBAL WM*>(m + wk.head);
        GLOBAL WV* __restrict__ vu = reinterpret_cast<GLOBAL WV*>(v + wk.head);
        GLOBAL WC* __restrict__ cu = reinterpret_cast<GLOBAL WC*>(cc + wk.head);
        const auto update = [&](const W16& G, W16& Pv, WM& M, WV& V, WC& C) {
            const uint32_t* gw = reinterpret_cast<const uint32_t*>(&G);
            uint32_t* pw = reinterpret_cast<uint32_t*>(&Pv);
            uint32_t* cw = reinterpret_cast<uint32_t*>(&C);
            uint32_t* mw = reinterpret_cast<uint32_t*>(&M);
            uint32_t* vw = reinterpret_cast<uint32_t*>(&V);
#pragma unroll
            for (int j = 0; j < H; ++j) {
                const f32x2 gg = widen2<false>(gw[j]);
                const f32x2 pp = widen2<false>(pw[j]);
                float ma, mb, va, vb;
                if constexpr (M32) {
                    ma = __uint_as_float(mw[2 * j]);
                    mb = __uint_as_float(mw[2 * j + 1]);
                } else {
                    const f32x2 t2 = widen2<false>(mw[j]);
                    ma = t2.x;
                    mb = t2.y;
                }
                if constexpr (V32) {
                    va = __uint_as_float(vw[2 * j]);
                    vb = __uint_as_float(vw[2 * j + 1]);
                } else {
                    const f32x2 t2 = widen2<false>(vw[j]);
                    va = t2.x;
                    vb = t2.y;
                }
                if constexpr (SPLIT) {
                    float wa = __uint_as_float(join_bits(pw[j] & 0xffffu, cw[j] & 0xffffu));
                    float wb = __uint_as_float(join_bits(pw[j] >> 16, cw[j] >> 16));
                    mixed_elem(gg.x, wa, ma, va, c);
                    mixed_elem(gg.y, wb, mb, vb, c);
                    uint32_t ra, rb;
                    const uint32_t pa = split_bits(__float_as_uint(wa), ra);
                    const uint32_t pb = split_bits(__float_as_uint(wb), rb);
                    pw[j] = pa | (pb << 16);
                    cw[j] = ra | (rb << 16);
                } else if constexpr (KAHAN) {
                    const f32x2 cf = widen2<false>(cw[j]);
                    float sa, sb;
                    const float ta = kahan_sum(gg.x, pp.x, cf.x, ma, va, c, sa);
                    const float tb = kahan_sum(gg.y, pp.y, cf.y, mb, vb, c, sb);
                    pw[j] = narrow2<false>(ta, tb);
                    const f32x2 pn = widen2<false>(pw[j]);
                    cw[j] = narrow2<false>(sa - (pn.x - pp.x), sb - (pn.y - pp.y));
                } else if constexpr (KAHAN32) {
                    float sa, sb;
                    const float ta = kahan_sum(gg.x, pp.x, __uint_as_float(cw[2 * j]), ma, va, c, sa);
                    const float tb = kahan_sum(gg.y, pp.y, __uint_as_float(cw[2 * j + 1]), mb, vb, c, sb);
                    pw[j] = narrow2<false>(ta, tb);
                    const f32x2 pn = widen2<false>(pw[j]);
                    cw[2 * j] = __float_as_uint(sa - (pn.x - pp.x));
                    cw[2 * j + 1] = __float_as_uint(sb - (pn.y - pp.y));
                } else {
                    float wa = pp.x, wb = pp.y;
                    mixed_elem(gg.x, wa, ma, va, c);
                    mixed_elem(gg.y, wb, mb, vb, c);
                    pw[j] = narrow2<false>(wa, wb);
                }
                if constexpr (M32) {
                    mw[2 * j] = __float_as_uint(ma);
                    mw[2 * j + 1] = __float_as_uint(mb);
                } else {
                    mw[j] = narrow2<false>(ma, mb);
                }
                if constexpr (V32) {
                    vw[2 * j] = __float_as_uint(va);
                    vw[2 * j + 1] = __float_as_uint(vb);
                } else {
                    vw[j] = narrow2<false>(va, vb);
                }
            }
        };
        const auto load = [&](uint32_t k, W16& G, W16& Pv, WM& M, WV& V, WC& C) {
            G = ld<NTG>(gu + k);
            Pv = ld<NT>(pu + k);
            M = ld<NT>(mu + k);
            V = ld<NT>(vu + k);
            if constexpr (AUX != kAuxNone) C = ld<NT>(cu + k);
            else C = WC(0u);
        };
        const auto store = [&](uint32_t k, const W16& Pv, const WM& M, const WV& V, const WC& C) {
            st<NT>(pu + k, Pv);
            st<NT>(mu + k, M);
            st<NT>(vu + k, V);
            if constexpr (AUX != kAuxNone) st<NT>(cu + k, C);
        };
        if constexpr (N == 1) {
            // One unit per lane and pass, lane by lane.  With the tests of the wide mixes below /
            // so: Kahan steps of 1 M elements 7.0 / 6.9 us, 128 tensors of 4,096 6.8 / 6.0, BERT
            // blocked 147.8 / 146.7, OPT-1.3B 3,664 / 3,670 blocked and 4,062 / 4,070 per tensor;
            // bf16 moments without compensation, OPT-1.3B blocked, 2,822 / 2,854.
            for (uint32_t k = unit_at<P, 1>(tid, wk, 0); k < units; k += pass) {
                W16 G[N], Pv[N];
                WM M[N];
                WV V[N];
                WC C[N];
                load(k, G[0], Pv[0], M[0], V[0], C[0]);
                fused_coef<FUSED>(fs, in, c);   // while the loads are in flight
                update(G[0], Pv[0], M[0], V[0], C[0]);
                store(k, Pv[0], M[0], V[0], C[0]);
            }
        } else if constexpr (FUSED) {
            // A wave's whole passes without a test, as in the mixed kernel: a single launch is
            // short of time, not of bandwidth (split step, 4,096 elements 5.4 -> 5.2 us,
            // 1 M 7.9 -> 7.65; fp32 moments and bf16 compensation 1 M 7.1 -> 6.8).
            const uint32_t last = __builtin_amdgcn_readfirstlane(unit_at<P, N>(tid | 63u, wk, N - 1));
            uint32_t at = 0;
            for (; at + last < units; at += pass) {
                W16 G[N], Pv[N];
                WM M[N];
                WV V[N];
                WC C[N];
#pragma unroll
                for (int h = 0; h < N; ++h) load(at + unit_at<P, N>(tid, wk, h), G[h], Pv[h], M[h], V[h], C[h]);
                __builtin_amdgcn_sched_barrier(0);
                if (at == 0) fused_coef<FUSED>(fs, in, c);
#pragma unroll
                for (int h = 0; h < N; ++h) update(G[h], Pv[h], M[h], V[h], C[h]);
#pragma unroll
                for (int h = 0; h < N; ++h) store(at + unit_at<P, N>(tid, wk, h), Pv[h], M[h], V[h], C[h]);
            }
            if (at < units) {   // the last units, which do not fill a pass of the wave
                if (at == 0) fused_coef<FUSED>(fs, in, c);
#pragma unroll
                for (int h = 0; h < N; ++h) {
                    const uint32_t k = at + unit_at<P, N>(tid, wk, h);
                    if (k >= units) continue;
                    W16 G, Pv;
                    WM M;
                    WV V;
                    WC C;
                    load(k, G, Pv, M, V, C);
                    update(G, Pv, M, V, C);
                    store(k, Pv, M, V, C);
                }
            }
        } else {
            for (uint32_t at = 0; at < units; at += pass) {
                W16 G[N], Pv[N];
                WM M[N];
                WV V[N];
                WC C[N];
                const auto load_unit = [&](int h, uint32_t k) {
                    G[h] = ld<NTG>(gu + k);
                    Pv[h] = ld<NT>(pu + k);
                    M[h] = ld<NT>(mu + k);
                    V[h] = ld<NT>(vu + k);
                    if constexpr (AUX != kAuxNone) C[h] = ld<NT>(cu + k);
                };
                // Uniform: no lane is past the item's end.  Here the stores keep a test each: a
                // straight pass as in the mixed kernel was 0.5-3 points of peak slower.
                const bool whole = at + pass <= units;
                if (whole) {
#pragma unroll
                    for (int h = 0; h < N; ++h) load_unit(h, at + unit_at<P, N>(tid, wk, h));
                } else {
#pragma unroll
                    for (int h = 0; h < N; ++h) {
                        const uint32_t k = at + unit_at<P, N>(tid, wk, h);
                        G[h] = Pv[h] = W16(0u);
                        M[h] = WM(0u);
                        V[h] = WV(0u);
                        C[h] = WC(0u);
                        if (k < units) load_unit(h, k);
                    }
                }
#pragma unroll
                for (int h = 0; h < N; ++h) update(G[h], Pv[h], M[h], V[h], C[h]);
#pragma unroll
                for (int h = 0; h < N; ++h) {
                    const uint32_t k = at + unit_at<P, N>(tid, wk, h);
                    if (!whole && k >= units) continue;
                    st<NT>(pu + k, Pv[h]);
                    st<NT>(mu + k, M[h]);
                    st<NT>(vu + k, V[h]);
                    if constexpr (AUX != kAuxNone) st<NT>(cu + k, C[h]);
                }
            }
        }
    }
    if (wk.edge) {
        // where the lanes that take the ends (up to 14, the first of part 0) may have had no
        // unit to form the scalars at, they do it here
        if (wk.body < (N == 1 ? 16u * kPack : 1u)) fused_coef<FUSED>(fs, in, c);
        for (uint32_t e = wk.part * kBlockPure + tid; e < wk.edge; e += wk.parts * kBlockPure) {
            const uint32_t i = edge_at(wk, e);
            const float pf = widen1<false>(p[i]);
            float mi, vi;
            if constexpr (M32) mi = m[i]; else mi = widen1<false>(m[i]);
            if constexpr (V32) vi = v[i]; else vi = widen1<false>(v[i]);
            const float gi = widen1<false>(g[i]);
            if constexpr (SPLIT) {
                float w = __uint_as_float(join_bits(p[i], cc[i]));
                mixed_elem(gi, w, mi, vi, c);
                uint32_t ri;
                const uint32_t pi = split_bits(__float_as_uint(w), ri);
                p[i] = (uint16_t)pi;
                cc[i] = (uint16_t)ri;
            } else if constexpr (KAHAN) {
                float s;
                const float tot = kahan_sum(gi, pf, widen1<false>(cc[i]), mi, vi, c, s);
                const uint16_t pn = narrow1<false>(tot);
                cc[i] = narrow1<false>(s - (widen1<false>(pn) - pf));
                p[i] = pn;
            } else if constexpr (KAHAN32) {
                float s;
                const float tot = kahan_sum(gi, pf, cc[i], mi, vi, c, s);
                const uint16_t pn = narrow1<false>(tot);
                cc[i] = s - (widen1<false>(pn) - pf);
                p[i] = pn;
            } else {
                float w = pf;
                mixed_elem(gi, w, mi, vi, c);
                p[i] = narrow1<false>(w);
            }
            if constexpr (M32) m[i] = mi; else m[i] = narrow1<false>(mi);
            if constexpr (V32) v[i] = vi; else v[i] = narrow1<false>(vi);
        }
    }
    end_step<FUSED>(fs, in);
}

// ---------------------------------------------------------------------------
// Overflow check
// ---------------------------------------------------------------------------

__global__ void zero_flag_kernel(int32_t* __restrict__ flag)
{
    if (threadIdx.x == 0 && blockIdx.x == 0) *flag = 0;
}

// Nonzero iff one of the two 16-bit elements in w has an all-ones exponent
// field (EXP = 0x7c00 for fp16, 0x7f80 for bf16).
template <uint32_t EXP>
__device__ __forceinline__ uint32_t nonfinite2(uint32_t w)
{
    const uint32_t x = ~w & (EXP | (EXP << 16));
    return (uint32_t)((x & 0xffffu) == 0) | (uint32_t)((x >> 16) == 0);
}

// FUSED: a single launch that also replaces the zeroing of the flag: the
// workgroups count themselves with their verdicts (grid_done_verdict), and the last
// one stores the flag, 1 if any workgroup saw a non-finite value, else 0.
template <bool F16, bool FUSED>
__global__ __launch_bounds__(kBlockCheck) void check_kernel(const DevSeg* __restrict__ segs,
                                                       const DevChunk* __restrict__ chunks,
                                                       int32_t* __restrict__ flag, uint32_t* __restrict__ done)
{
    constexpr uint32_t EXP = F16 ? 0x7c00u : 0x7f80u;
    const DevChunk ch = chunks[chunk_index(blockIdx.x, gridDim.x)];
    const GLOBAL uint16_t* __restrict__ g = gptr<const uint16_t>(segs[ch.seg].ptr[ADAMW_STREAM_GRAD], ch.off);
    const uint32_t n = ch.n_kind & kCountMask;
    uint32_t bad = 0;
    if (ch.n_kind & kVecBit) {
        // each lane issues kCheckUnroll loads before testing any: one pass
        // covers a default check chunk
        const GLOBAL u32x4* __restrict__ g4 = reinterpret_cast<const GLOBAL u32x4*>(g);
        const uint32_t npack = n / kPack;
        for (uint32_t k0 = threadIdx.x; k0 < npack; k0 += kBlockCheck * kCheckUnroll) {
            u32x4 q[kCheckUnroll];
#pragma unroll
            for (int u = 0; u < kCheckUnroll; ++u) {
                const uint32_t k = k0 + u * kBlockCheck;
                q[u] = k < npack ? ld<ADAMW_NT_CHECK>(g4 + k) : u32x4{0u, 0u, 0u, 0u};
            }
#pragma unroll
            for (int u = 0; u < kCheckUnroll; ++u)
                bad |= nonfinite2<EXP>(q[u].x) | nonfinite2<EXP>(q[u].y) | nonfinite2<EXP>(q[u].z) |
                       nonfinite2<EXP>(q[u].w);
        }
    } else {
        for (uint32_t i = threadIdx.x; i < n; i += kBlockCheck) bad |= (uint32_t)((g[i] & EXP) == EXP);
    }
    if constexpr (FUSED) {
        const int any = __syncthreads_or((int)bad);
        uint32_t hit = 0;
        if (threadIdx.x == 0 && grid_done_verdict(done, any ? 1u : 0u, &hit))
            __hip_atomic_store(flag, hit ? 1 : 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    } else {
        // one atomic per wavefront that saw a non-finite value
        if (__any((int)bad) && (threadIdx.x % warpSize) == 0)
            __hip_atomic_fetch_or(flag, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

// ---------------------------------------------------------------------------
// Host launchers
// ---------------------------------------------------------------------------

hipError_t launch_prologue(const adamw_hparams& hp, int32_t* d_step, const int32_t* d_found_inf,
                           LaunchScalars* d_scalars, adamw_loss_scale_state* d_amp, const adamw_loss_scaler& scaler,
                           const ClipRule& clip, hipStream_t stream)
{
    hipLaunchKernelGGL(prologue_kernel, dim3(1), dim3(64), 0, stream, hp, d_step, d_found_inf, d_scalars, d_amp,
                       scaler, clip);
    return hipGetLastError();
}

// Two-launch form (fused == nullptr): the update kernel reads the prologue's
// scalars at d_scalars.  Single launch: the kernel forms them from *fused.
template <bool FUSED>
static hipError_t launch_update_as(int kernel, const DevSeg* segs, const DevChunk* items, const UpdateGrid& work,
                                   const LaunchScalars* d_scalars, const FusedStep& fs, hipStream_t stream)
{
    // at most kXcdParts workgroups per chunk (the plan's chunk limit keeps the grid in range)
    const uint32_t n_shared = (uint32_t)work.n_shared, n_single = (uint32_t)work.n_single;
    const dim3 grid((unsigned)work.workgroups()), block(kBlockMixed), block_pure(kBlockPure);
    const size_t lds = update_lds(kernel);
#define ADAMW_UPDATE(KERNEL, BLOCK) \
    hipLaunchKernelGGL(KERNEL, grid, BLOCK, lds, stream, segs, items, n_shared, n_single, d_scalars, fs)
    switch (kernel) {
    case kKernelMixedBf16: ADAMW_UPDATE((update_kernel<0, FUSED>), block); break;
    case kKernelMixedF16: ADAMW_UPDATE((update_kernel<1, FUSED>), block); break;
    case kKernelSplit: ADAMW_UPDATE((update_pure_kernel<true, true, kAuxSplit, FUSED>), block_pure); break;
#define ADAMW_PURE_CASE(M, V, K)                                                                         \
    case kKernelPure + (M) * 4 + (V) * 2 + (K):                                                          \
        ADAMW_UPDATE((update_pure_kernel<M, V, (K) ? kAuxKahan : kAuxNone, FUSED>), block_pure); break;
        ADAMW_PURE_CASE(0, 0, 0) ADAMW_PURE_CASE(0, 0, 1) ADAMW_PURE_CASE(0, 1, 0) ADAMW_PURE_CASE(0, 1, 1)
        ADAMW_PURE_CASE(1, 0, 0) ADAMW_PURE_CASE(1, 0, 1) ADAMW_PURE_CASE(1, 1, 0) ADAMW_PURE_CASE(1, 1, 1)
#undef ADAMW_PURE_CASE
#define ADAMW_PURE_C32_CASE(M, V)                                                                        \
    case kKernelPureC32 + (M) * 2 + (V):                                                                 \
        ADAMW_UPDATE((update_pure_kernel<M, V, kAuxKahan32, FUSED>), block_pure); break;
        ADAMW_PURE_C32_CASE(0, 0) ADAMW_PURE_C32_CASE(0, 1) ADAMW_PURE_C32_CASE(1, 0) ADAMW_PURE_C32_CASE(1, 1)
#undef ADAMW_PURE_C32_CASE
    default:
        return hipErrorInvalidValue;
    }
#undef ADAMW_UPDATE
    return hipGetLastError();
}

hipError_t launch_update(int kernel, const DevSeg* segs, const DevChunk* items, const UpdateGrid& grid,
                         const LaunchScalars* d_scalars, const FusedStep* fused, hipStream_t stream)
{
    if (grid.workgroups() <= 0) return hipSuccess;
    if (fused) return launch_update_as<true>(kernel, segs, items, grid, nullptr, *fused, stream);
    return launch_update_as<false>(kernel, segs, items, grid, d_scalars, FusedStep{}, stream);
}

// ---------------------------------------------------------------------------
// State copy between per-tensor (or flat) state buffers and the blocked buffer
// ---------------------------------------------------------------------------

// One workgroup per chunk of the copy plan: the chunk's elements of each state
// stream, element by element (the two sides need not share their alignment).
template <typename T>
__device__ __forceinline__ void copy_elems(uint64_t dst, uint64_t src, uint64_t off, uint32_t n)
{
    GLOBAL T* __restrict__ d = gptr<T>(dst, off);
    const GLOBAL T* __restrict__ s = gptr<const T>(src, off);
    for (uint32_t i = threadIdx.x; i < n; i += blockDim.x) d[i] = s[i];
}

__global__ __launch_bounds__(kBlockCopy) void state_copy_kernel(const DevCopySeg* __restrict__ segs,
                                                         const DevChunk* __restrict__ chunks, int esz_m, int esz_v,
                                                         int esz_aux, int to_blocked)
{
    const DevChunk ch = chunks[blockIdx.x];
    const DevCopySeg& sg = segs[ch.seg];
    const uint32_t n = ch.n_kind & kCountMask;
    const int esz[3] = {esz_m, esz_v, esz_aux};
    for (int s = 0; s < 3; ++s) {
        const uint64_t dst = to_blocked ? sg.blocked_side[s] : sg.tensor_side[s];
        const uint64_t src = to_blocked ? sg.tensor_side[s] : sg.blocked_side[s];
        if (esz[s] == 4) copy_elems<uint32_t>(dst, src, ch.off, n);
        else if (esz[s] == 2) copy_elems<uint16_t>(dst, src, ch.off, n);
    }
}

hipError_t launch_state_copy(const DevCopySeg* segs, const DevChunk* chunks, int64_t n_chunks, const int esz[3],
                             bool to_blocked, hipStream_t stream)
{
    if (n_chunks <= 0) return hipSuccess;
    hipLaunchKernelGGL(state_copy_kernel, dim3((unsigned)n_chunks), dim3(kBlockCopy), 0, stream, segs, chunks, esz[0],
                       esz[1], esz[2], to_blocked ? 1 : 0);
    return hipGetLastError();
}

__global__ void zero_words_kernel(uint32_t* __restrict__ p, int64_t n)
{
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x) p[i] = 0u;
}

// Zeroes n 32-bit words (a fill kernel rather than a memset, so that it may
// sit in a captured graph).
hipError_t launch_zero_words(uint32_t* p, int64_t n, hipStream_t stream)
{
    hipLaunchKernelGGL(zero_words_kernel, dim3(1), dim3(256), 0, stream, p, n);
    return hipGetLastError();
}

// fused: one launch of the check (it stores the flag itself, through the
// completion counters at done); else zero the flag, then the check ORs into it.
hipError_t launch_check(adamw_dtype g_dtype, const DevSeg* segs, const DevChunk* chunks, int64_t n_chunks,
                        int32_t* d_flag, uint32_t* done, bool fused, hipStream_t stream)
{
    const dim3 grid((unsigned)(n_chunks > 0 ? n_chunks : 1)), block(kBlockCheck);
    if (fused && n_chunks > 0) {
        if (g_dtype == ADAMW_F16)
            hipLaunchKernelGGL((check_kernel<true, true>), grid, block, 0, stream, segs, chunks, d_flag, done);
        else
            hipLaunchKernelGGL((check_kernel<false, true>), grid, block, 0, stream, segs, chunks, d_flag, done);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(zero_flag_kernel, dim3(1), dim3(64), 0, stream, d_flag);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || n_chunks <= 0) return e;
    if (g_dtype == ADAMW_F16)
        hipLaunchKernelGGL((check_kernel<true, false>), grid, block, 0, stream, segs, chunks, d_flag, nullptr);
    else
        hipLaunchKernelGGL((check_kernel<false, false>), grid, block, 0, stream, segs, chunks, d_flag, nullptr);
    return hipGetLastError();
}

}  // namespace adamw
