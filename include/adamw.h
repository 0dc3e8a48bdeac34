/*
 * adamw.h -- C ABI of the MI355X (gfx950) fused AdamW optimizer step.
 *
 * One call updates a whole list of parameter tensors (or one data-parallel
 * rank's share of it) in place on the GPU: one HBM pass over param, grad,
 * exp_avg, exp_avg_sq and an auxiliary buffer, with the arithmetic in fp32
 * registers.
 *
 * The operation.  AdamW: Adam's bias-corrected moment estimates (Kingma & Ba,
 * "Adam", ICLR 2015, Algorithm 1) with weight decay decoupled from the
 * gradient (Loshchilov & Hutter, "Decoupled Weight Decay Regularization",
 * ICLR 2019, Algorithm 2).  The pages that motivate this library name it and
 * its settings without printing the rule: "Distributed optimizer support for
 * BERT" (Usage: fused_adam / distributed_fused_adam; the A40 and A100 tables,
 * "BF16 with O2 optimizations") and "[pure bf16 training] w/ AnyPrecisionAdamW
 * and Kahan summation" (the opt-1.3b command: lr 0.0002, betas 0.9/0.95,
 * weight decay 0.1; --optim_args with bf16 momentum, variance and Kahan
 * compensation buffer).  With t the 1-based index of the step being taken:
 *
 *   g   = grad * inv_loss_scale
 *   m   = beta1*m + (1-beta1)*g
 *   v   = beta2*v + (1-beta2)*g*g
 *   u   = m / (sqrt(v / (1-beta2^t)) + eps)
 *   ADAMW_MIXED:      w = w*(1 - lr*wd) - (lr/(1-beta1^t))*u;  param = round16(w)
 *   ADAMW_PURE_KAHAN: d = -(lr*wd)*p - (lr/(1-beta1^t))*u
 *                     s = c + d;  p' = round_bf16(p + s);  c = round_bf16(s - (p' - p))
 *   ADAMW_MIXED_SPLIT: the ADAMW_MIXED rule on w = join(param, remainder), then
 *                     (param, remainder) = split(w), where join(p, r) is the fp32 whose
 *                     bit pattern is (p << 16) + r in 32-bit two's complement (r read as
 *                     int16) and split(w) takes p = w's nearest bf16, ties away from zero
 *                     (so r = w - (p << 16) always fits int16), and p = w's high half with
 *                     the quiet bit set for a NaN w.  join(split(w)) == w for every
 *                     non-NaN w, so the master is exact fp32 (a reading of the 16-bit
 *                     master copy counted in the ZeRO saving estimate of "Distributed
 *                     optimizer support for BERT").
 *
 * Numerics: every element operation is one IEEE binary32 operation rounded to
 * nearest even, in the order written above, without fused multiply-add;
 * sqrt and division are correctly rounded; subnormals are kept.  The
 * per-launch scalars 1/(1-beta1^t) etc. are formed in binary64 from +,-,*,/
 * (beta^t by right-to-left square-and-multiply) and rounded once to fp32.
 * Narrowing to bf16/fp16 rounds to nearest even.
 *
 * Streams.  Index s of the five per-element buffers:
 *   0 param       ADAMW_MIXED: bf16 or fp16 (= p_dtype), written only
 *                 ADAMW_PURE_KAHAN: bf16, read and written
 *   1 grad        same 16-bit dtype as param; read only, never unscaled in place
 *   2 exp_avg     ADAMW_MIXED: fp32 / ADAMW_PURE_KAHAN: bf16 (first moment m)
 *   3 exp_avg_sq  ADAMW_MIXED: fp32 / ADAMW_PURE_KAHAN: bf16 (second moment v)
 *   4 aux         ADAMW_MIXED: fp32 master weight w / ADAMW_PURE_KAHAN: bf16
 *                 compensation c / ADAMW_MIXED_SPLIT: int16 remainder of the master
 *   (ADAMW_MIXED_SPLIT: param is bf16 and read as well as written; exp_avg and
 *   exp_avg_sq are fp32.)
 * Every buffer is contiguous, 1-D, in device memory, aligned to its element
 * size.  16-byte alignment is not required but is what the fast path uses;
 * misaligned heads and tails are peeled, and a segment whose streams cannot
 * be aligned together is processed element by element.
 *
 * Step counter and skip flag.  *d_step (device int32) is the number of steps
 * taken so far; a step that is taken uses t = *d_step + 1 and stores t.  If
 * d_found_inf is non-null and *d_found_inf != 0 when the step runs (stream
 * order), nothing is written at all and *d_step is left as it is: the fp16
 * loss-scaling skip.  The caller fills the flag with adamw_check_finite.
 * The counter must lie in [0, INT32_MAX) when the step runs: at INT32_MAX (or
 * below 0) no step t fits in int32, and the call writes nothing at all -- no
 * buffer, no counter, no loss scale -- so the parameters stay finite and a
 * caller can detect the saturated counter by reading it.
 *
 * Ownership and execution.  The caller owns every tensor, d_step, d_found_inf
 * and the stream; the library never frees or reallocates them.  All work is
 * enqueued on hip_stream (a hipStream_t; NULL = the null stream of the calling
 * thread's current device) and the call returns without synchronising, unless a list
 * whose chunk table is not on the device takes the place of another list's table: the
 * call then waits until that table's upload, queued by an earlier call, has run, and if
 * the new table is larger than the old one's buffer, for the work queued on the stream.  Every
 * buffer must live on the stream's device.  The library owns only a small
 * device workspace per (device, stream), on the stream's device, holding the
 * launch scalars, the single-launch completion counters (about 8.7 KB) and the
 * chunk table, grown on demand and kept until adamw_release_workspace().  The
 * host arrays inside adamw_tensor_list are read during the call only.
 *
 * HIP graphs.  After one call on a stream with a given list (which allocates
 * the workspace and uploads the list's chunk table), the same call captured on
 * that stream records kernel launches only: no allocation, copy or memset.  A
 * call under capture whose table is not yet on the device (or on a stream
 * without a workspace) is refused with ADAMW_E_INVALID.  A captured step may be
 * replayed any number of times.  It uses the capture stream's workspace
 * (launch scalars, completion counters, chunk table, a norm's partial sums).  The chunk table a
 * capture used is pinned: later calls on the stream, with however many other
 * lists, never evict, move or rewrite it (besides the pinned ones, the stream keeps
 * the tables of the last 8 lists for each kind of call -- a step of one mode, a check, a
 * norm, a clipping -- and of the last 32 while all of them take 64 MiB or less); pinned
 * tables are freed only by
 * adamw_release_workspace(), which therefore must not run while such a graph
 * is in use.  A replay must not overlap other work that uses that workspace:
 * steps enqueued on the capture stream, or replays of other graphs captured on
 * it.  Replaying on the capture stream itself keeps all of these in stream
 * order.
 *
 * Errors.  Arguments are validated before anything is enqueued; on an error
 * nothing is enqueued, no buffer is touched, and adamw_last_error() describes
 * it.  A HIP failure while enqueuing returns ADAMW_E_HIP.  Faults inside a
 * kernel surface at the caller's next synchronisation.  One launch's grid
 * holds at most 2^32 - 1 lanes, so a step plan of more than 2,097,151 chunks
 * (8 workgroups of 256 lanes each: about 34e9 elements at the default chunk,
 * or that many tensors of under 8 elements), a check plan of more than
 * 16,777,215, a norm of more than 16,777,215 (32 KiB each, or one per shorter
 * tensor), or a clipping of more than 2,097,151 (128 KiB each) is rejected with
 * ADAMW_E_INVALID.
 *
 * Concurrency.  Calls may come from several host threads.  Calls on different
 * streams run independently (each stream has its own workspace); two calls
 * must not update the same buffers concurrently.
 */
#ifndef ADAMW_H
#define ADAMW_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define ADAMW_ABI_VERSION 10

typedef enum {
    ADAMW_OK = 0,
    ADAMW_E_INVALID = 1,      /* bad argument: null, negative size, range, alignment, hyper-parameter */
    ADAMW_E_UNSUPPORTED = 2,  /* mode / dtype combination not provided */
    ADAMW_E_NOMEM = 3,        /* workspace allocation failed */
    ADAMW_E_HIP = 4           /* a HIP call failed while enqueuing */
} adamw_status;

typedef enum { ADAMW_F32 = 0, ADAMW_BF16 = 1, ADAMW_F16 = 2 } adamw_dtype;

typedef enum {
    ADAMW_MIXED = 0,       /* 16-bit param/grad (bf16 or fp16) + fp32 master, exp_avg, exp_avg_sq */
    ADAMW_PURE_KAHAN = 1,  /* bf16 param, grad, exp_avg, exp_avg_sq + bf16 Kahan compensation */
    ADAMW_MIXED_SPLIT = 2  /* ADAMW_MIXED with the fp32 master split into the bf16 param and an
                              int16 remainder: 14 B/param resident instead of 16, 26 B moved */
} adamw_mode;

enum {
    ADAMW_STREAM_PARAM = 0,
    ADAMW_STREAM_GRAD = 1,
    ADAMW_STREAM_EXP_AVG = 2,
    ADAMW_STREAM_EXP_AVG_SQ = 3,
    ADAMW_STREAM_AUX = 4,
    ADAMW_NUM_STREAMS = 5
};

/* Hyper-parameters, as fp32.  Requirements: all finite; 0 <= beta1, beta2 < 1;
 * eps >= 0; lr >= 0; weight_decay >= 0; inv_loss_scale > 0 (1.0f = no
 * unscaling; 1/65536 for fp16 loss scale 65536). */
typedef struct {
    float lr;
    float beta1;
    float beta2;
    float eps;
    float weight_decay;
    float inv_loss_scale;
} adamw_hparams;

/* A ragged list of tensors, optionally restricted to one data-parallel rank's
 * ZeRO shard: the elements [shard_begin, shard_end) of the list's flat
 * concatenation in list order (the optimizer-state sharding of "Distributed
 * optimizer support for BERT": each rank keeps and updates 1/DP of the
 * state).  Tensors may straddle the shard's edges; only their elements inside
 * the range are touched.  shard_begin = 0, shard_end = -1 means the whole list.
 *
 * ptr[s] is a host array of device pointers for stream s:
 *   flat_mask bit s == 0: ptr[s][i] is tensor i's buffer (numel[i] elements);
 *   flat_mask bit s == 1: ptr[s][0] is ONE flat buffer of shard_end-shard_begin
 *                         elements holding this rank's share, element 0 being
 *                         flat position shard_begin (e.g. a reduce-scattered
 *                         gradient shard, or ZeRO-sharded master/m/v).
 *   flat_mask & ADAMW_BLOCKED_STATE, flat_mask & ADAMW_FLAT_PAD8: see below.
 * numel is a host array of n_tensors element counts (each >= 0). */
/* flat_mask bit: the blocked state layout.  exp_avg, exp_avg_sq and aux share
 * ONE flat buffer of the shard, ptr[2][0] (16-byte aligned; ptr[3], ptr[4] and
 * flat_mask bits 2-4 are ignored), made of ceil((shard_end - shard_begin) / B)
 * blocks of B = ADAMW_STATE_BLOCK_ELEMS = 16384 elements (every mode).  Block k
 * holds the state of the shard's elements [k*B, (k+1)*B), stream after stream:
 *     [exp_avg x B][exp_avg_sq x B][aux x B]
 * each in its stream's dtype (an unused aux stream takes no room; a block is
 * 192 KiB in ADAMW_MIXED, 160 KiB in ADAMW_MIXED_SPLIT, 96 KiB in
 * ADAMW_PURE_KAHAN, B times the three streams' element sizes for the other
 * pure-bf16 precisions); the last block is padded to B.  For optimizer-owned ZeRO state: the step's per-element
 * state traffic becomes one contiguous region per block instead of three
 * separate streams (fewer concurrently open DRAM rows; measured faster on
 * MI355X).  B is one default update chunk, so splitting work at block edges
 * never leaves a workgroup's lanes idle.  param and grad keep their own layout
 * (adamw_check_finite, which reads only grads, ignores the bit).  The 16-byte
 * vector path needs an element's state address and its param/grad addresses
 * to share their alignment: with per-tensor param/grad buffers that start
 * 16-byte aligned, a tensor whose flat start is not a multiple of 8 elements
 * runs element-wise (correct, but slower: on 10,000 tensors of random lengths
 * the mixed fp16 step fell from 5.6 to 4.2 TB/s on MI355X), so give such lists
 * tensor lengths, or padding, that are multiples of 8 (see ADAMW_FLAT_PAD8). */
#define ADAMW_BLOCKED_STATE (1u << 8)
#define ADAMW_STATE_BLOCK_ELEMS 16384
/* flat_mask bit: the padded flat index.  The list's flat concatenation places
 * every tensor at a multiple of 8 elements: tensor i starts at the sum over
 * j < i of numel[j] rounded up to a multiple of 8, and the gaps hold no
 * element (nothing reads or writes them).  shard_begin and shard_end, flat
 * shard buffers and the blocked state are all indexed in this padded space,
 * as in ZeRO implementations that pad each tensor inside their flat buffers;
 * shard_end may reach the padded total.  With per-tensor buffers that start
 * 16-byte aligned and a shard_begin that is a multiple of 8, every tensor of
 * any length keeps the 16-byte vector path in every layout. */
#define ADAMW_FLAT_PAD8 (1u << 9)

typedef struct {
    int64_t n_tensors;
    const int64_t* numel;
    void* const* ptr[ADAMW_NUM_STREAMS];
    int64_t shard_begin;
    int64_t shard_end;
    uint32_t flat_mask;
} adamw_tensor_list;

/* One AdamW step over one contiguous range of n elements: a single tensor, or
 * one data-parallel rank's flat shard with every pointer already offset to it
 * -- the unit of work of the ZeRO-sharded optimizer of "Distributed optimizer
 * support for BERT" (the remark under the 4 x A40 table: each of the DP ranks
 * keeps the fp32 optimizer state and the 16-bit master copy of 1/DP of the
 * parameters, and steps only that share).
 * param, grad, exp_avg, exp_avg_sq, aux: device buffers of n elements in the
 * layouts above.  p_dtype: ADAMW_BF16 or ADAMW_F16 in ADAMW_MIXED, ADAMW_BF16
 * in ADAMW_PURE_KAHAN and ADAMW_MIXED_SPLIT.  n == 0 is valid (the counter
 * still advances unless skipped).  See the file comment for d_step /
 * d_found_inf. */
adamw_status adamw_step(adamw_mode mode, adamw_dtype p_dtype, int64_t n,
                        void* param, const void* grad, void* exp_avg, void* exp_avg_sq, void* aux,
                        const adamw_hparams* hp, int32_t* d_step, const int32_t* d_found_inf,
                        void* hip_stream);

/* One AdamW step over a ragged tensor list (or its shard), in one launch of
 * the update kernel: the chunked multi-tensor form of the fused optimizer
 * ("fused_adam" in "Distributed optimizer support for BERT").  Same element
 * rule, dtypes, counter and skip semantics as adamw_step. */
adamw_status adamw_multi_tensor_step(adamw_mode mode, adamw_dtype p_dtype, const adamw_tensor_list* list,
                                     const adamw_hparams* hp, int32_t* d_step, const int32_t* d_found_inf,
                                     void* hip_stream);

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the step of
 * adamw_multi_tensor_step -- same arguments, same results bit for bit -- with
 * no device allocation, free or allocating library call.  Its workspace (the
 * launch scalars, the single-launch completion counters and the list's chunk
 * table) lives in one static device array of ADAMW_NOALLOC_SCRATCH_BYTES per
 * GPU, which the library's code object holds on every GPU it runs on until
 * the process ends.  The chunk table takes 64 bytes per segment and 16 per
 * chunk (adamw_plan_inspect lists both) and must fit in
 * ADAMW_NOALLOC_SCRATCH_BYTES - 16384 bytes: about a million chunks of a few
 * large tensors (every chunk 16384 elements: some 1.7e10 elements), about
 * 200,000 of a list with blocked state (one segment per block: some 3.3e9
 * elements; OPT-1.3B takes 6.4 MB).  A larger list is rejected with
 * ADAMW_E_INVALID before anything is enqueued.  A call copies the list's table
 * into the array (a host-to-device copy on hip_stream) unless the last call on
 * this GPU used the same list; under graph capture that copy is refused, as in
 * adamw_multi_tensor_step.  A call captured into a graph pins the table it
 * used, since every replay reads it: later calls on that GPU with another list
 * are then refused with ADAMW_E_INVALID (calls with the same list still run)
 * until adamw_release_workspace(), which unpins it and must not run while
 * such a graph may still be replayed.  Every call on a GPU shares that GPU's
 * array and its contents: calls on one GPU that may overlap (on different
 * streams, or from host threads without an order between them) race on it and
 * must be ordered by the caller, e.g. by issuing them on one stream.  It has no
 * clipped form: adamw_clip_grads before it clips the gradients in place (whose own
 * workspace and table the first call on a stream allocates). */
#define ADAMW_NOALLOC_SCRATCH_BYTES (16u << 20)
adamw_status adamw_multi_tensor_step_noalloc(adamw_mode mode, adamw_dtype p_dtype, const adamw_tensor_list* list,
                                             const adamw_hparams* hp, int32_t* d_step, const int32_t* d_found_inf,
                                             void* hip_stream);

/* State precisions of a pure-bf16 step (the AnyPrecisionAdamW knobs of
 * "[pure bf16 training] w/ AnyPrecisionAdamW and Kahan summation":
 * momentum_dtype, variance_dtype, use_kahan_summation and
 * compensation_buffer_dtype). */
#define ADAMW_KAHAN_NONE 0   /* no compensation: stream 4 (aux) is unused */
#define ADAMW_KAHAN_BF16 1   /* stream 4 (aux) is a bf16 compensation buffer */
#define ADAMW_KAHAN_F32 2    /* stream 4 (aux) is an fp32 compensation buffer */
typedef struct {
    adamw_dtype exp_avg;     /* ADAMW_F32 or ADAMW_BF16 */
    adamw_dtype exp_avg_sq;  /* ADAMW_F32 or ADAMW_BF16 */
    int32_t kahan;           /* ADAMW_KAHAN_NONE, ADAMW_KAHAN_BF16 or ADAMW_KAHAN_F32; other values are rejected */
} adamw_pure_precision;

/* Pure-bf16 step with chosen state precisions: param and grad bf16, exp_avg and
 * exp_avg_sq in the dtypes of *prec (fp32 moments are kept and used exactly;
 * bf16 ones are widened, updated in fp32 and stored rounded to nearest even).
 * With a compensation buffer: the ADAMW_PURE_KAHAN rule, the residual
 * s - (p' - p) stored rounded to bf16 (ADAMW_KAHAN_BF16) or kept as the fp32
 * value it is computed in (ADAMW_KAHAN_F32: 2 more bytes per element each way,
 * and p + c then carries an fp32 master); without: p = round_bf16(p*(1 - lr*wd)
 * - (lr/(1-beta1^t))*u).  {ADAMW_BF16, ADAMW_BF16, ADAMW_KAHAN_BF16} is
 * ADAMW_PURE_KAHAN.
 * Everything else (list, shard, counter, skip flag, errors) as
 * adamw_multi_tensor_step. */
adamw_status adamw_pure_multi_tensor_step(const adamw_pure_precision* prec, const adamw_tensor_list* list,
                                          const adamw_hparams* hp, int32_t* d_step, const int32_t* d_found_inf,
                                          void* hip_stream);

/* Dynamic loss scaling state, in device memory owned by the caller (8 bytes,
 * 4-byte aligned).  growth_tracker counts consecutive steps taken since the
 * scale last changed and must start in [0, growth_interval). */
typedef struct {
    float scale;
    int32_t growth_tracker;
} adamw_loss_scale_state;

/* Dynamic loss scaling rule (host values): after growth_interval consecutive
 * steps without an inf/NaN gradient the scale is multiplied by growth_factor
 * (kept unchanged if the product is not finite); a step with an inf/NaN gradient
 * multiplies it by backoff_factor.  Either event resets the tracker.
 * Requirements: growth_factor finite and >= 1; 0 < backoff_factor <= 1;
 * growth_interval >= 1.  The pages show an fp16-amp run but not its scaler's
 * constants; the usual choice is growth 2, backoff 0.5, interval 2000. */
typedef struct {
    float growth_factor;
    float backoff_factor;
    int32_t growth_interval;
} adamw_loss_scaler;

/* fp16-AMP step with a device-resident dynamic loss scale: as
 * adamw_multi_tensor_step with d_found_inf required, except that the gradient
 * multiplier is (float)(1 / (double)d_scale->scale) read on the device when the
 * step runs (hp->inv_loss_scale is ignored), and that the same launch then
 * advances *d_scale by the rule above using *d_found_inf -- whether or not the
 * step itself was skipped.  No host synchronisation is involved.  Typical
 * sequence per iteration: adamw_check_finite, then this call with the same flag
 * (the opt-125m fp16-amp run on the page "[pure bf16 training] w/
 * AnyPrecisionAdamW and Kahan summation"). */
adamw_status adamw_multi_tensor_step_amp(adamw_mode mode, adamw_dtype p_dtype, const adamw_tensor_list* list,
                                         const adamw_hparams* hp, int32_t* d_step, const int32_t* d_found_inf,
                                         adamw_loss_scale_state* d_scale, const adamw_loss_scaler* scaler,
                                         void* hip_stream);

/* fp16-AMP overflow check, for the fp16 mixed-precision training of the
 * "opt-125m / fp16-amp training from scratch" run on the page "[pure bf16
 * training] w/ AnyPrecisionAdamW and Kahan summation": its loss is scaled, and
 * a step whose scaled gradients hold an inf or NaN must be skipped (see the
 * skip flag in the file comment).  Stores 0 to *d_found_inf (stream
 * ordered), then 1 if any gradient element of the list (stream 1 only; shard range and
 * flat_mask bit 1 honoured) has an all-ones exponent field, i.e. is inf or NaN.
 * g_dtype: ADAMW_F16 or ADAMW_BF16.  Scaled gradients are tested as stored,
 * before any unscaling.  Intended order: adamw_check_finite, then the step
 * with the same d_found_inf (an all-reduce(max) of the flag across ranks
 * would sit between the two in a multi-GPU job). */
adamw_status adamw_check_finite(adamw_dtype g_dtype, const adamw_tensor_list* grads, int32_t* d_found_inf,
                                void* hip_stream);

/* The global norm of a list's gradients, as gradient clipping (Pascanu et al., "On
 * the difficulty of training recurrent neural networks", ICML 2013, section 3.2)
 * and training logs need it: with S = the sum of g*g over the list's elements (stream 1 only;
 * shard range, flat_mask bit 1 and ADAMW_FLAT_PAD8 honoured, as in
 * adamw_check_finite),
 *   *d_sumsq = S, or *d_sumsq + S with accumulate != 0 (required; binary64),
 *   *d_norm = sqrt(*d_sumsq), rounded to binary32 (nullable),
 *   *d_found_inf = 1 if *d_sumsq is not finite, else 0 (nullable).
 * g_dtype: ADAMW_F16, ADAMW_BF16 or ADAMW_F32.  Squares and sums are binary64, so
 * none overflows or underflows and S is within n * 2^-53 (relative) of the exact
 * sum; S is not finite exactly if an element is inf or NaN, which makes
 * *d_found_inf that of adamw_check_finite, in the same pass.  The order of the
 * sum depends only on the list and the tuning knobs: the same call gives the
 * same bits.  Scaled gradients are summed as stored: with a loss scale s the
 * norm of the unscaled gradients is sqrt(S) / s (adamw_clip_grads and
 * adamw_multi_tensor_step_clipped divide by it themselves).
 * Several lists (parameter groups, other dtypes): the first call with accumulate
 * = 0, the others with accumulate = 1, on one stream, d_norm and d_found_inf in
 * the last.  Several ranks: each sums its own shard, then an all-reduce(sum) of
 * *d_sumsq (one binary64 value).  An empty list (or shard) has S = 0. */
adamw_status adamw_grad_norm(adamw_dtype g_dtype, const adamw_tensor_list* grads, int accumulate, double* d_sumsq,
                             float* d_norm, int32_t* d_found_inf, void* hip_stream);

/* The norm of every tensor of a list (stream 1: gradients, or any other tensors
 * handed in there, such as master weights), as a training run logs them, in one
 * pass: entry i of the device arrays of n_tensors entries
 *   d_tensor_sumsq[i] = S_i = the sum of g*g over tensor i's elements inside the
 *                       shard (binary64), d_tensor_norms[i] = sqrt(S_i) (binary32)
 * (either may be null, not both unless the list is empty; a tensor with no element in
 * the shard gets 0),
 * and *d_sumsq = the list's S, the value of adamw_grad_norm bit for bit
 * (nullable).  dtypes, arithmetic and order as adamw_grad_norm. */
adamw_status adamw_tensor_norms(adamw_dtype g_dtype, const adamw_tensor_list* grads, float* d_tensor_norms,
                                double* d_tensor_sumsq, double* d_sumsq, void* hip_stream);

/* Clipping by the global norm: with S = *d_sumsq (adamw_grad_norm's sum over every
 * list and rank), inv the inverse loss scale and total = sqrt(S) * inv the norm of
 * the unscaled gradients, every gradient is multiplied by
 *   f = min(1, max_norm / (total + eps)).
 * S is read when the call runs, in stream order, so the norm's call and an
 * all-reduce of it may be queued just before.  f is formed in binary64.
 * d_sumsq: device, 8-byte aligned.  max_norm: finite, >= 0.  eps: finite, >= 0
 * (usually 1e-6); with max_norm = eps = 0 a zero norm clips nothing. */
typedef struct {
    const double* d_sumsq;
    float max_norm;
    float eps;
} adamw_grad_clip;

/* Clips a list's gradients in place: g = round(g * f) for every element of the
 * list (stream 1 only; shard range, flat_mask bit 1 and ADAMW_FLAT_PAD8 honoured),
 * f rounded once to binary32, one binary32 product, rounded to nearest even in
 * g_dtype (ADAMW_F16, ADAMW_BF16 or ADAMW_F32).  Scaled gradients stay scaled: inv
 * is 1 / d_scale->scale read on the device if d_scale is non-null, else
 * inv_loss_scale (finite, > 0), and only f depends on it.  With f = 1 no element
 * changes and nothing is written.  If S is not finite (an inf or NaN gradient)
 * nothing is written either: the step that follows is to be skipped
 * (adamw_grad_norm's d_found_inf).  A list whose buffers overlap inside the shard (a
 * gradient listed twice) is refused.  For optimizers that take no clipping factor,
 * and for gradients that others read; adamw_multi_tensor_step_clipped needs no such
 * pass. */
adamw_status adamw_clip_grads(adamw_dtype g_dtype, const adamw_tensor_list* grads, const adamw_grad_clip* clip,
                              float inv_loss_scale, const adamw_loss_scale_state* d_scale, void* hip_stream);

/* AdamW step with its gradients clipped by the global norm as they are read: the
 * step of (mode, p_dtype) -- or, with prec non-null, of
 * adamw_pure_multi_tensor_step with *prec (mode and p_dtype ignored) -- whose
 * gradient multiplier is round_f32(inv * f), inv the inverse loss scale and f the
 * factor of *clip, in place of inv.  The gradients are read once and not written,
 * and no 16-bit rounding comes between clipping and moments.  inv is
 * hp->inv_loss_scale, or with d_scale non-null (float)(1 / (double)d_scale->scale)
 * read on the device, which then also advances by *scaler as in
 * adamw_multi_tensor_step_amp.  If *clip->d_sumsq is not finite, or *d_found_inf
 * (nullable) is set, the step is skipped: nothing is written, the counter is kept
 * and the loss scale backs off.  Typical sequence per iteration: adamw_grad_norm
 * over every list, an all-reduce(sum) of *d_sumsq across ranks, then this call per
 * list.  With scaler null *d_scale is read
 * and not advanced: for every list but the last of a step that spans several
 * (parameter groups, each with its own counter).  List, shard, state layouts,
 * counter, graphs and errors as adamw_multi_tensor_step. */
adamw_status adamw_multi_tensor_step_clipped(adamw_mode mode, adamw_dtype p_dtype, const adamw_pure_precision* prec,
                                             const adamw_tensor_list* list, const adamw_hparams* hp,
                                             const adamw_grad_clip* clip, int32_t* d_step, const int32_t* d_found_inf,
                                             adamw_loss_scale_state* d_scale, const adamw_loss_scaler* scaler,
                                             void* hip_stream);

/* Matrices.  A list of matrices is an adamw_tensor_list with a host array `cols` of
 * n_tensors column counts (each >= 1): tensor i is the row-major matrix of
 * numel[i] / cols[i] rows (numel[i] a multiple of cols[i]; 0 elements: nothing is done
 * for it).  A convolution's weight is the matrix of its flattened filters, the experts of
 * a stacked weight are matrices at consecutive addresses, and so are the parts of a fused
 * projection that lie one under another.  A shard takes whole matrices: shard_begin and
 * shard_end have to lie between matrices (the matrices of a ZeRO job are dealt out whole,
 * since a matrix's singular values are no rank's share of it).  flat_mask bits of the streams
 * used and ADAMW_FLAT_PAD8 are honoured; ADAMW_BLOCKED_STATE is refused
 * (ADAMW_E_UNSUPPORTED).
 *
 * Newton-Schulz products.  For a matrix U let X = U / (|U| + eps), |U| the root of the
 * sum of its squares, and `steps` times
 *     X <- a X + b (X X^T) X + c (X X^T)^2 X ,
 * which moves every singular value x of X to a x + b x^3 + c x^5 and keeps the singular
 * vectors; coefficients that take (0, 1] towards 1 make X the nearest
 * (semi-)orthogonal matrix U (U^T U)^(-1/2), approximately (Higham, "Functions of Matrices",
 * SIAM 2008, section 8.3).  With the default coefficients (3.4445, -4.7750, 2.0315) and
 * five steps singular values above about a hundredth of |U| end between 0.68 and 1.14, as
 * the Muon optimizer uses them.
 *
 * Numerics.  |U| is summed in binary64.  The results are those of the definition within the distances below (relative, in
 * the Frobenius norm), beside the rounding to bf16 where that is the result's type (1.7e-3); the same call gives
 * the same bits.
 * Matrices of more than 64 rows and columns: X is held as a sum of two fp16 values (22 bits)
 * under a power of two, X X^T and the polynomial of it as fp16 with their diagonals in
 * fp32; products are of fp16 values with fp32 sums, and the linear term a X keeps all 22
 * bits, so that small singular values, which a step multiplies by a, are not drowned in rounding.  With the default
 * coefficients 3e-4 to 1e-3 after up to five steps where the singular values are of one order, and at most, on any spectrum,
 * 1e-3 after one or two steps, 1.5e-3 after three, 3.5e-3 after five, 5e-3 after seven and 8e-3 after eight (bounds from the
 * roundings' model, held by tests on 65 to 768 rows).  Where singular values are missing, each step multiplies by a what
 * rounding put in their place: 2.5e-2 after nine steps, 3.4 times that with each step more, until from 12 steps on the result
 * holds directions that are rounding's (binary32 throughout comes there with 12 as well).  Elements of X below 2^-49, as
 * of a matrix whose norm is far below eps, count as zero.
 * Matrices of at most 64 rows or columns: everything between U and the result is binary64, and the result is rounded once
 * to binary32: 7e-7 up to seven steps on any spectrum.  Of more steps X is rounded to binary32 once or twice on the way,
 * which each step after that multiplies by a where singular values are missing: 1.3e-5 after eight steps, 2.3e-4 after
 * twelve, 3.3e-2 after sixteen.
 * A matrix with an inf or NaN element has NaN in every element of its result, a zero matrix
 * zeros.  No matrix changes another's result: its bits are the same alone, in any list and with any workspace.
 *
 * Requirements: a, b, c finite, eps finite and >= 0, 1 <= steps <= ADAMW_NS_MAX_STEPS;
 * coefficients under which a singular value of [0, 1] passes 64 on the way are refused. */
enum { ADAMW_NS_MAX_STEPS = 16 };
typedef struct {
    float a;
    float b;
    float c;
    float eps;
    int32_t steps;
} adamw_newton_schulz;

/* Bytes of device workspace with which the two calls below work through `list` (its
 * numel, shard and ADAMW_FLAT_PAD8; pointers are not looked at) at full speed: room for
 * all its matrices, or of a longer list for 4 GiB of them at a time.  With `least` != 0, the smallest workspace that they
 * take: room for the largest matrix.  -1 on an invalid argument.  No GPU work, no HIP call.
 * A matrix of n elements with sides s <= l, both rounded up to multiples of 64, takes
 *     8 s + 4 s l + max(2 s l + 4 s^2, 4 n)
 * bytes, and 8 for every run of 4,096 elements or more (at most 256 runs), each part rounded up to 256 bytes.  That is 10
 * bytes an element of a large square matrix and 8 of a long one, but far more of one whose shorter side is
 * much less than 64, which counts as 64: 24.6 of 16 x 2048, 384 of a vector. */
int64_t adamw_orthogonalize_workspace_bytes(const adamw_tensor_list* list, const int64_t* cols, int least);

/* Orthogonalises every matrix of a list: stream 0 (bf16, written) = the result of the
 * Newton-Schulz products of stream 1 (u_dtype: ADAMW_F32, ADAMW_BF16 or ADAMW_F16; read
 * only), for optimizers with a rule of their own.  A bf16 matrix may be its own
 * result (equal addresses); any other overlap of a result with a matrix, a result or the
 * workspace is refused.
 * workspace: device memory of the caller, 256-byte aligned, of at least
 * adamw_orthogonalize_workspace_bytes(list, cols, 1) bytes; its contents need not be kept between
 * calls and are not read before they are written.  Calls that may overlap in time,
 * replays of captured ones among them, need a workspace each.
 * Execution, graphs and errors as adamw_multi_tensor_step. */
adamw_status adamw_orthogonalize(adamw_dtype u_dtype, const adamw_tensor_list* list, const int64_t* cols,
                                 const adamw_newton_schulz* ns, void* workspace, int64_t workspace_bytes,
                                 void* hip_stream);

/* The factor s of a Muon step's update of an R x C matrix. */
enum {
    ADAMW_MUON_SCALE_NONE = 0,      /* 1 */
    ADAMW_MUON_SCALE_SPECTRAL = 1,  /* sqrt(max(1, R / C)) */
    ADAMW_MUON_SCALE_RMS = 2        /* 0.2 sqrt(max(R, C)): the usual root mean square of an AdamW update, so
                                       that learning rate and weight decay may be those of the AdamW step */
};

/* Hyper-parameters of a Muon step.  Requirements: all finite; lr, weight_decay >= 0;
 * 0 <= momentum < 1; inv_loss_scale > 0; nesterov 0 or 1; scaling as above. */
typedef struct {
    float lr;
    float momentum;
    float weight_decay;
    float inv_loss_scale;
    int32_t nesterov;
    int32_t scaling;
    adamw_newton_schulz ns;
} adamw_muon_hparams;

/* One Muon step over a list of matrices, for the hidden layers' weights beside an AdamW
 * step over everything else (embeddings, vectors).  Momentum, orthogonalised,
 * with decoupled weight decay:
 *
 *   g = grad * mult
 *   m = momentum*m + (1-momentum)*g
 *   u = momentum*m + (1-momentum)*g if nesterov, else m
 *   O = the Newton-Schulz products of u (above)
 *   ADAMW_MIXED:       w = w*(1 - lr*wd) - (lr*s)*O;  param = round16(w)
 *   ADAMW_MIXED_SPLIT: the same on the split master
 *   ADAMW_PURE_KAHAN, or with prec non-null the pure-bf16 step of *prec (mode and p_dtype
 *                      ignored; its exp_avg_sq is not used): d = -(lr*wd)*p - (lr*s)*O;
 *                      s' = c + d;  p' = round_bf16(p + s');  c = s' - (p' - p) rounded to its
 *                      dtype; without compensation p = round_bf16(p*(1 - lr*wd) - (lr*s)*O)
 *
 * Streams, dtypes and roundings as in the AdamW step of the same mode; exp_avg is m (bf16
 * m is widened, updated and used in fp32 and stored rounded), stream 3 (exp_avg_sq) is
 * not used.  Each line but O's is in binary32, as written, without fused multiply-add; lr*s, lr*wd and
 * 1 - lr*wd are formed in binary64 and rounded once.  O is used as the fp32 sum it is, without a 16-bit rounding.
 * mult is the inverse loss scale, hp->inv_loss_scale or with d_scale non-null
 * (float)(1 / (double)d_scale->scale) read on the device, and with clip non-null
 * round_f32(that * f), f the clipping factor of adamw_multi_tensor_step_clipped.  *d_scale is
 * never advanced here: the AdamW call of the same iteration does that, and comes last.  The step is skipped, and nothing written,
 * if *d_found_inf (nullable) is set or *clip->d_sumsq is not finite; else the counter
 * *d_step advances as in adamw_multi_tensor_step.  The buffers of the list may not overlap each other
 * or the workspace, which is that of adamw_orthogonalize.  Execution, graphs and
 * errors as adamw_multi_tensor_step. */
adamw_status adamw_muon_multi_tensor_step(adamw_mode mode, adamw_dtype p_dtype, const adamw_pure_precision* prec,
                                          const adamw_tensor_list* list, const int64_t* cols,
                                          const adamw_muon_hparams* hp, const adamw_grad_clip* clip, int32_t* d_step,
                                          const int32_t* d_found_inf, const adamw_loss_scale_state* d_scale,
                                          void* workspace, int64_t workspace_bytes, void* hip_stream);

/* Description of the last error on the calling thread ("" if none).  Valid
 * until the next call into the library on that thread. */
const char* adamw_last_error(void);

/* Frees every workspace the library holds (all devices and streams) and
 * releases the allocation-free entry point's table on every GPU (its static
 * array stays).  The caller must make sure no enqueued step is still running,
 * no graph holding a captured step will be replayed again, and no other
 * thread is inside a library call. */
void adamw_release_workspace(void);

/* ADAMW_ABI_VERSION of the built library. */
int adamw_abi_version(void);

/* Optimizer-owned state in the blocked layout (ADAMW_BLOCKED_STATE), set up and
 * read back from ordinary per-tensor (or flat) state buffers: the layout of the
 * fastest steps made easy to adopt, and a blocked state checkpointed in the
 * usual per-tensor form.  Layout only, no arithmetic.
 *
 * `list` describes the per-tensor state as a step of (mode, p_dtype) -- or,
 * with prec non-null, of adamw_pure_multi_tensor_step with *prec -- would see
 * it WITHOUT ADAMW_BLOCKED_STATE: numel, the shard range, ptr[2..4] and
 * flat_mask bits 2-4 for exp_avg, exp_avg_sq and aux, and ADAMW_FLAT_PAD8,
 * which selects the flat index the blocked buffer is laid out in.  ptr[0] and
 * ptr[1] (param, grad) are not used.  The blocked buffer then serves the step
 * whose list has the same numel, shard and ADAMW_FLAT_PAD8 choice,
 * ADAMW_BLOCKED_STATE set and ptr[2][0] = the buffer.
 *
 * adamw_blocked_state_bytes: the size in bytes of that blocked buffer (whole
 * blocks of ADAMW_STATE_BLOCK_ELEMS elements), or -1 on an invalid argument.
 * No GPU work, no HIP call.
 *
 * adamw_blocked_state_copy: copies every element of the shard's state between
 * the per-tensor buffers and `blocked` (device memory, 16-byte aligned,
 * adamw_blocked_state_bytes long): to_blocked != 0 fills the blocked buffer
 * from the per-tensor buffers, 0 the reverse.  The blocked buffer's padding
 * (the ends of the last block and, with ADAMW_FLAT_PAD8, the gaps between
 * tensors) is neither read nor written.  The copy runs on hip_stream, after
 * the work already queued there, and the call returns once it is done (it
 * allocates and frees a small device table: a setup and checkpoint routine,
 * not for the training loop; on a stream under graph capture it is refused
 * with ADAMW_E_INVALID). */
int64_t adamw_blocked_state_bytes(adamw_mode mode, adamw_dtype p_dtype, const adamw_pure_precision* prec,
                                  const adamw_tensor_list* list);
adamw_status adamw_blocked_state_copy(adamw_mode mode, adamw_dtype p_dtype, const adamw_pure_precision* prec,
                                      const adamw_tensor_list* list, void* blocked, int to_blocked, void* hip_stream);

/* Planner introspection, for tests: no GPU work, no HIP call.  Builds the
 * chunk plan of adamw_multi_tensor_step (for_check = 0),
 * adamw_check_finite (for_check = 1), adamw_grad_norm and adamw_tensor_norms
 * (for_check = 2), or adamw_clip_grads (3; both with g_dtype = p_dtype, mode ignored),
 * and writes up to cap rows of 6 int64 each to out (a step's workgroups take items made
 * of these chunks, see adamw_plan_inspect_bytes; the other calls' take the chunks):
 *   {tensor index, element offset inside the tensor, element count,
 *    kind (0 = element-wise, 1 = 16-byte vector, 2 = any elements, whose 16-byte
 *    words the workgroup finds), flat position, segment}.
 * Returns the number of chunks (which may exceed cap), or -1 on an invalid
 * argument (see adamw_last_error). */
int64_t adamw_plan_inspect(adamw_mode mode, adamw_dtype p_dtype, const adamw_tensor_list* list, int for_check,
                           int64_t* out, int64_t cap);

/* Planner introspection, for tests: no GPU work, no HIP call.  The device
 * bytes each chunk of the plan covers: for the step of (mode, p_dtype), or with
 * prec non-null the step of adamw_pure_multi_tensor_step with *prec (mode and
 * p_dtype ignored), or with for_check the pass over the gradients of
 * adamw_plan_inspect's for_check (g_dtype = p_dtype), writes up to cap rows of 16 uint64 to out:
 *   {the 6 fields of an adamw_plan_inspect row, lo[0], hi[0], ..., lo[4], hi[4]}
 * With for_check = 4 (this call only) a row is an item of the step's launch table, in the
 * table's order: one or several neighbouring chunks, its kind 256 * the workgroups that
 * share it + 16 * the elements before its vector part + 1, or 256 * the workgroups for an
 * item without a vector part.
 * [lo[s], hi[s]) is the address range of stream s that the chunk's (item's)
 * workgroups read and write (lo = hi = 0 for a stream the launch does not
 * touch; a blocked state buffer shows as streams 2-4 at their places inside
 * the blocks).  Returns the number of chunks, or -1 on an invalid argument. */
int64_t adamw_plan_inspect_bytes(adamw_mode mode, adamw_dtype p_dtype, const adamw_pure_precision* prec,
                                 const adamw_tensor_list* list, int for_check, uint64_t* out, int64_t cap);

/* Launch form.  A step whose grid has at most max_workgroups workgroups
 * (default 4096: 512 chunks of 16384 elements, about 8.4e6 elements, or 4096 tensors
 * of at most 4096 elements) runs as
 * ONE kernel launch: every workgroup reads *d_found_inf, *d_step and the loss
 * scale itself, forms the step's scalars (the same binary64 formulas, so the
 * same bits), and the last workgroup to finish stores t into *d_step and
 * advances the loss scale.  Larger plans and empty lists run a one-lane
 * prologue kernel first.  Likewise adamw_check_finite over a grid of at most
 * max_workgroups (one per check chunk) is one launch whose last workgroup
 * stores the flag, instead of a zeroing kernel and the check.  The results are
 * bit-identical either way; the single launch saves a kernel launch and its
 * dependency, which dominate steps of a few million elements.  A chunk
 * of an update plan takes 8 workgroups, one of at most 4096 elements (element-wise:
 * 512) one; the element-wise ends of a tensor go with its vector chunks.  (A plan of at
 * most 128 chunks -- 64 in ADAMW_MIXED and with fp32 moments and compensation -- takes 8
 * for every chunk.)  max_workgroups: 0 = always two
 * launches, < 0 = restore the default.  Affects later calls on every stream.
 * Returns the value now in force. */
int64_t adamw_set_single_launch_max_workgroups(int64_t max_workgroups);

/* Tuning knob: elements per vector chunk, a multiple of 2048 in [2048, 1<<22],
 * for every kernel (an update chunk of more than 4096 is shared by 8 workgroups,
 * one per XCD, each lane taking 8 elements per 16384; a check chunk, or a norm's, is
 * one workgroup's; a clipping chunk of more than 16 KiB is shared by 8); 0 restores
 * the built-in defaults (16384 for the update kernels and the check, 32 KiB for the
 * norms, 128 KiB for clipping).  Affects plans built after the call.  Returns the value now
 * in force (0 = defaults), or -1 if rejected. */
int64_t adamw_set_chunk_elems(int64_t elems);

#ifdef __cplusplus
}
#endif

#endif /* ADAMW_H */
