// layout.hpp -- device-side launch metadata shared by the host planner and the
// gfx950 kernels of the fused AdamW step.
//
// A launch processes a list of segments (a tensor, or the part of a tensor that
// falls inside a ZeRO shard).  Each segment is split into chunks, which one or
// several workgroups process.  Chunks of the "vector" kind hold a multiple
// of 8 elements whose addresses in every stream are 16-byte aligned, so every
// lane moves whole dwordx4 words; the other kind ("element") covers peeled
// heads and tails and segments whose streams cannot be aligned together.
#pragma once

#include <stdint.h>

#include "adamw.h"

namespace adamw {

constexpr int kStreams = 5;            // param, grad, exp_avg, exp_avg_sq, aux
// Threads per workgroup, per kernel family, with the occupancy caps in
// kernels.hip: the mixed kernels run 256-lane workgroups, two per CU (8 waves);
// the VALU-heavier pure-bf16 family 256-lane workgroups, four per CU (16 waves);
// the overflow check 256-lane workgroups at full occupancy (it only reads).
// Chosen by interleaved A/B runs on MI355X (OPT-1.3B list, state in the blocked
// layout and per tensor): for the pure family 256 x 4 and 512 x 2 beat 1024 x 1
// by 5% on blocked state and tie with it per tensor; for the mixed family
// 256 x 2 leads every other shape tried, by 0-10% on blocked state.  The chunk
// and tile shapes below assume these sizes.
#ifndef ADAMW_BLOCK_MIXED
#define ADAMW_BLOCK_MIXED 256
#endif
#ifndef ADAMW_BLOCK_PURE
#define ADAMW_BLOCK_PURE 256
#endif
constexpr int kBlockMixed = ADAMW_BLOCK_MIXED;
constexpr int kBlockPure = ADAMW_BLOCK_PURE;
constexpr int kBlockCheck = 256;
constexpr int kPack = 8;               // elements per lane per dwordx4 of a 16-bit stream
constexpr uint32_t kVecBit = 0x80000000u;
constexpr uint32_t kCountMask = 0x7fffffffu;
constexpr int64_t kTagCheck = -1;      // plan tags: an update kernel's id, the overflow check,
constexpr int64_t kTagNorm = -2;       // or a gradient sweep: sum of squares, clipping
constexpr int64_t kTagClip = -3;
constexpr int64_t kElemChunkElems = 4096;       // element chunk
// An update kernel's chunk is shared by kXcdParts workgroups, consecutive in
// launch order, so one on each XCD (the dispatcher hands workgroup b to XCD
// b % 8).  The chunk is cut into tiles of 64 units, a unit being what one lane
// moves of every stream in one access: 8 elements where all streams are 16-bit, 4
// where one is fp32.  A tile is one access of a wave (1 KiB of its widest stream);
// tile t goes to part t % 8, so that all XCDs sweep one contiguous region together.
// On MI355X (OPT-1.3B list, against giving each XCD one contiguous run of
// 2048-element chunks) the sharing streamed the mixed step 7 % faster on blocked
// state (16384-element blocks) and 4-6.5 % per tensor, and the Kahan step 1 %
// faster blocked and 5-9 % per tensor.  Units of 4 elements, against 8 elements
// whose fp32 words lie 32 bytes apart from lane to lane (each wave access then
// touches every 128-byte line of twice its length for half of its bytes, and
// non-temporal loads fetch the lines twice): with non-temporal loads the mixed
// step gained 1-1.5 points of peak, up to 4.6 per tensor on other placements, and
// 14 % at 1 M elements; the steps with fp32 moments 3-8 points per tensor and 0-5
// blocked.  Tiles of 32 units were 1-4 points slower, tiles of 128 units 1-3.
constexpr int kXcdParts = 8;
constexpr int kTilePacksMixed = 64;   // units of a tile where a stream is fp32 (256 elements)
constexpr int kTilePacks = 64;        // where all streams are 16-bit (512 elements)
// The unit of a chunk taken by lane tid of part `part` (per kXcdParts * block
// units): tile t of p units belongs to part t % kXcdParts, so
//     ((tid / p) * kXcdParts + part) * p + tid % p,
// a bijection of (part, tid) onto [0, kXcdParts * block) whenever p divides
// the workgroup size.  (parts = 1: a chunk that one workgroup takes alone.)
constexpr uint32_t tile_pack(uint32_t tid, uint32_t part, uint32_t p, uint32_t parts = kXcdParts)
{
    return ((tid / p) * parts + part) * p + tid % p;
}
// Default vector chunk of an update kernel: 8 elements per lane of each part.
constexpr int64_t update_chunk_elems(int block) { return (int64_t)kXcdParts * block * kPack; }
// Blocked state: elements per block, one update chunk (every mode).
constexpr int64_t kStateBlockElems = ADAMW_STATE_BLOCK_ELEMS;
static_assert(kStateBlockElems % update_chunk_elems(kBlockMixed) == 0 &&
                  kStateBlockElems % update_chunk_elems(kBlockPure) == 0,
              "a state block holds whole default chunks");
// The overflow check moves 2 B per element (the step 18-28 B): one workgroup
// per chunk, each lane reading this many packs in one pass, so that a
// workgroup's fixed cost (two dependent table loads) is spread over as many
// bytes as a step workgroup moves.
#ifndef ADAMW_CHECK_CHUNK_MULT
#define ADAMW_CHECK_CHUNK_MULT 8
#endif
constexpr int kCheckChunkMult = ADAMW_CHECK_CHUNK_MULT;
constexpr int64_t kCheckChunkElems = (int64_t)kBlockCheck * kPack * kCheckChunkMult;
// A launch's grid counts at most 2^32 - 1 lanes: the chunk limit of a plan
// follows from the lanes one chunk takes (kXcdParts workgroups of an update
// kernel, one check workgroup).
constexpr int kMaxUpdateBlock = kBlockMixed > kBlockPure ? kBlockMixed : kBlockPure;
constexpr int64_t kMaxUpdateChunks = (int64_t)UINT32_MAX / ((int64_t)kXcdParts * kMaxUpdateBlock);
constexpr int64_t kMaxCheckChunks = (int64_t)UINT32_MAX / kBlockCheck;
// The gradient sweeps (sum of squares, clipping) touch the gradient stream alone.
// A sweep's chunks are not cut at 16-byte edges: the workgroup takes the elements
// before the first edge and after the last one by themselves, so a tensor costs one
// workgroup however short or misaligned it is.
//   sum of squares: one workgroup per chunk of 32 KiB, 8 16-byte words per lane;
//   clipping: chunks of 128 KiB shared by 8 consecutive workgroups as in an update
//     kernel, in tiles of 64 words (1 KiB), 4 words per lane; a chunk of at most 16 KiB
//     is one workgroup's.
constexpr int kBlockSweep = 256;
constexpr int kNormUnroll = 8;
constexpr int kClipUnroll = 4;
constexpr int kTileWords = 64;
constexpr int64_t kNormChunkBytes = (int64_t)kBlockSweep * 16 * kNormUnroll;
constexpr int64_t kClipWholeBytes = (int64_t)kBlockSweep * 16 * kClipUnroll;
constexpr int64_t kClipChunkBytes = kXcdParts * kClipWholeBytes;
constexpr int64_t kMaxSweepChunks = (int64_t)UINT32_MAX / kBlockSweep;
// A sum of squares runs as one launch (its last workgroup joins the partial sums) up
// to this many workgroups, if the single-launch limit allows as many: past it the
// counting atomics cost more than a launch.  MI355X, one launch / two, in graphs of 30
// norms of one bf16 tensor: 4.0 / 4.25 us at 16 workgroups, 5.6 / 5.9 at 512, 8.4 / 8.6 at
// 1,024 (33.6 MB), 11.3 / 11.05 at 1,536, 14.3 / 13.9 at 2,048, 25.4 / 24.1 at 4,096; fp32 the
// same within 0.3 us up to 2,048, 26.4 / 24.6 at 4,096.
constexpr int64_t kSingleSumMaxWorkgroups = 1024;
// Partial sums are joined by 256-lane workgroups, this many each.
constexpr int kBlockJoin = 256;
constexpr int kJoin = 4096;
// The state copy (setup and checkpoint) runs one 256-lane workgroup per chunk.
constexpr int kBlockCopy = 256;
constexpr int64_t kMaxCopyChunks = (int64_t)UINT32_MAX / kBlockCopy;

// Clipping by the global norm: the factor min(1, max_norm / (sqrt(*sumsq) * inv + eps))
// with inv the gradients' inverse loss scale (sumsq null: no clipping).
struct ClipRule {
    const double* sumsq;
    float max_norm;
    float eps;
};

// What a sum of squares leaves in device memory (null: not wanted).
struct NormOut {
    double* sumsq;          // the list's sum of squares (accumulate: added to what is there)
    float* norm;            // its square root
    int32_t* found_inf;     // 1 if the sum is not finite, else 0
    int32_t accumulate;
    float* tensor_norm;     // per tensor of the list
    double* tensor_sumsq;
};

// Workgroup b of a grid of nb -> the chunk it processes.  The dispatcher hands
// workgroup b to XCD b % 8 (the MI355X has 8 XCDs, each with its own L2); this
// map lets XCD x walk one contiguous run of chunks, so the workgroups in flight
// on an XCD stream neighbouring addresses.  XCD x receives the q + (x < r)
// workgroups b = 8j + x < nb (q = nb / 8, r = nb % 8) and owns as many chunks,
// starting at x*q + min(x, r): a bijection on [0, nb) for every nb.  Plain
// constexpr code, so that the kernels and a host-side test share it.
constexpr uint32_t xcd_chunk(uint32_t b, uint32_t nb)
{
    return (b & 7u) * (nb >> 3) + ((b & 7u) < (nb & 7u) ? (b & 7u) : (nb & 7u)) + (b >> 3);
}

// Update kernels, by launch id.  The pure-bf16 family adds
// 4 * (fp32 exp_avg) + 2 * (fp32 exp_avg_sq) + (bf16 Kahan compensation) to
// kKernelPure; with an fp32 compensation buffer, 2 * (fp32 exp_avg) + (fp32
// exp_avg_sq) to kKernelPureC32.
constexpr int kKernelMixedBf16 = 0;
constexpr int kKernelMixedF16 = 1;
constexpr int kKernelSplit = 3;
constexpr int kKernelPure = 4;
constexpr int kKernelKahan = kKernelPure + 1;   // bf16 moments + compensation
constexpr int kKernelPureC32 = kKernelPure + 8;

// Occupancy cap, per kernel: the update kernels use no LDS, but reserving this much
// per workgroup leaves room for only 160 KiB / bytes workgroups on a CU: fewer
// concurrent address streams keep more DRAM rows open.  Two 256-lane workgroups (8
// waves) for the mixed step and for fp32 moments beside an fp32 compensation buffer
// (28 and 30 B per element), four for the others.  MI355X, OPT-1.3B list, % of peak
// with two / four, state per tensor, then blocked: mixed 78.3 / 77.1, 84.2 / 82.0;
// fp32 moments and compensation 78.5 / 73.9, 81.3 / 80.2; split master 75.6 / 75.5,
// 76.2 / 77.7; fp32 moments and bf16 compensation 76.0 / 75.5, 77.4 / 77.7; fp32
// moments alone 77.2 / 78.2, 74.3 / 82.4; bf16 state (Kahan) 73.5 / 76.9, 74.4 / 79.0.
#ifndef ADAMW_LDS_MIXED
#define ADAMW_LDS_MIXED 81920
#endif
#ifndef ADAMW_LDS_PURE
#define ADAMW_LDS_PURE 40960
#endif
#ifndef ADAMW_LDS_C32_WIDE
#define ADAMW_LDS_C32_WIDE 81920
#endif
constexpr int64_t update_lds(int kernel)
{
    return kernel == kKernelMixedBf16 || kernel == kKernelMixedF16 ? ADAMW_LDS_MIXED
         : kernel == kKernelPureC32 + 3 ? ADAMW_LDS_C32_WIDE : ADAMW_LDS_PURE;
}
// The workgroups of an update kernel that the card holds at once: 256 CUs of 160 KiB.
constexpr int64_t resident_workgroups(int kernel) { return 256 * (160 * 1024 / update_lds(kernel)); }

// One segment: the device address of its element 0 in each stream (0 for a
// stream the launch does not touch).
struct alignas(64) DevSeg {
    uint64_t ptr[kStreams];
    uint64_t pad[3];
};

// One chunk of a plan: elements [off, off + count) of segment `seg`; kVecBit in n_kind
// marks the vector kind.  The overflow check's kernel takes the chunks as they are, one
// workgroup each; the update kernels take items made of them (below).
struct alignas(16) DevChunk {
    uint32_t seg;
    uint32_t n_kind;
    uint64_t off;
};

// One item of an update's table, made from the chunks of a plan: elements
// [off, off + count) of segment `seg`, a vector chunk with the element chunks before
// and after it (up to 7 elements each), or an element chunk (kVecBit clear).  Bits of
// n_kind: kVecBit, the elements before the vector part at kItemHeadShift, the count.
// The first n_shared items are taken by kXcdParts workgroups each, the others, of at
// most kSingleVecElems or kSingleElems elements, by one: 8 workgroups for every chunk
// made short tensors a matter of launching workgroups.  MI355X, clipped fp16 mixed
// step, 4,000 tensors of log-uniform length packed tightly: 190 -> 38 us at up to
// 4,000 elements (1.9 M in all), 565 -> 453 us at up to 2^18 (82.6 M), 492 -> 388
// where every tensor starts aligned; 40 us and 397 with at most 2048 elements alone,
// 37.5 and 385 with 8192.
constexpr int kItemHeadShift = 28;
constexpr uint32_t kItemCountMask = (1u << kItemHeadShift) - 1;
#ifndef ADAMW_SINGLE_VEC_ELEMS
#define ADAMW_SINGLE_VEC_ELEMS 4096
#endif
constexpr uint32_t kSingleVecElems = ADAMW_SINGLE_VEC_ELEMS;
constexpr uint32_t kSingleElems = 512;
// A list whose chunks fit on the card all at once with 8 workgroups each
// (resident_workgroups) is taken as planned instead, every chunk shared: such a step is
// one latency, and a chunk of 4,096 elements that one workgroup takes alone is two passes of
// it.  Graph replays of mixed steps, shared / alone: one tensor of 4,096 elements 5.0 /
// 5.8 us, 64 of them 5.7 / 6.5; beyond, 128 of them 9.0 / 6.7 (Kahan, four workgroups per
// CU: 128 5.9 / 6.8, 256 9.8 / 7.2).
struct UpdateGrid {
    int64_t n_shared = 0, n_single = 0;
    int64_t workgroups() const { return n_shared * kXcdParts + n_single; }
};

// The item and part of workgroup b of an update grid.  The items of one workgroup come
// first: at the end of the grid their latency showed (Kahan step, OPT-125m 1-2 %, BERT 1 %).
// The 8 workgroups of a shared item follow one another, in the order that puts part p on
// XCD p.
struct ItemPart {
    uint32_t item, part, parts;
};
constexpr ItemPart update_item(uint32_t b, uint32_t n_shared, uint32_t n_single)
{
    return b < n_single ? ItemPart{n_shared + b, 0, 1} : ItemPart{(b - n_single) / kXcdParts, b % kXcdParts, kXcdParts};
}

// What a workgroup of an update kernel does of its item: `part` of `parts`, of the
// `body` elements from `head` on in units, and of the `edge` elements before and after
// them one by one.
struct Work {
    uint64_t off;      // the item's first element in its segment
    uint32_t seg, part, parts;
    uint32_t head, body, edge;
};
constexpr Work item_work(const DevChunk& it, const ItemPart& ip)
{
    const uint32_t n = it.n_kind & kItemCountMask;
    const bool vec = (it.n_kind & kVecBit) != 0;
    const uint32_t head = vec ? it.n_kind >> kItemHeadShift & 7u : n;
    const uint32_t body = vec ? (n - head) / kPack * kPack : 0;
    return Work{it.off, it.seg, ip.part, ip.parts, head, body, n - body};
}

// Per parts * BLOCK * N units of an item, wave w of a workgroup takes tiles w * N + h
// (h < N) of its part, a lane one unit of each: access h of lane tid is
// unit_at(tid, work, h), and every access of a wave is one contiguous stretch of
// its stream.
template <int P, int N>
constexpr uint32_t unit_at(uint32_t tid, const Work& w, int h)
{
    static_assert(P == 64, "a tile is one access of a wave");
    return tile_pack((tid / P * N + (uint32_t)h) * P + tid % P, w.part, P, w.parts);
}

// The k-th of the elements outside the vector part.
constexpr uint32_t edge_at(const Work& w, uint32_t k) { return k < w.head ? k : k + w.body; }

// One workgroup's work in a gradient sweep: n elements from address addr, shared by
// kXcdParts workgroups of which this is number `part`, or its own (kWholeChunk).
constexpr uint32_t kWholeChunk = UINT32_MAX;
struct alignas(16) DevSweep {
    uint64_t addr;
    uint32_t n;
    uint32_t part;
};

// One piece of a state copy between the blocked buffer and per-tensor (or flat)
// state buffers: the address of the piece's first element on each side, per
// state stream (exp_avg, exp_avg_sq, aux; 0 for a stream the step does not use).
struct alignas(64) DevCopySeg {
    uint64_t tensor_side[3];
    uint64_t blocked_side[3];
    uint64_t pad[2];
};

// Scalars of one step, written by the prologue kernel and read by the update
// kernel on the same stream.
struct alignas(64) LaunchScalars {
    int32_t skip;        // nonzero: the step is not taken, nothing is written
    int32_t t;           // 1-based index of the step taken
    float step_size;     // lr / (1 - beta1^t)
    float rbc2;          // 1 / (1 - beta2^t)
    float decay;         // 1 - lr*wd
    float lrwd;          // lr*wd
    float omb1;          // 1 - beta1 (fp32)
    float omb2;          // 1 - beta2 (fp32)
    float beta1;
    float beta2;
    float eps;
    float inv_scale;
};

constexpr int64_t kScalarsBytes = 256;
// Counts of finished workgroups of a single-launch step, after the scalars in
// the same workspace block: kDoneLanes first-level counters (workgroup b counts
// in lane b % kDoneLanes) and one second-level counter, each in its own
// 256-byte line so that their atomics do not queue on one address.  All are
// zero between launches.
constexpr int kDoneLanes = 32;
constexpr int64_t kDoneStrideWords = 64;
constexpr int64_t kDoneOffset = kScalarsBytes;
constexpr int64_t kDoneWords = (kDoneLanes + 1) * kDoneStrideWords;
constexpr int64_t kWorkspaceBytes = kDoneOffset + kDoneWords * 4;

// Default largest grid, in workgroups, that runs as a single launch.  Measured
// on MI355X (mixed step, one tensor, pipelined steps): the single launch takes
// 28-32 % off a step of 64k-256k elements, 7 % at 1M and 2 % at 4M, and ties
// from 8M (4096 workgroups) up, where the prologue launch no longer shows.
constexpr int64_t kSingleLaunchMaxWorkgroups = 4096;

// A single-launch step: the update kernel forms the step's scalars itself in
// every workgroup, and the last workgroup to finish stores the advanced counter.
struct FusedStep {
    adamw_hparams hp;
    int32_t* step;              // the caller's step counter
    const int32_t* found_inf;   // nullable skip flag
    uint32_t* done;             // the finished-workgroup counters (kDoneLanes + 1 lines)
    adamw_loss_scale_state* amp;   // nullable: the device-resident dynamic loss scale
    adamw_loss_scaler scaler;      // its rule (with amp)
    ClipRule clip;                 // its sumsq null: no clipping
};

}  // namespace adamw
