// muon.hpp -- the Newton-Schulz products and the Muon step over a list of matrices:
// what the host planner (muon_plan.cpp, no HIP calls) lays out and the gfx950 kernels
// (muon.hip) work through.
//
// A list is worked through in batches of matrices that fit the caller's workspace
// together.  One batch is a fixed sequence of launches, each over every matrix of it:
//
//   moments    sum of squares of each matrix; a step also advances m and writes u
//   normalise  X = u / (|u| + eps) as fp16 pairs
//   per product step:  gram  A = X X^T (the shorter side),  poly  B = b A + c A A,
//                      apply X = a X + B X, the last one with the result's own epilogue
//
// Matrices whose shorter side is at most kPad go in batches of their own: all steps go on in one workgroup, on
// polynomials of the first Gram matrix, and X is read twice instead:
//
//   moments      as above
//   small gram   partial sums of U U^T for runs of columns, in binary64
//   small chain  A = U U^T / (|U| + eps)^2, and Q, the product of every step's a I + b A + c A A
//   small apply  Q X with the result's own epilogue
//
// (of more than NsScales::run steps, run by run, with X in fp32 between them).
//
// The matrices of the products are held in the workspace with both sides padded to
// kPad by zeros, so that the product kernels have no ragged edge in the summed dimension.
#pragma once

#include <stdint.h>

#include <memory>
#include <string>
#include <vector>

#include "adamw.h"
#include "layout.hpp"

namespace adamw {

constexpr int64_t kTagMuon = -4;          // plan tag
constexpr int kPad = 64;                  // padding of both sides, and elements of a summing step
constexpr int64_t kNsAlign = 256;         // of every part of the workspace
constexpr int64_t kNsHeadBytes = 256;     // the step's scalars, at the workspace's start
constexpr int64_t kNsBatchBytes = INT64_C(4) << 30;   // workspace of a batch of a long list
// Elements of a workgroup of the moments kernel: a multiple of this, so that a matrix has at
// most kMaxPartials partial sums, which every workgroup of the normalisation adds up.
constexpr int64_t kMomentElems = 4096, kMaxPartials = 256;
constexpr int kBlockMoments = 256;
// Columns of X of a workgroup of small gram, a multiple of kPad, so that a matrix has at most kMaxSmallRuns partial Gram
// matrices: 32 of them, which chain adds up quickly, until a run has 2,048 columns, and then more, since one
// CU multiplies in binary64 no faster than 64 x 64 x 2,048 in 35 us. A partial Gram matrix is its lower triangle in
// binary64, row after row (kSmallTri elements). They lie one after another from the matrix's base on, before u: runs of
// 128 columns or more leave 32 KiB for each.
constexpr int64_t kMaxSmallRuns = 256;
constexpr int64_t kSmallTri = (int64_t)kPad * (kPad + 1) / 2;
constexpr int64_t small_gram_cols(int64_t lp)
{
    int64_t each = (lp + 31) / 32;
    if (each > 2048) {
        each = (lp + kMaxSmallRuns - 1) / kMaxSmallRuns;
        if (each < 2048) each = 2048;
    }
    if (each < 2 * kPad) each = 2 * kPad;
    return (each + kPad - 1) / kPad * kPad;
}
constexpr int64_t small_apply_cols(int64_t lp) { return lp <= 4096 ? kPad : 4 * kPad; }

// Tiles of the product kernels: rows, columns, and lanes of a workgroup.
constexpr int kTileKinds = 3;
constexpr int kTileRows[kTileKinds] = {256, 128, 64};
constexpr int kTileCols[kTileKinds] = {256, 128, 64};
constexpr int kTileLanes[kTileKinds] = {512, 256, 256};
// Of a symmetric product, the tiles that reach the diagonal or lie below it are computed;
// those wholly below it are written to the mirrored place too.
constexpr bool tile_needed(int kind, int64_t row, int64_t col)
{
    return col * kTileCols[kind] < (row + 1) * kTileRows[kind];
}
constexpr bool tile_mirrored(int kind, int64_t row, int64_t col)
{
    return (col + 1) * kTileCols[kind] <= row * kTileRows[kind];
}

// Gram matrices of more columns are summed in two levels, the first over kLongRun summing steps (an even number): of shorter
// ones the fp32 sums are off by at most 2^-11, of these by 2^-14 and 2^-25 for each run.
constexpr int64_t kLongSum = INT64_C(1) << 18;
constexpr uint32_t kLongRun = 512;

constexpr int64_t kMaxNsSide = INT64_C(1) << 30, kMaxNsShort = INT64_C(1) << 20;
// A grid counts at most 2^32 - 1 lanes.
constexpr int64_t kMaxNsTiles = (int64_t)UINT32_MAX / 512;

// One matrix's parts of the workspace, one after another from byte `base` of it, where X is sp x lp: X is held
// wide whatever the matrix is, s rows of l elements, s <= l, transposed for a matrix that is taller than wide, both
// padded by zeros.
// da, db: the diagonals of the squares A and B in fp32.  hi, lo: X is (hi + lo * 2^-11) * 2^-sx; hi has
// two buffers, since workgroups of the product with B write new values while others read the
// old.  a, b: the squares, sp x sp.  u, a step's fp32 matrix as it lies in the caller's
// buffers, has the room of hi(1), a and b.
struct NsParts {
    uint64_t base;
    uint32_t sp, lp;

    constexpr uint64_t whole() const { return (uint64_t)sp * lp * 2; }
    constexpr uint64_t square() const { return (uint64_t)sp * sp * 2; }
    constexpr uint64_t da() const { return base; }
    constexpr uint64_t db() const { return base + (uint64_t)sp * 4; }
    constexpr uint64_t lo() const { return base + (uint64_t)sp * 8; }
    constexpr uint64_t hi(int k) const { return lo() + whole() * (uint64_t)(1 + k); }
    constexpr uint64_t u() const { return hi(1); }
    constexpr uint64_t a() const { return hi(1) + whole(); }
    constexpr uint64_t b() const { return a() + square(); }
    constexpr uint64_t end() const { return b() + square(); }
};

// One matrix of a batch; its partial sums lie behind its parts.
struct alignas(16) DevMatrix {
    uint64_t ptr[4];          // element 0: result or param; u or grad; exp_avg; aux
    NsParts parts;
    uint64_t partials;        // offset in the workspace
    double factor;            // s of the step
    int32_t rows, cols;
    uint32_t tall;            // rows > cols
    uint32_t chunk, n_partials;
    uint32_t flat16;          // every stream's element 0 is 16-byte aligned
    uint32_t row16;           // and so is every row of 8 elements' multiples
    uint32_t pad;
};

// One workgroup's part of a matrix: a tile of the products (row and column of the tile),
// a 64 x 64 tile of the normalisation, or a run of elements (its number).  With the parts in
// it a product's first loads hang on one load of its own.
struct alignas(16) DevTile {
    NsParts parts;
    uint32_t mat, row, col, pad;
};

struct NsLaunch {
    int64_t first = 0, count = 0;   // workgroups, in the tile table
    int kind = 0;                   // tile kind of a product
};

struct NsBatch {
    bool small = false;
    bool long_sums = false;   // a matrix has more than kLongSum columns, and the squares' tiles are of kind 1 or 2
    // square: gram and poly.  Of a small batch, normalise: the runs of columns of small gram, square: the matrices
    // (small chain), apply: the runs of small apply
    NsLaunch moments, normalise, square, apply;
};

// The batches of one sort of matrices, small ones (at most kPad on the shorter side) or others; where a list has both,
// the small ones' are a plan beside the others'.  So a matrix's launches, and the bits of its result, depend on its shape
// alone, not on what else is in the list or how the workspace cuts it into batches.
struct NsPlan {
    std::vector<DevMatrix> mats;
    std::vector<DevTile> tiles;
    std::vector<NsBatch> batches;
    std::unique_ptr<NsPlan> small;

    void flatten();   // one plan of both, the small ones' batches last
};

// What the two entry points do at both ends of the products.
enum NsEnd {
    kEndOrtho = 0,
    kEndMixedBf16,
    kEndMixedF16,
    kEndSplit,
    kEndPure,
    kEndKahan,
    kEndKahan32,
    kNumEnds
};
struct NsKind {
    int esz[kStreams];
    int end;
    adamw_dtype in;        // of stream 1
    bool m16;              // exp_avg is bf16
};

// Powers of two under which X, A and B are held in fp16 (sx, sa, sb).  What small chain holds, a I + b A + c A A, that times A,
// and the product of a run's polynomials, would fit fp16 under sp, sz and sq; it is binary64 and needs no scale, but
// these say how far its values can reach.
struct NsScales {
    int sx, sa, sb;
    int sp, sz, sq;
    // Steps that small chain takes of one Gram matrix.  A rounding of 2^-53 in it grows by a^2 with every step where X has
    // no singular value, and nothing in the polynomials brings it back, as products with X do.  So the largest
    // a + b q + c q^2 of all of them but the last may multiply to 2^11, which takes it to 2^-31 (the usual coefficients:
    // 7 steps); after them X is formed, in fp32, and its Gram matrix anew.
    int run;
    // Last steps of the larger matrices in which B's diagonal takes part in the product with lo (muon.hip): as many as
    // multiply what that leaves in absent directions by at most 16 after it (the usual coefficients: 3).
    int lo_steps;
};

adamw_status check_ns(const adamw_newton_schulz* ns, NsScales* scales, std::string& err);
adamw_status check_muon_hparams(const adamw_muon_hparams* hp, NsScales* scales, std::string& err);

// Bytes for all matrices (at most kNsBatchBytes, or the largest one's), or with `least`
// the largest matrix's.
adamw_status ns_workspace_bytes(const adamw_tensor_list* list, const int64_t* cols, bool least, int64_t* bytes,
                                std::string& err);

// Validates the list and, with `out`, lays the work out for a workspace of
// `workspace_bytes` at address `workspace`.
adamw_status build_ns_plan(const NsKind& kind, const adamw_tensor_list* list, const int64_t* cols, int scaling,
                           uint64_t workspace, int64_t workspace_bytes, NsPlan* out, std::string& err);

// What the moments kernel leaves for the others at the start of the workspace.
struct NsScalars {
    int32_t skip;
};

}  // namespace adamw
