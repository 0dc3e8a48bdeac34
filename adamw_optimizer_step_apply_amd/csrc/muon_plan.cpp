// muon_plan.cpp -- host planner of the Newton-Schulz products (no HIP calls): shapes,
// overlaps, the batches that fit a workspace, and the tiles of each launch.
#include "muon.hpp"

#include <stdio.h>

#include <algorithm>
#include <cmath>

#include "plan.hpp"

namespace adamw {

namespace {

struct Shape {
    int64_t tensor, rows, cols;
};

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// The whole matrices inside the shard, in list order.
adamw_status shapes_of(const adamw_tensor_list* list, const int64_t* cols, std::vector<Shape>* out, std::string& err)
{
    char buf[200];
    adamw_status st = basic_list_check(list, err);
    if (st != ADAMW_OK) return st;
    if (list->flat_mask & ~(0x1fu | ADAMW_BLOCKED_STATE | ADAMW_FLAT_PAD8)) {
        err = "flat_mask has unknown bits";
        return ADAMW_E_INVALID;
    }
    if (list->flat_mask & ADAMW_BLOCKED_STATE) {
        err = "matrices with blocked state are not provided";
        return ADAMW_E_UNSUPPORTED;
    }
    const int64_t nt = list->n_tensors, align = (list->flat_mask & ADAMW_FLAT_PAD8) ? 8 : 1;
    if (nt > 0 && !cols) { err = "cols array is null"; return ADAMW_E_INVALID; }
    int64_t total = 0;
    for (int64_t i = 0; i < nt; ++i) {
        const int64_t n = list->numel[i];
        if (n < 0 || n > (INT64_C(1) << 56) || total > (INT64_C(1) << 56)) {
            snprintf(buf, sizeof buf, "numel[%lld] = %lld < 0 or too large", (long long)i, (long long)n);
            err = buf;
            return ADAMW_E_INVALID;
        }
        total += round_up(n, align);
    }
    const int64_t b = list->shard_begin, e = list->shard_end < 0 ? total : list->shard_end;
    if (list->shard_end < -1 || b < 0 || b > e || e > total) {
        snprintf(buf, sizeof buf, "shard range [%lld, %lld) outside [0, %lld]", (long long)b,
                 (long long)list->shard_end, (long long)total);
        err = buf;
        return ADAMW_E_INVALID;
    }
    int64_t base = 0;
    for (int64_t i = 0; i < nt; ++i) {
        const int64_t n = list->numel[i], c = cols[i];
        if (c < 1 || n % c != 0) {
            snprintf(buf, sizeof buf, "cols[%lld] = %lld does not divide numel %lld", (long long)i, (long long)c,
                     (long long)n);
            err = buf;
            return ADAMW_E_INVALID;
        }
        const int64_t lo = std::max(b, base), hi = std::min(e, base + n);
        if (lo < hi) {
            if (hi - lo != n) {
                snprintf(buf, sizeof buf, "matrix %lld lies in the shard in part: shards take whole matrices",
                         (long long)i);
                err = buf;
                return ADAMW_E_INVALID;
            }
            const Shape s{i, n / c, c};
            // 32-bit row numbers, and byte counts that stay far from 2^63; the normalisation's launch has the most
            // workgroups, one for 64 x 64 elements
            if (s.rows > kMaxNsSide || s.cols > kMaxNsSide || std::min(s.rows, s.cols) > kMaxNsShort ||
                round_up(s.rows, kPad) / kPad * (round_up(s.cols, kPad) / kPad) > kMaxNsTiles) {
                snprintf(buf, sizeof buf,
                         "matrix %lld of %lld x %lld is larger than 2^30 on a side, 2^20 on both or %lld tiles of 64 x 64",
                         (long long)i, (long long)s.rows, (long long)s.cols, (long long)kMaxNsTiles);
                err = buf;
                return ADAMW_E_INVALID;
            }
            out->push_back(s);
        }
        base += round_up(n, align);
    }
    return ADAMW_OK;
}

// Lays one matrix out from byte `at` of the workspace; returns the end.
int64_t place(const Shape& sh, int64_t at, DevMatrix* m)
{
    const int64_t n = sh.rows * sh.cols, s = std::min(sh.rows, sh.cols), l = std::max(sh.rows, sh.cols);
    m->rows = (int32_t)sh.rows;
    m->cols = (int32_t)sh.cols;
    m->tall = sh.rows > sh.cols;
    m->parts = NsParts{(uint64_t)at, (uint32_t)round_up(s, kPad), (uint32_t)round_up(l, kPad)};
    m->chunk = (uint32_t)round_up((n + kMaxPartials - 1) / kMaxPartials, kMomentElems);
    m->n_partials = (uint32_t)((n + m->chunk - 1) / m->chunk);
    const int64_t end = std::max((int64_t)m->parts.end(), (int64_t)m->parts.u() + round_up(4 * n, kNsAlign));
    m->partials = (uint64_t)end;
    return end + round_up(8 * (int64_t)m->n_partials, kNsAlign);
}

// Bytes of a matrix's part of the workspace, the same for both calls.
int64_t bytes_of(const Shape& s)
{
    DevMatrix m;
    return place(s, 0, &m);
}

// Workgroup order of a launch's tiles: those of the longest sums first, and runs of
// neighbouring tiles (which read the same rows) to one XCD, whose L2 they then share.
// Workgroup b runs on XCD b % 8.  Runs of n / 16 tiles against n / 64: Gram products of four of 768 x 2304
// 20.7 -> 18.2 us, products with X of four of 1024 x 1024 27.0 -> 23.4 us (MI355X).
void deal_tiles(const std::vector<DevTile>& in, std::vector<DevTile>* out)
{
    const size_t n = in.size(), run = std::min<size_t>(32, (n + 15) / 16);
    std::vector<std::vector<DevTile>> of(kXcdParts);
    for (size_t i = 0; i < n; ++i) of[i / run % kXcdParts].push_back(in[i]);
    for (size_t q = 0, left = n; left; ++q)
        for (auto& v : of)
            if (q < v.size()) {
                out->push_back(v[q]);
                --left;
            }
}

int64_t tiles_of(int64_t n, int side) { return (n + side - 1) / side; }

int64_t square_tiles(int64_t s, int kind)
{
    int64_t n = 0;
    for (int64_t y = 0; y < tiles_of(s, kTileRows[kind]); ++y)
        n += std::min(tiles_of(s, kTileCols[kind]), ((y + 1) * kTileRows[kind] - 1) / kTileCols[kind] + 1);
    return n;
}

// The tiles' costs in microseconds: a tile of K summed elements alone on a CU takes cost + K * per_k, as fitted to
// single launches on MI355X (K from 64 to 8192, 3 to 8192 tiles).  One launch takes about `start` and
// the larger of its longest tile and its tiles in rounds: of the largest kind one workgroup fits on a CU, of the middle
// one two, which take 1.8 times as long together, and the smallest one's overlap freely.  Measured with kinds 0 / 1 / 2,
// in us: Gram products of 768 x 768 27.6 / 13.9 / 6.6, of four of 768 x 2304 59.9 / 31.0 / 20.7, of four of
// 2048 x 8192 389 / 258 / 270; products with X of four of 768 x 2304 36.1 / 25.8 / 40.6, of 64 of 512 x 1024
// 75 / 80 / 137, of four of 2048 x 2048 86 / 100 / 189.
struct TileCost {
    double start, square, apply, per_k;
};
constexpr TileCost kTileCost[kTileKinds] = {{2.0, 10.0, 22.0, 0.0285}, {3.0, 4.0, 4.6, 0.0115}, {2.5, 2.0, 2.0, 0.0032}};
constexpr int64_t kCus = 256;

// A launch's cost with one kind of tile: `each` calls back with every matrix's tiles and summed elements.
template <typename Each>
double launch_cost(int kind, bool square, const Each& each)
{
    const TileCost& c = kTileCost[kind];
    double sum = 0.0, longest = 0.0;
    int64_t n = 0;
    each([&](int64_t tiles, int64_t k) {
        const double one = (square ? c.square : c.apply) + c.per_k * (double)k;
        sum += one * (double)tiles;
        longest = std::max(longest, one);
        n += tiles;
    });
    double rounds = (double)n / (double)kCus;   // of one tile a CU
    if (kind == 0) {
        rounds = std::ceil(rounds);
    } else if (kind == 1) {
        const int64_t two = n / (2 * kCus), rest = n - two * 2 * kCus;
        rounds = 1.8 * (double)two + (rest > kCus ? 1.8 : rest > 0 ? 1.0 : 0.0);
    }
    return c.start + std::max(longest, n ? sum / (double)n * rounds : 0.0);
}

template <typename Cost>
int cheapest(int first, const Cost& cost)
{
    int best = first;
    for (int kind = first + 1; kind < kTileKinds; ++kind)
        if (cost(kind) < cost(best)) best = kind;
    return best;
}

// Matrices of one sort: every batch by the launches for small ones, or by the others.
struct PlacedShape {
    Shape shape;
    uint64_t ptr[4];
};
constexpr int kStreamOf[4] = {ADAMW_STREAM_PARAM, ADAMW_STREAM_GRAD, ADAMW_STREAM_EXP_AVG, ADAMW_STREAM_AUX};

bool is_small(const Shape& s) { return std::min(s.rows, s.cols) <= kPad; }

void lay_out(const std::vector<PlacedShape>& shapes, bool small, int scaling, int64_t workspace_bytes, NsPlan* out)
{
    const size_t n = shapes.size();
    out->mats.resize(n);
    for (size_t i = 0; i < n;) {
        size_t end = i;
        int64_t at = kNsHeadBytes, n_tiles = 0;
        for (; end < n; ++end) {
            DevMatrix m{};
            const int64_t next = place(shapes[end].shape, at, &m);
            const int64_t t = tiles_of(shapes[end].shape.rows, kPad) * tiles_of(shapes[end].shape.cols, kPad);
            if (next > workspace_bytes || (end > i && n_tiles + t > kMaxNsTiles)) break;
            at = next;
            n_tiles += t;
            m.flat16 = 1;
            for (int s = 0; s < 4; ++s) {
                m.ptr[s] = shapes[end].ptr[s];
                if (m.ptr[s] % 16) m.flat16 = 0;
            }
            m.row16 = m.flat16 && m.cols % 8 == 0;
            const double R = (double)m.rows, C = (double)m.cols;
            m.factor = scaling == ADAMW_MUON_SCALE_SPECTRAL ? std::sqrt(std::max(1.0, R / C))
                     : scaling == ADAMW_MUON_SCALE_RMS ? 0.2 * std::sqrt(std::max(R, C)) : 1.0;
            out->mats[end] = m;
        }
        // the longest sums first
        std::vector<size_t> order;
        for (size_t k = i; k < end; ++k) order.push_back(k);
        NsBatch b;
        std::vector<DevTile> tiles;
        const auto tile = [&](size_t k, int64_t row, int64_t col) {
            return DevTile{out->mats[k].parts, (uint32_t)k, (uint32_t)row, (uint32_t)col, 0};
        };
        const auto take = [&](NsLaunch* l) {
            l->first = (int64_t)out->tiles.size();
            l->count = (int64_t)tiles.size();
            deal_tiles(tiles, &out->tiles);
            tiles.clear();
        };
        for (size_t k : order)
            for (uint32_t c = 0; c < out->mats[k].n_partials; ++c) tiles.push_back(tile(k, c, 0));
        take(&b.moments);
        b.small = small;
        if (small) {
            const auto runs = [&](int64_t (*cols)(int64_t)) {
                for (size_t k : order) {
                    const int64_t lp = out->mats[k].parts.lp;
                    for (int64_t x = 0; x < (lp + cols(lp) - 1) / cols(lp); ++x) tiles.push_back(tile(k, 0, x));
                }
            };
            runs(small_gram_cols);
            take(&b.normalise);
            for (size_t k : order) tiles.push_back(tile(k, 0, 0));
            take(&b.square);
            runs(small_apply_cols);
            take(&b.apply);
            out->batches.push_back(b);
            i = end;
            continue;
        }
        for (size_t k : order)
            for (uint32_t y = 0; y < out->mats[k].parts.sp / kPad; ++y)
                for (uint32_t x = 0; x < out->mats[k].parts.lp / kPad; ++x)
                    tiles.push_back(tile(k, y, x));
        take(&b.normalise);
        std::stable_sort(order.begin(), order.end(), [&](size_t x, size_t y) { return out->mats[x].parts.lp > out->mats[y].parts.lp; });
        const auto parts = [&](size_t k) -> const NsParts& { return out->mats[k].parts; };
        b.long_sums = std::any_of(order.begin(), order.end(), [&](size_t k) { return parts(k).lp > kLongSum; });
        b.square.kind = cheapest(b.long_sums ? 1 : 0, [&](int kind) {
            const auto gram = [&](const auto& add) {
                for (size_t k : order) add(square_tiles(parts(k).sp, kind), parts(k).lp);
            };
            const auto poly = [&](const auto& add) {
                for (size_t k : order) add(square_tiles(parts(k).sp, kind), parts(k).sp);
            };
            return launch_cost(kind, true, gram) + launch_cost(kind, true, poly);
        });
        b.apply.kind = cheapest(0, [&](int kind) {
            return launch_cost(kind, false, [&](const auto& add) {
                for (size_t k : order)
                    add(tiles_of(parts(k).sp, kTileRows[kind]) * tiles_of(parts(k).lp, kTileCols[kind]), parts(k).sp);
            });
        });
        // bands of 4 tile rows, column by column
        constexpr int64_t kBand = 4;
        for (size_t k : order) {
            const int kind = b.square.kind;
            const int64_t ty = tiles_of(out->mats[k].parts.sp, kTileRows[kind]), tx = tiles_of(out->mats[k].parts.sp, kTileCols[kind]);
            for (int64_t y0 = 0; y0 < ty; y0 += kBand)
                for (int64_t x = 0; x < tx; ++x)
                    for (int64_t y = y0; y < std::min(ty, y0 + kBand); ++y)
                        if (tile_needed(kind, y, x)) tiles.push_back(tile(k, y, x));
        }
        take(&b.square);
        std::stable_sort(order.begin(), order.end(), [&](size_t x, size_t y) { return out->mats[x].parts.sp > out->mats[y].parts.sp; });
        for (size_t k : order) {
            const int64_t ty = tiles_of(out->mats[k].parts.sp, kTileRows[b.apply.kind]);
            const int64_t tx = tiles_of(out->mats[k].parts.lp, kTileCols[b.apply.kind]);
            for (int64_t y0 = 0; y0 < ty; y0 += kBand)
                for (int64_t x = 0; x < tx; ++x)
                    for (int64_t y = y0; y < std::min(ty, y0 + kBand); ++y)
                        tiles.push_back(tile(k, y, x));
        }
        take(&b.apply);
        out->batches.push_back(b);
        i = end;
    }
}

}  // namespace

adamw_status check_ns(const adamw_newton_schulz* ns, NsScales* scales, std::string& err)
{
    if (!ns) { err = "Newton-Schulz coefficients are null"; return ADAMW_E_INVALID; }
    if (!std::isfinite(ns->a) || !std::isfinite(ns->b) || !std::isfinite(ns->c) || !std::isfinite(ns->eps)) {
        err = "Newton-Schulz coefficients and eps must be finite";
        return ADAMW_E_INVALID;
    }
    if (ns->eps < 0.0f) { err = "Newton-Schulz eps < 0"; return ADAMW_E_INVALID; }
    if (ns->steps < 1 || ns->steps > ADAMW_NS_MAX_STEPS) {
        err = "Newton-Schulz steps must lie in [1, ADAMW_NS_MAX_STEPS]";
        return ADAMW_E_INVALID;
    }
    // What the polynomials reach on the singular values of each step, [0, top]: at the ends or where a derivative is
    // zero, in q = x^2.
    const double a = ns->a, b = ns->b, c = ns->c;
    double top = 1.0, most = 1.0, poly = 0.0, whole = 0.0, times_a = 0.0;
    for (int k = 0; k < ns->steps; ++k) {
        const double end = top * top;
        double at[7] = {0.0, end}, next = 0.0, one = 0.0;
        int n = 2;
        const auto roots = [&](double r0, double r1, double r2) {   // of r0 + r1 q + r2 q^2 in (0, end)
            double q[2];
            int m = 0;
            if (r2 != 0.0) {
                const double d = r1 * r1 - 4.0 * r0 * r2;
                if (d >= 0.0) {
                    // without the difference of like numbers
                    const double h = -0.5 * (r1 + (r1 < 0.0 ? -std::sqrt(d) : std::sqrt(d)));
                    q[m++] = h / r2;
                    if (h != 0.0) q[m++] = r0 / h;
                }
            } else if (r1 != 0.0) {
                q[m++] = -r0 / r1;
            }
            for (int i = 0; i < m; ++i)
                if (q[i] > 0.0 && q[i] < end) at[n++] = q[i];
        };
        roots(a, 3.0 * b, 5.0 * c);   // of x (a + b q + c q^2)
        roots(b, 2.0 * c, 0.0);       // of b q + c q^2
        roots(a, 2.0 * b, 3.0 * c);   // of q (a + b q + c q^2)
        for (int i = 0; i < n; ++i) {
            const double q = at[i], p = q * (b + c * q);
            next = std::max(next, std::sqrt(q) * std::fabs(a + p));
            poly = std::max(poly, std::fabs(p));
            one = std::max(one, std::fabs(a + p));
            times_a = std::max(times_a, q * std::fabs(a + p));
        }
        whole = std::max(whole, one * 1.02);
        top = next * 1.01;   // rounding
        most = std::max(most, top);
        if (!(most <= 64.0)) {
            err = "Newton-Schulz coefficients take singular values of [0, 1] past 64";
            return ADAMW_E_INVALID;
        }
    }
    // no element of a matrix passes its largest singular value
    const auto under = [](double v) { return (int)std::floor(std::log2(61440.0 / std::max(v, 1e-3))); };
    scales->sx = under(most);
    scales->sa = under(most * most);
    scales->sb = under(poly * 1.02);
    scales->sp = under(whole);
    scales->sz = under(times_a * 1.02);
    // runs of equal length, of at most the steps whose polynomials stay under 2^11
    const int most_run = whole > 1.0 ? 1 + (int)std::min(std::log(2048.0) / std::log(whole), (double)ADAMW_NS_MAX_STEPS)
                                     : (int)ADAMW_NS_MAX_STEPS;
    scales->lo_steps = whole > 1.0 ? 1 + (int)std::min(std::log(16.0) / std::log(whole), (double)ADAMW_NS_MAX_STEPS)
                                   : (int)ADAMW_NS_MAX_STEPS;
    const int runs = (ns->steps + most_run - 1) / most_run;
    scales->run = (ns->steps + runs - 1) / runs;
    scales->sq = under(std::pow(std::max(whole, 1.0), scales->run));
    return ADAMW_OK;
}

adamw_status check_muon_hparams(const adamw_muon_hparams* hp, NsScales* scales, std::string& err)
{
    if (!hp) { err = "hparams is null"; return ADAMW_E_INVALID; }
    const float v[4] = {hp->lr, hp->momentum, hp->weight_decay, hp->inv_loss_scale};
    for (float x : v)
        if (!std::isfinite(x)) { err = "hyper-parameters must be finite"; return ADAMW_E_INVALID; }
    if (!(hp->momentum >= 0.0f && hp->momentum < 1.0f)) { err = "momentum must lie in [0, 1)"; return ADAMW_E_INVALID; }
    if (hp->lr < 0.0f) { err = "lr < 0"; return ADAMW_E_INVALID; }
    if (hp->weight_decay < 0.0f) { err = "weight_decay < 0"; return ADAMW_E_INVALID; }
    if (!(hp->inv_loss_scale > 0.0f)) { err = "inv_loss_scale must be > 0"; return ADAMW_E_INVALID; }
    if (hp->nesterov != 0 && hp->nesterov != 1) { err = "nesterov must be 0 or 1"; return ADAMW_E_INVALID; }
    if (hp->scaling < ADAMW_MUON_SCALE_NONE || hp->scaling > ADAMW_MUON_SCALE_RMS) {
        err = "unknown scaling of a Muon step";
        return ADAMW_E_INVALID;
    }
    return check_ns(&hp->ns, scales, err);
}

adamw_status ns_workspace_bytes(const adamw_tensor_list* list, const int64_t* cols, bool least, int64_t* bytes,
                                std::string& err)
{
    std::vector<Shape> shapes;
    adamw_status st = shapes_of(list, cols, &shapes, err);
    if (st != ADAMW_OK) return st;
    int64_t all = 0, largest = 0;
    for (const Shape& s : shapes) {
        const int64_t n = bytes_of(s);
        largest = std::max(largest, n);
        if (all <= kNsBatchBytes) all += n;
    }
    *bytes = kNsHeadBytes + (least ? largest : std::max(largest, std::min(all, kNsBatchBytes)));
    return ADAMW_OK;
}

adamw_status build_ns_plan(const NsKind& kind, const adamw_tensor_list* list, const int64_t* cols, int scaling,
                           uint64_t workspace, int64_t workspace_bytes, NsPlan* out, std::string& err)
{
    char buf[200];
    std::vector<Shape> shapes;
    adamw_status st = shapes_of(list, cols, &shapes, err);
    if (st != ADAMW_OK) return st;
    // the streams' addresses: each whole matrix is one segment of a step's plan
    Plan plan;
    st = build_plan(kind.esz, list, INT64_C(1) << 30, INT64_MAX, &plan, err);
    if (st != ADAMW_OK) return st;
    if (plan.segs.size() != shapes.size()) { err = "matrix list: internal error"; return ADAMW_E_INVALID; }

    int64_t least = kNsHeadBytes;
    for (const Shape& s : shapes) least = std::max(least, kNsHeadBytes + bytes_of(s));
    if (!workspace || workspace % kNsAlign) {
        err = "workspace is null or not 256-byte aligned";
        return ADAMW_E_INVALID;
    }
    if (workspace_bytes < least) {
        snprintf(buf, sizeof buf, "workspace of %lld bytes: the list's largest matrix needs %lld",
                 (long long)workspace_bytes, (long long)least);
        err = buf;
        return ADAMW_E_INVALID;
    }

    // what is written overlaps nothing else
    const bool step = kind.end != kEndOrtho;
    struct Range {
        uint64_t lo, hi;
        size_t mat;
        int stream;   // -1: the workspace
    };
    std::vector<Range> r;
    const auto written = [&](int s) { return s != ADAMW_STREAM_GRAD; };
    for (size_t i = 0; i < shapes.size(); ++i)
        for (int s = 0; s < kStreams; ++s)
            if (kind.esz[s]) {
                const uint64_t a = plan.segs[i].ptr[s];
                r.push_back(Range{a, a + (uint64_t)(shapes[i].rows * shapes[i].cols) * (uint64_t)kind.esz[s], i, s});
            }
    r.push_back(Range{workspace, workspace + (uint64_t)workspace_bytes, 0, -1});
    std::sort(r.begin(), r.end(), [](const Range& x, const Range& y) { return x.lo < y.lo; });
    // the furthest ends of what is written and of what is read so far
    uint64_t end_w = 0, end_r = 0;
    for (size_t i = 0; i < r.size(); ++i) {
        const bool w = written(r[i].stream);
        // a bf16 matrix that is its own result: the two ranges are one
        if (!step && kind.in == ADAMW_BF16 && i + 1 < r.size() && r[i + 1].lo == r[i].lo && r[i].stream >= 0 &&
            r[i + 1].stream >= 0 && r[i + 1].mat == r[i].mat) {
            if (r[i].lo < end_w || r[i].lo < end_r) { err = "buffers of the matrix list overlap"; return ADAMW_E_INVALID; }
            end_w = r[i].hi;
            ++i;
            continue;
        }
        if (r[i].lo < end_w || (w && r[i].lo < end_r)) {
            err = r[i].stream < 0 ? "the workspace overlaps a buffer of the matrix list"
                                  : "buffers of the matrix list overlap each other or the workspace";
            return ADAMW_E_INVALID;
        }
        (w ? end_w : end_r) = std::max(w ? end_w : end_r, r[i].hi);
    }
    if (!out) return ADAMW_OK;

    // the matrices in the workspace by themselves, each sort for its own launches
    std::vector<PlacedShape> of[2];
    for (size_t i = 0; i < shapes.size(); ++i) {
        PlacedShape p{shapes[i], {}};
        for (int s = 0; s < 4; ++s) p.ptr[s] = plan.segs[i].ptr[kStreamOf[s]];
        of[is_small(shapes[i])].push_back(p);
    }
    *out = NsPlan();
    const bool first = of[0].empty();
    lay_out(of[first], first, scaling, workspace_bytes, out);
    if (!first && !of[1].empty()) {
        out->small.reset(new NsPlan());
        lay_out(of[1], true, scaling, workspace_bytes, out->small.get());
    }
    return ADAMW_OK;
}

void NsPlan::flatten()
{
    if (!small) return;
    const uint32_t n_mats = (uint32_t)mats.size();
    const int64_t n_tiles = (int64_t)tiles.size();
    mats.insert(mats.end(), small->mats.begin(), small->mats.end());
    for (DevTile t : small->tiles) {
        t.mat += n_mats;
        tiles.push_back(t);
    }
    for (NsBatch b : small->batches) {
        for (NsLaunch* l : {&b.moments, &b.normalise, &b.square, &b.apply}) l->first += n_tiles;
        batches.push_back(b);
    }
    small.reset();
}

}  // namespace adamw
