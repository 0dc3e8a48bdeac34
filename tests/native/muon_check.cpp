// muon_check.cpp -- the planner of the Newton-Schulz products under AddressSanitizer and
// UndefinedBehaviorSanitizer, on the CPU with synthetic (never dereferenced) device
// addresses.  Built by tests/test_muon_cpu.py with g++ together with muon_plan.cpp, plan.cpp and
// validate.cpp; prints "muon_check ok" and a checksum of every plan (the same with and without
// the sanitizers), or aborts.
//
// Every plan is checked: each matrix lies in one batch; its parts of the workspace lie inside the
// workspace and apart from each other and from the other matrices' of the batch; and each launch's
// workgroups cover every matrix of the batch exactly once (the square ones: the tiles on and below
// the diagonal).  The overlap search is compared with a quadratic one.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <cmath>
#include <map>
#include <string>
#include <utility>
#include <vector>

#include "muon.hpp"
#include "plan.hpp"

using namespace adamw;

namespace {

uint64_t g_sum = 1469598103934665603ull;
void mix(uint64_t x) { g_sum = (g_sum ^ x) * 1099511628211ull; }

#define CHECK(c)                                                                  \
    do {                                                                          \
        if (!(c)) {                                                               \
            fprintf(stderr, "%s:%d: check failed: %s\n", __FILE__, __LINE__, #c); \
            abort();                                                              \
        }                                                                         \
    } while (0)

struct Rng {
    uint64_t s;
    uint64_t next()
    {
        s ^= s << 13;
        s ^= s >> 7;
        s ^= s << 17;
        return s;
    }
    int64_t below(int64_t n) { return n > 0 ? (int64_t)(next() % (uint64_t)n) : 0; }
};

struct Range {
    uint64_t lo, hi;
};
bool apart(const Range& x, const Range& y) { return x.hi <= y.lo || y.hi <= x.lo; }

struct List {
    std::vector<int64_t> numel, cols;
    std::vector<void*> ptr[kStreams];
    adamw_tensor_list c;
    adamw_tensor_list* get()
    {
        c.n_tensors = (int64_t)numel.size();
        c.numel = numel.data();
        for (int s = 0; s < kStreams; ++s) c.ptr[s] = ptr[s].data();
        return &c;
    }
};

void check_batch(const NsPlan& plan, const NsBatch& b, std::vector<int>& seen, int64_t bytes, bool step)
{
    // the matrices of the batch, by its moments' workgroups
    std::map<uint32_t, std::vector<int>> runs;
    for (int64_t i = 0; i < b.moments.count; ++i) {
        const DevTile& t = plan.tiles[(size_t)(b.moments.first + i)];
        CHECK(t.mat < plan.mats.size());
        auto& v = runs[t.mat];
        if (v.empty()) v.resize(plan.mats[t.mat].n_partials);
        CHECK(t.row < v.size() && !v[t.row]);
        v[t.row] = 1;
    }
    std::vector<Range> parts;
    for (auto& kv : runs) {
        CHECK(!seen[kv.first]);
        seen[kv.first] = 1;
        const DevMatrix& m = plan.mats[kv.first];
        for (int x : kv.second) CHECK(x);
        const NsParts& p = m.parts;
        const int64_t n = (int64_t)m.rows * m.cols, s = std::min(m.rows, m.cols), l = std::max(m.rows, m.cols);
        CHECK((int64_t)m.n_partials * m.chunk >= n && ((int64_t)m.n_partials - 1) * m.chunk < n && m.chunk % kMomentElems == 0);
        CHECK(m.n_partials <= kMaxPartials && (m.tall != 0) == (m.rows > m.cols));
        CHECK(p.sp % kPad == 0 && p.sp >= s && p.sp < s + kPad && p.lp % kPad == 0 && p.lp >= l && p.lp < l + kPad);
        const uint64_t whole = (uint64_t)2 * p.sp * p.lp, square = (uint64_t)2 * p.sp * p.sp;
        const Range r[8] = {{p.hi(0), p.hi(0) + whole}, {p.lo(), p.lo() + whole}, {p.hi(1), p.hi(1) + whole},
                            {p.a(), p.a() + square}, {p.b(), p.b() + square}, {p.da(), p.da() + 4 * p.sp},
                            {p.db(), p.db() + 4 * p.sp}, {m.partials, m.partials + 8 * (uint64_t)m.n_partials}};
        for (const Range& x : r) parts.push_back(x);
        if (step) {   // u's room: that of hi(1), a and b, and nothing else's
            const Range u{p.u(), p.u() + 4 * (uint64_t)n};
            CHECK(u.hi <= (uint64_t)bytes);
            for (int k : {0, 1, 5, 6, 7}) CHECK(apart(u, r[k]));
        }
        for (const Range& x : r) CHECK(x.lo % kNsAlign == 0);
        for (uint64_t x : {(uint64_t)m.rows, (uint64_t)m.cols, (uint64_t)p.sp, (uint64_t)m.tall, p.base, m.partials}) mix(x);
    }
    for (const Range& x : parts) CHECK(x.lo >= (uint64_t)kNsHeadBytes && x.hi <= (uint64_t)bytes);
    std::sort(parts.begin(), parts.end(), [](const Range& x, const Range& y) { return x.lo < y.lo; });
    for (size_t i = 1; i < parts.size(); ++i) CHECK(apart(parts[i - 1], parts[i]));

    if (b.small) {
        CHECK(b.square.count == (int64_t)runs.size());
        std::map<uint32_t, int> once;
        for (int64_t i = 0; i < b.square.count; ++i) CHECK(!once[plan.tiles[(size_t)(b.square.first + i)].mat]++);
        for (const bool gram : {true, false}) {
            const NsLaunch& l = gram ? b.normalise : b.apply;
            std::map<uint32_t, std::vector<int>> got;
            for (int64_t i = 0; i < l.count; ++i) {
                const DevTile& t = plan.tiles[(size_t)(l.first + i)];
                const NsParts& p = plan.mats[t.mat].parts;
                const int64_t cols = gram ? small_gram_cols(p.lp) : small_apply_cols(p.lp), n = (p.lp + cols - 1) / cols;
                CHECK(runs.count(t.mat) && p.sp == kPad && cols % kPad == 0 && t.parts.base == p.base && t.row == 0);
                // the partial Gram matrices lie before u's room
                if (gram) CHECK(n <= kMaxSmallRuns && p.lo() + (uint64_t)n * kPad * kPad * 4 <= p.u());
                auto& v = got[t.mat];
                v.resize((size_t)n);
                CHECK((int64_t)t.col < n && !v[t.col]++);
            }
            CHECK(got.size() == runs.size());
            for (auto& kv : got)
                for (int x : kv.second) CHECK(x == 1);
        }
        return;
    }
    // 64 x 64 of the padded matrix each, the tiles of a kind of the matrix, or of its square
    const auto cover = [&](const NsLaunch& l, int th, int tw, bool square) {
        std::map<uint32_t, std::map<std::pair<uint32_t, uint32_t>, int>> got;
        for (int64_t i = 0; i < l.count; ++i) {
            const DevTile& t = plan.tiles[(size_t)(l.first + i)];
            CHECK(runs.count(t.mat) && !got[t.mat][std::make_pair(t.row, t.col)]++);
            const NsParts &x = t.parts, &y = plan.mats[t.mat].parts;
            CHECK(x.base == y.base && x.sp == y.sp && x.lp == y.lp);
            mix(t.mat * 31 + t.row * 7 + t.col);
        }
        CHECK(got.size() == runs.size());
        for (auto& kv : got) {
            const DevMatrix& m = plan.mats[kv.first];
            const int64_t h = m.parts.sp, w = square ? m.parts.sp : m.parts.lp;
            for (auto& t : kv.second) CHECK(t.first.first * (int64_t)th < h && t.first.second * (int64_t)tw < w);
            if (!square) {
                CHECK((int64_t)kv.second.size() == (h + th - 1) / th * ((w + tw - 1) / tw));
                continue;
            }
            // every 64 x 64 block is written once: by its own tile, or as the mirror of a tile
            const int64_t n = h / kPad;
            std::vector<int> hit((size_t)(n * n));
            for (auto& t : kv.second)
                for (int64_t y = t.first.first * th / kPad; y < std::min(n, (int64_t)(t.first.first + 1) * th / kPad); ++y)
                    for (int64_t x = t.first.second * tw / kPad; x < std::min(n, (int64_t)(t.first.second + 1) * tw / kPad); ++x) {
                        ++hit[(size_t)(y * n + x)];
                        if (tile_mirrored(l.kind, t.first.first, t.first.second)) ++hit[(size_t)(x * n + y)];
                    }
            for (int x : hit) CHECK(x == 1);
        }
        CHECK(l.count <= kMaxNsTiles);
    };
    cover(b.normalise, kPad, kPad, false);
    cover(b.square, kTileRows[b.square.kind], kTileCols[b.square.kind], true);
    cover(b.apply, kTileRows[b.apply.kind], kTileCols[b.apply.kind], false);
}

void one_list(Rng& r)
{
    const bool step = r.below(2), f32 = r.below(2);
    NsKind kind{};
    kind.end = step ? kEndMixedBf16 : kEndOrtho;
    kind.in = !step && f32 ? ADAMW_F32 : ADAMW_BF16;
    kind.esz[ADAMW_STREAM_PARAM] = 2;
    kind.esz[ADAMW_STREAM_GRAD] = kind.in == ADAMW_F32 ? 4 : 2;
    if (step) kind.esz[ADAMW_STREAM_EXP_AVG] = kind.esz[ADAMW_STREAM_AUX] = 4;
    List l{};
    const int64_t nt = r.below(12), pad8 = r.below(2);
    const int64_t most = r.below(4) == 0 ? 3000 : 200;
    uint64_t at = 0x7f0000000000ull;
    std::vector<Range> buffers;
    std::vector<int> writes;
    int64_t total = 0;
    std::vector<int64_t> starts;
    for (int64_t i = 0; i < nt; ++i) {
        const int64_t rows = r.below(20) ? 1 + r.below(most) : 0, cols = 1 + r.below(most);
        l.numel.push_back(rows * cols);
        l.cols.push_back(cols);
        starts.push_back(total);
        total += pad8 ? (rows * cols + 7) / 8 * 8 : rows * cols;
        for (int s = 0; s < kStreams; ++s) {
            if (!kind.esz[s]) {
                l.ptr[s].push_back(nullptr);
                continue;
            }
            at += (uint64_t)kind.esz[s] * (uint64_t)r.below(9);
            at = (at + 3) / 4 * 4;
            l.ptr[s].push_back(reinterpret_cast<void*>(at));
            if (rows) {
                buffers.push_back(Range{at, at + (uint64_t)(rows * cols * kind.esz[s])});
                writes.push_back(s != ADAMW_STREAM_GRAD);
            }
            at += (uint64_t)(rows * cols * kind.esz[s]);
        }
    }
    starts.push_back(total);
    l.c.shard_begin = 0;
    l.c.shard_end = -1;
    l.c.flat_mask = pad8 ? ADAMW_FLAT_PAD8 : 0;
    std::string err;
    int64_t bytes = 0, least = 0;
    CHECK(ns_workspace_bytes(l.get(), l.cols.data(), false, &bytes, err) == ADAMW_OK);
    CHECK(ns_workspace_bytes(l.get(), l.cols.data(), true, &least, err) == ADAMW_OK);
    CHECK(least <= bytes && least >= kNsHeadBytes);
    const int64_t take = r.below(2) ? bytes : least + r.below(bytes - least + 1);
    const uint64_t ws = 0x600000000000ull;
    NsPlan plan;
    CHECK(build_ns_plan(kind, l.get(), l.cols.data(), (int)r.below(3), ws, take, &plan, err) == ADAMW_OK);
    std::vector<int> seen(plan.mats.size());
    for (const NsBatch& b : plan.batches) check_batch(plan, b, seen, take, step);
    for (int x : seen) CHECK(x);
    if (take == bytes) CHECK(plan.batches.size() <= 1);
    CHECK(build_ns_plan(kind, l.get(), l.cols.data(), 0, ws, least - 1, nullptr, err) == ADAMW_E_INVALID);
    CHECK(build_ns_plan(kind, l.get(), l.cols.data(), 0, ws + 8, take, nullptr, err) == ADAMW_E_INVALID);

    // a buffer moved somewhere near another one
    if (buffers.size() >= 2) {
        const int64_t i = r.below(nt);
        int s = (int)r.below(kStreams);
        while (!kind.esz[s]) s = (s + 1) % kStreams;
        if (l.numel[(size_t)i]) {
            const uint64_t to = (buffers[(size_t)r.below((int64_t)buffers.size())].lo + 4 * (uint64_t)r.below(64)) / 4 * 4;
            l.ptr[s][(size_t)i] = reinterpret_cast<void*>(to);
            std::vector<Range> now;
            std::vector<int> w, mat;
            for (int64_t k = 0; k < nt; ++k)
                for (int q = 0; q < kStreams; ++q)
                    if (kind.esz[q] && l.numel[(size_t)k]) {
                        const uint64_t a = (uint64_t)(uintptr_t)l.ptr[q][(size_t)k];
                        now.push_back(Range{a, a + (uint64_t)(l.numel[(size_t)k] * kind.esz[q])});
                        w.push_back(q != ADAMW_STREAM_GRAD);
                        mat.push_back((int)k);
                    }
            bool bad = false;
            for (size_t x = 0; x < now.size(); ++x)
                for (size_t y = 0; y < x; ++y) {
                    const bool own = !step && kind.in == ADAMW_BF16 && mat[x] == mat[y] && now[x].lo == now[y].lo;
                    if (!own && (w[x] || w[y]) && !apart(now[x], now[y])) bad = true;
                }
            const adamw_status st = build_ns_plan(kind, l.get(), l.cols.data(), 0, ws, take, nullptr, err);
            CHECK((st != ADAMW_OK) == bad);
            mix((uint64_t)bad);
        }
    }
    // a shard between two matrices, and one that cuts a matrix
    if (nt >= 2) {
        l.c.shard_begin = starts[(size_t)r.below(nt)];
        l.c.shard_end = starts[(size_t)nt];
        CHECK(ns_workspace_bytes(l.get(), l.cols.data(), true, &least, err) == ADAMW_OK);
        const size_t k = (size_t)r.below(nt);
        if (l.numel[k] >= 2) {
            l.c.shard_begin = starts[k] + 1;
            CHECK(ns_workspace_bytes(l.get(), l.cols.data(), true, &least, err) == ADAMW_E_INVALID);
        }
    }
}

}  // namespace

// Random coefficients: refused where a singular value passes 64 on a grid, and else the powers of two hold what a
// grid of singular values reaches, and a run of steps multiplies a rounding by at most 2^11 before its last step.
static void one_scale(Rng& r)
{
    const auto value = [&](double most) { return (float)((double)(r.below(2000001) - 1000000) * 1e-6 * most); };
    const adamw_newton_schulz ns{value(8.0), value(16.0), value(8.0), 1e-7f, (int32_t)(1 + r.below(ADAMW_NS_MAX_STEPS))};
    NsScales s{};
    std::string err;
    const bool taken = check_ns(&ns, &s, err) == ADAMW_OK;
    double top = 1.0, most = 1.0, poly = 0.0, whole = 0.0, times_a = 0.0;
    for (int k = 0; k < ns.steps && most <= 64.0; ++k) {
        double next = 0.0;
        for (int i = 0; i <= 400; ++i) {
            const double x = top * i / 400, q = x * x, b = q * ((double)ns.b + (double)ns.c * q), p = (double)ns.a + b;
            next = std::max(next, std::fabs(x * p));
            poly = std::max(poly, std::fabs(b));
            whole = std::max(whole, std::fabs(p));
            times_a = std::max(times_a, std::fabs(q * p));
        }
        most = std::max(most, top = next);
    }
    if (!taken) return;
    CHECK(most <= 64.0 && s.run >= 1 && s.run <= ns.steps);
    CHECK(std::ldexp(most, s.sx) <= 61440.0 && std::ldexp(most * most, s.sa) <= 61440.0 && std::ldexp(poly, s.sb) <= 61440.0);
    CHECK(std::ldexp(whole, s.sp) <= 61440.0 && std::ldexp(times_a, s.sz) <= 61440.0);
    CHECK(std::ldexp(std::pow(whole, s.run), s.sq) <= 61440.0 && std::pow(whole, s.run - 1) <= 2048.0);
    mix((uint64_t)s.run);
    mix((uint64_t)(int64_t)s.sq);
}

// The usual coefficients' runs: 7 steps in one, more in runs of like length.
static void usual_runs()
{
    const int want[ADAMW_NS_MAX_STEPS] = {1, 2, 3, 4, 5, 6, 7, 4, 5, 5, 6, 6, 7, 7, 5, 6};
    for (int steps = 1; steps <= ADAMW_NS_MAX_STEPS; ++steps) {
        const adamw_newton_schulz ns{3.4445f, -4.7750f, 2.0315f, 1e-7f, steps};
        NsScales s{};
        std::string err;
        CHECK(check_ns(&ns, &s, err) == ADAMW_OK && s.run == want[steps - 1]);
    }
}

int main()
{
    Rng r{88172645463325252ull};
    for (int i = 0; i < 1500; ++i) one_list(r);
    for (int i = 0; i < 20000; ++i) one_scale(r);
    usual_runs();
    printf("muon_check ok %016llx\n", (unsigned long long)g_sum);
    return 0;
}
