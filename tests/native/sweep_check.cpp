// sweep_check.cpp -- the planner of the gradient sweeps (norms, clipping) and the
// update kernels' tables under AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU with synthetic (never
// dereferenced) device addresses.  Built by tests/test_sweep_sanitizers.py with g++
// together with plan.cpp and validate.cpp; prints "sweep_check ok" and a checksum of
// every plan (the same with and without the sanitizers), or aborts.
//
// Every plan is checked: the chunks of each tensor cover exactly its elements inside
// the shard, in order, each chunk but a tensor's first starts at a 16-byte edge, the
// tensors' first chunks are where Plan::tensor_first says, and the workgroups of a
// shared plan are the 8 parts of each long chunk.  check_disjoint is compared with a
// quadratic search.
#include <stdio.h>
#include <stdlib.h>

#include <string>
#include <vector>

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

void one_list(Rng& r)
{
    const int esz = r.below(2) ? 4 : 2;
    const int64_t nt = r.below(20);
    const bool pad8 = r.below(3) == 0, flat = r.below(4) == 0;
    const int64_t chunk = 2048 << r.below(8);
    static const int64_t lens[] = {0, 1, 7, 8, 9, 100, 2047, 2048, 2049, 16384, 16391, 70000, 600000};
    std::vector<int64_t> numel, start;
    std::vector<void*> ptr;
    int64_t total = 0;
    uint64_t at = 0x7f0000000000ull + (uint64_t)r.below(16) * esz;
    for (int64_t i = 0; i < nt; ++i) {
        numel.push_back(lens[r.below(13)]);
        start.push_back(total);
        total += pad8 ? (numel[i] + 7) / 8 * 8 : numel[i];
        // mostly one after another, now and then back over what came before
        if (r.below(8) == 0 && at > 0x7f0000000000ull + 4096) at -= (uint64_t)r.below(2048) * esz;
        ptr.push_back((void*)(uintptr_t)at);
        at += (uint64_t)numel[i] * esz + (uint64_t)r.below(3) * 16;
    }
    const int64_t b = r.below(total + 1), e = b + r.below(total - b + 1);
    if (flat) {
        ptr.assign(1, (void*)(uintptr_t)(0x7f0000000000ull + (uint64_t)r.below(16) * esz));
    }
    adamw_tensor_list l{};
    l.n_tensors = nt;
    l.numel = numel.data();
    l.ptr[ADAMW_STREAM_GRAD] = ptr.data();
    l.shard_begin = b;
    l.shard_end = e;
    l.flat_mask = (pad8 ? ADAMW_FLAT_PAD8 : 0u) | (flat ? 2u : 0u);
    Plan plan;
    std::string err;
    CHECK(build_sweep_plan(esz, &l, chunk, kMaxSweepChunks, &plan, err) == ADAMW_OK);
    CHECK(build_sweep_plan(esz, &l, chunk, kMaxSweepChunks, nullptr, err) == ADAMW_OK);
    CHECK((int64_t)plan.tensor_first.size() == nt + 1);
    struct Range { uint64_t lo, hi; };
    std::vector<Range> pieces;
    for (int64_t i = 0; i < nt; ++i) {
        const int64_t lo = b > start[i] ? b - start[i] : 0;
        const int64_t hi = e - start[i] < numel[i] ? e - start[i] : numel[i];
        const uint64_t base = flat ? (uint64_t)(uintptr_t)ptr[0] + (uint64_t)(start[i] - b) * esz
                                   : (uint64_t)(uintptr_t)ptr[i];
        int64_t pos = lo;
        for (uint32_t c = plan.tensor_first[i]; c < plan.tensor_first[i + 1]; ++c) {
            const DevChunk& ch = plan.chunks[c];
            const uint64_t addr = plan.segs[ch.seg].ptr[ADAMW_STREAM_GRAD] + ch.off * esz;
            CHECK(plan.info[ch.seg].tensor == i && plan.info[ch.seg].tensor_off + (int64_t)ch.off == pos);
            CHECK(addr == base + (uint64_t)pos * esz && (pos == lo || addr % 16 == 0));
            const int64_t n = ch.n_kind & kCountMask;
            CHECK(n > 0 && n < chunk + 16 / esz);
            pos += n;
            mix(addr);
            mix((uint64_t)n);
        }
        CHECK(pos == (hi > lo ? hi : lo));
        if (hi > lo) pieces.push_back(Range{base + (uint64_t)lo * esz, base + (uint64_t)hi * esz});
    }
    CHECK(plan.tensor_first.empty() || plan.tensor_first.back() == plan.chunks.size());
    const std::vector<DevSweep> whole = sweep_groups(plan, esz, false), shared = sweep_groups(plan, esz, true);
    CHECK(whole.size() == plan.chunks.size());
    size_t k = 0;
    for (const DevSweep& w : whole) {
        CHECK(w.part == kWholeChunk);
        const uint32_t parts = (int64_t)w.n * esz > kClipWholeBytes ? kXcdParts : 1;
        for (uint32_t p = 0; p < parts; ++p, ++k)
            CHECK(k < shared.size() && shared[k].addr == w.addr && shared[k].n == w.n &&
                  shared[k].part == (parts == 1 ? kWholeChunk : p));
    }
    CHECK(k == shared.size());
    bool overlap = false;
    for (size_t x = 0; x < pieces.size() && !flat; ++x)
        for (size_t y = x + 1; y < pieces.size(); ++y)
            overlap |= pieces[x].lo < pieces[y].hi && pieces[y].lo < pieces[x].hi;
    CHECK((check_disjoint(esz, &l, err) == ADAMW_OK) == !overlap);
    mix(overlap);
}

// The update table of a step's plan: its items cover the plan's chunks once and in
// order within each of the two kinds, vector parts keep their alignment in every
// stream, ends of up to 7 elements go with them, and short items are one workgroup's.
void one_update(Rng& r)
{
    int esz[kStreams] = {2, 2, 4, 4, 4};
    if (r.below(2))
        for (int s = 2; s < kStreams; ++s) esz[s] = 2;
    const int64_t nt = 1 + r.below(12);
    static const int64_t lens[] = {0, 1, 6, 7, 8, 9, 15, 16, 500, 512, 513, 4089, 4096, 4097, 4111, 16384, 16400, 50000};
    std::vector<int64_t> numel;
    std::vector<std::vector<void*>> ptr(kStreams);
    uint64_t at[kStreams];
    const bool apart = r.below(4) == 0;   // streams that cannot be aligned together
    const int64_t phase = r.below(8);
    for (int s = 0; s < kStreams; ++s)
        at[s] = 0x7f0000000000ull + ((uint64_t)s << 36) + (uint64_t)(apart ? r.below(8) : phase) * esz[s];
    for (int64_t i = 0; i < nt; ++i) {
        numel.push_back(lens[r.below(18)]);
        for (int s = 0; s < kStreams; ++s) {
            ptr[s].push_back((void*)(uintptr_t)at[s]);
            at[s] += (uint64_t)numel[i] * esz[s];
        }
    }
    adamw_tensor_list l{};
    l.n_tensors = nt;
    l.numel = numel.data();
    for (int s = 0; s < kStreams; ++s) l.ptr[s] = ptr[s].data();
    l.shard_end = -1;
    Plan plan;
    std::string err;
    const int64_t chunk = 2048 << r.below(4);
    CHECK(build_plan(esz, &l, chunk, kMaxUpdateChunks, &plan, err) == ADAMW_OK);
    const UpdateTable t = update_table(plan);
    CHECK(t.grid.n_shared + t.grid.n_single == (int64_t)t.items.size() && t.items.size() <= plan.chunks.size());
    CHECK(t.grid.workgroups() == 8 * t.grid.n_shared + t.grid.n_single);
    std::vector<std::vector<uint8_t>> seen(plan.segs.size());
    for (size_t i = 0; i < seen.size(); ++i) seen[i].assign((size_t)plan.info[i].count, 0);
    int64_t vector_elems = 0, planned_vector = 0;
    for (const DevChunk& c : plan.chunks)
        if (c.n_kind & kVecBit) planned_vector += c.n_kind & kCountMask;
    for (size_t i = 0; i < t.items.size(); ++i) {
        const DevChunk& it = t.items[i];
        const bool vec = (it.n_kind & kVecBit) != 0, alone = (int64_t)i >= t.grid.n_shared;
        const uint32_t n = it.n_kind & kItemCountMask, head = vec ? it.n_kind >> kItemHeadShift & 7u : n;
        const uint32_t body = vec ? (n - head) / kPack * kPack : 0;
        CHECK(n > 0 && (!vec || body > 0) && (vec || (it.n_kind >> kItemHeadShift) == 0));
        CHECK(alone == (n <= (vec ? kSingleVecElems : kSingleElems)));
        if (i > 0 && (int64_t)i != t.grid.n_shared) {
            const DevChunk& before = t.items[i - 1];
            CHECK(before.seg < it.seg || (before.seg == it.seg && before.off < it.off));
        }
        for (int s = 0; s < kStreams && vec; ++s) CHECK((plan.segs[it.seg].ptr[s] + (it.off + head) * esz[s]) % 16 == 0);
        CHECK(it.off + n <= seen[it.seg].size());
        for (uint32_t k = 0; k < n; ++k) ++seen[it.seg][it.off + k];
        vector_elems += body;
        mix(it.off);
        mix(it.n_kind);
    }
    for (const auto& v : seen)
        for (uint8_t x : v) CHECK(x == 1);
    CHECK(vector_elems == planned_vector);
}

}  // namespace

int main()
{
    Rng r{88172645463325252ull};
    for (int i = 0; i < 3000; ++i) one_list(r);
    for (int i = 0; i < 2000; ++i) one_update(r);
    // the grid limit, and the arguments of clipping
    int64_t n = 0;
    void* p = (void*)(uintptr_t)0x7f0000000000ull;
    adamw_tensor_list l{};
    l.n_tensors = 1;
    l.numel = &n;
    l.ptr[ADAMW_STREAM_GRAD] = &p;
    l.shard_end = -1;
    std::string err;
    n = 100 * 2048;
    CHECK(build_sweep_plan(2, &l, 2048, 100, nullptr, err) == ADAMW_OK);
    n += 1;
    CHECK(build_sweep_plan(2, &l, 2048, 100, nullptr, err) == ADAMW_E_INVALID);
    double s = 0;
    adamw_grad_clip c{&s, 1.0f, 0.0f};
    CHECK(check_clip(&c, err) == ADAMW_OK);
    c.max_norm = -1.0f;
    CHECK(check_clip(&c, err) == ADAMW_E_INVALID);
    int esz = 0;
    CHECK(check_sweep_dtype(ADAMW_F32, &esz, err) == ADAMW_OK && esz == 4);
    CHECK(check_sweep_dtype((adamw_dtype)9, &esz, err) == ADAMW_E_UNSUPPORTED);
    printf("sweep_check ok %016llx\n", (unsigned long long)g_sum);
    return 0;
}
