// launch_check.cpp -- what the update kernels' workgroups touch, on the CPU: the table
// that a step uploads (update_table) and the kernels' own maps from workgroup and lane to
// elements (layout.hpp), walked workgroup by workgroup and lane by lane over random
// lists: shards, flat buffers, blocked state, the padded index, streams that share no
// alignment.  Built by tests/test_launch_tables.py under the sanitizers with plan.cpp;
// prints "launch_check ok" and a checksum, or aborts.  The segments' addresses and the
// plan's chunks are checked by plan_check.cpp; here every element of every segment has to
// be taken exactly once, whole units at 16-byte addresses of every stream.
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

// The elements of one workgroup, by a kernel of units of E elements, N units per lane
// and pass, 256 lanes.
template <int E, int N>
void walk(const Work& w, std::vector<uint8_t>& seen)
{
    constexpr uint32_t kBlock = 256;
    const uint32_t units = w.body / E, pass = w.parts * kBlock * N;
    const auto take = [&](uint64_t i) {
        CHECK(i < seen.size());
        ++seen[i];
    };
    for (uint32_t at = 0; at < units; at += pass)
        for (uint32_t tid = 0; tid < kBlock; ++tid)
            for (int h = 0; h < N; ++h) {
                const uint32_t k = at + unit_at<64, N>(tid, w, h);
                for (uint32_t e = 0; k < units && e < E; ++e) take(w.off + w.head + (uint64_t)k * E + e);
            }
    for (uint32_t tid = 0; tid < kBlock; ++tid)
        for (uint32_t e = w.part * kBlock + tid; e < w.edge; e += w.parts * kBlock) take(w.off + edge_at(w, e));
}

void check_table(const Plan& plan, const UpdateTable& t, const int esz[kStreams])
{
    bool wide = false;
    for (int s = 2; s < kStreams; ++s) wide |= esz[s] == 4;
    std::vector<std::vector<uint8_t>> seen(plan.segs.size());
    for (size_t i = 0; i < seen.size(); ++i) seen[i].assign((size_t)plan.info[i].count, 0);
    const uint32_t n_shared = (uint32_t)t.grid.n_shared, n_single = (uint32_t)t.grid.n_single;
    CHECK(t.items.size() == (size_t)n_shared + n_single);
    std::vector<uint32_t> parts_seen(t.items.size(), 0);
    for (uint32_t b = 0; b < (uint32_t)t.grid.workgroups(); ++b) {
        const ItemPart ip = update_item(b, n_shared, n_single);
        CHECK(ip.item < t.items.size() && ip.part < ip.parts);
        CHECK((ip.parts == 1) == (b < n_single));                       // one workgroup's items run first
        if (ip.parts > 1) CHECK(ip.part == b % 8);                      // part p runs on XCD p
        CHECK(!(parts_seen[ip.item] >> ip.part & 1u));
        parts_seen[ip.item] |= 1u << ip.part;
        const Work w = item_work(t.items[ip.item], ip);
        CHECK(w.seg < plan.segs.size() && w.body + w.edge > 0 && w.body % kPack == 0);
        for (int s = 0; s < kStreams && w.body; ++s)
            if (esz[s]) CHECK((plan.segs[w.seg].ptr[s] + (w.off + w.head) * esz[s]) % 16 == 0);
        if (wide) walk<4, 2>(w, seen[w.seg]);
        else walk<8, 1>(w, seen[w.seg]);
        mix(w.off + w.part);
    }
    for (size_t i = 0; i < t.items.size(); ++i) CHECK(parts_seen[i] == (i < n_shared ? 0xffu : 1u));
    for (const auto& v : seen)
        for (uint8_t x : v) CHECK(x == 1);
}

const int kEsz[][kStreams] = {
    {2, 2, 4, 4, 4}, {2, 2, 2, 2, 2}, {2, 2, 4, 4, 2}, {2, 2, 4, 2, 2}, {2, 2, 2, 4, 0}, {2, 2, 2, 2, 0}, {2, 2, 4, 4, 4},
};

void one_list(Rng& r, int it)
{
    const int* esz = kEsz[r.below(7)];
    const int64_t nt = it % 40 == 0 ? 300 : r.below(24);
    std::vector<int64_t> numel((size_t)nt);
    for (auto& n : numel) {
        const int64_t k = nt == 300 ? r.below(2) : r.below(4);
        n = k == 0 ? r.below(20) : k == 1 ? r.below(1500) : k == 2 ? 4080 + r.below(40) : r.below(50000);
    }
    adamw_tensor_list l{};
    uint32_t mask = (r.below(2) ? ADAMW_BLOCKED_STATE : 0u) | (r.below(2) ? ADAMW_FLAT_PAD8 : 0u);
    const int64_t align = mask & ADAMW_FLAT_PAD8 ? 8 : 1;
    int64_t total = 0;
    for (int64_t n : numel) total += (n + align - 1) / align * align;
    l.shard_end = -1;
    if (total && r.below(2)) {
        l.shard_begin = r.below(total);
        if (r.below(2)) l.shard_begin -= l.shard_begin % 8;
        l.shard_end = l.shard_begin + 1 + r.below(total - l.shard_begin);
    }
    std::vector<std::vector<void*>> ptr(kStreams);
    const int64_t phase = r.below(8), pack = r.below(3) == 0 ? 1 : r.below(2) ? 8 : 64;
    const bool apart = r.below(5) == 0;
    for (int s = 0; s < kStreams; ++s) {
        if (!esz[s]) continue;
        uint64_t at = ((uint64_t)1 << 40) + ((uint64_t)s << 36) + (uint64_t)(apart ? r.below(8) : phase) * esz[s];
        if ((mask & ADAMW_BLOCKED_STATE) && s >= 2) {
            if (s == 2) ptr[2].push_back((void*)(uintptr_t)(at & ~(uint64_t)255));
        } else if (r.below(5) == 0) {
            mask |= 1u << s;
            ptr[s].push_back((void*)(uintptr_t)at);
        } else {
            for (int64_t n : numel) {
                ptr[s].push_back((void*)(uintptr_t)at);
                at += (uint64_t)((n + pack - 1) / pack * pack * esz[s]);
            }
        }
    }
    l.n_tensors = nt;
    l.numel = numel.data();
    l.flat_mask = mask;
    for (int s = 0; s < kStreams; ++s) l.ptr[s] = ptr[s].empty() ? nullptr : ptr[s].data();
    Plan plan;
    std::string err;
    const int64_t chunk = r.below(3) ? 16384 : 2048 << r.below(6);
    CHECK(build_plan(esz, &l, chunk, kMaxUpdateChunks, &plan, err) == ADAMW_OK);
    const int64_t all = (int64_t)plan.chunks.size() * kXcdParts;
    for (int64_t resident : {(int64_t)0, (int64_t)512, (int64_t)1024, all, all - 1}) {
        const UpdateTable t = update_table(plan, resident);
        check_table(plan, t, esz);
        CHECK(t.items.size() <= plan.chunks.size());
        // a list that fits on the card whole is launched as planned, all its chunks shared
        if (all <= resident) CHECK(t.grid.n_single == 0 && t.items.size() == plan.chunks.size());
        else
            for (size_t i = 0; i < t.items.size(); ++i) {
                const uint32_t n = t.items[i].n_kind & kItemCountMask;
                const bool vec = (t.items[i].n_kind & kVecBit) != 0;
                CHECK(((int64_t)i >= t.grid.n_shared) == (n <= (vec ? kSingleVecElems : kSingleElems)));
            }
    }
}

}  // namespace

int main()
{
    Rng r{0x2545f4914f6cdd1dull};
    for (int it = 0; it < 240; ++it) one_list(r, it);
    // the workgroups that the card holds, as the occupancy caps leave them
    CHECK(resident_workgroups(kKernelMixedBf16) == 512 && resident_workgroups(kKernelMixedF16) == 512);
    CHECK(resident_workgroups(kKernelKahan) == 1024 && resident_workgroups(kKernelSplit) == 1024);
    CHECK(resident_workgroups(kKernelPureC32 + 3) == 512 && resident_workgroups(kKernelPureC32) == 1024);
    printf("launch_check ok %016llx\n", (unsigned long long)g_sum);
    return 0;
}
