// cache_check.cpp -- the stream's plan-cache policy and the list of validated keys,
// simulated on the CPU with the library's own code (plan.cpp).  Built by
// tests/test_plan_cache.py under the sanitizers; prints "cache_check ok" and the misses
// counted, or aborts.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <vector>

#include "plan.hpp"

using namespace adamw;

namespace {

#define CHECK(c)                                                                  \
    do {                                                                          \
        if (!(c)) {                                                               \
            fprintf(stderr, "%s:%d: check failed: %s\n", __FILE__, __LINE__, #c); \
            abort();                                                              \
        }                                                                         \
    } while (0)

struct Cache {
    struct Slot {
        int64_t tag;
        int list;
        size_t bytes;
        bool pinned;
    };
    std::vector<Slot> slots;   // most recently used first
    int misses = 0;

    // A call of kind `tag` with a list whose table takes `bytes`; true on a hit.
    bool call(int64_t tag, int list, size_t bytes, bool capture = false)
    {
        for (size_t i = 0; i < slots.size(); ++i)
            if (slots[i].tag == tag && slots[i].list == list) {
                std::rotate(slots.begin(), slots.begin() + (long)i, slots.begin() + (long)i + 1);
                slots[0].pinned |= capture;
                return true;
            }
        ++misses;
        CHECK(!capture);
        std::vector<SlotInfo> info;
        for (const Slot& s : slots) info.push_back(SlotInfo{s.tag, s.bytes, s.pinned});
        const size_t pick = choose_plan_slot(info, tag, bytes);
        CHECK(pick <= slots.size());
        if (pick == slots.size()) {
            slots.push_back(Slot{tag, list, bytes, false});
        } else {
            CHECK(!slots[pick].pinned && slots[pick].tag == tag);
            slots[pick].list = list;
            slots[pick].bytes = std::max(bytes, slots[pick].bytes);   // a buffer only grows
        }
        std::rotate(slots.begin(), slots.begin() + (long)pick, slots.begin() + (long)pick + 1);
        return false;
    }
    size_t unpinned(int64_t tag) const
    {
        return (size_t)std::count_if(slots.begin(), slots.end(), [&](const Slot& s) { return s.tag == tag && !s.pinned; });
    }
    size_t unpinned_bytes() const
    {
        size_t b = 0;
        for (const Slot& s : slots) b += s.pinned ? 0 : s.bytes;
        return b;
    }
};

const int64_t kStep = kKernelMixedBf16;

// An iteration over `groups` lists with a norm, a clipping, a check and a step each, in
// the order a training loop makes them: nothing is planned again after the first.
void iterations(int groups, size_t bytes)
{
    Cache c;
    for (int it = 0; it < 4; ++it) {
        for (int g = 0; g < groups; ++g) c.call(kTagNorm, g, bytes);
        for (int g = 0; g < groups; ++g) {
            c.call(kTagClip, g, bytes);
            c.call(kTagCheck, g, bytes);
            c.call(kStep, g, bytes);
        }
        CHECK(c.misses == 4 * groups);
    }
}

void bounds()
{
    // lists that come once each: no kind keeps more than kPlansMost, and once the tables
    // take kPlanBytes, a kind with more than kPlansKept gets no further slot
    Cache c;
    for (int l = 0; l < 500; ++l) {
        c.call(kStep, l, 4096);
        c.call(kTagNorm, l, 4096);
    }
    CHECK(c.unpinned(kStep) == kPlansMost && c.unpinned(kTagNorm) == kPlansMost);
    Cache d;
    for (int l = 0; l < 500; ++l) d.call(kStep, l, (size_t)6 << 20);
    CHECK(d.unpinned(kStep) == kPlanBytes / ((size_t)6 << 20) && d.unpinned_bytes() <= kPlanBytes);
    Cache e;
    for (int l = 0; l < 500; ++l) e.call(kStep, l, (size_t)20 << 20);
    CHECK(e.unpinned(kStep) == kPlansKept);
    // a kind's own lists are kept whatever the others take
    for (int l = 0; l < 8; ++l) e.call(kTagNorm, l, (size_t)20 << 20);
    for (int l = 492; l < 500; ++l) CHECK(e.call(kStep, l, (size_t)20 << 20));
    for (int l = 0; l < 8; ++l) CHECK(e.call(kTagNorm, l, (size_t)20 << 20));
}

void pins()
{
    Cache c;
    for (int l = 0; l < 40; ++l) {
        c.call(kStep, l, 1 << 20);
        CHECK(c.call(kStep, l, 1 << 20, true));
    }
    for (int l = 100; l < 200; ++l) c.call(kStep, l, 1 << 20);
    for (int l = 0; l < 40; ++l) CHECK(c.call(kStep, l, 1 << 20));
    CHECK(c.unpinned(kStep) == kPlansMost);   // the pinned tables count towards no limit
    CHECK(choose_plan_slot(std::vector<SlotInfo>(), kStep, 0) == 0);
}

void keys()
{
    ValidatedKeys v;
    for (int it = 0; it < 3; ++it)
        for (int64_t g = 0; g < 12; ++g)
            for (int64_t tag : {kTagNorm, kTagClip, kTagCheck, kStep}) {
                const std::vector<int64_t> key{tag, g};
                CHECK(v.seen(key) == (it > 0));
                if (it == 0) v.remember(key);
            }
    for (int64_t g = 0; g < 300; ++g) v.remember({7, g});
    CHECK(!v.seen({7, 300 - 129}) && v.seen({7, 300 - 128}) && v.seen({7, 299}));
    // long keys: the last 16 stay, and no more than fit
    ValidatedKeys w;
    const auto key = [](int64_t g) {
        std::vector<int64_t> k((size_t)1 << 20, 0);
        k[5] = g;
        return k;
    };
    for (int64_t g = 0; g < 40; ++g) w.remember(key(g));
    for (int64_t g = 24; g < 40; ++g) CHECK(w.seen(key(g)));
    CHECK(!w.seen(key(23)));
}

}  // namespace

int main()
{
    for (int groups : {1, 2, 3, 5, 6, 8, 12, 32}) iterations(groups, 100 << 10);
    iterations(8, (size_t)9 << 20);
    bounds();
    pins();
    keys();
    printf("cache_check ok 0\n");
    return 0;
}
