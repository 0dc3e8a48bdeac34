"""Matrices of at most 64 on the shorter side on the CPU: their runs of columns, and their batches beside the others'."""
import os
import subprocess

from test_sanitizers import CSRC, ROOT, SAN, _build_and_run

SOURCE = r"""
#include <stdio.h>
#include <stdlib.h>
#include "muon.hpp"
using namespace adamw;
int main()
{
    for (int64_t lp = kPad; lp <= (INT64_C(1) << 30); lp += lp < 100000 ? kPad : lp / kPad / 50 * kPad) {
        const int64_t cols = small_gram_cols(lp), n = (lp + cols - 1) / cols;
        const NsParts p{kNsHeadBytes, (uint32_t)kPad, (uint32_t)lp};
        // whole tiles, as many partial Gram matrices as one workgroup adds up, and all of them before u
        if (cols < kPad || cols % kPad || n > kMaxSmallRuns || p.base + (uint64_t)(n * kSmallTri) * 8 > p.u()) {
            printf("%lld columns: runs of %lld\n", (long long)lp, (long long)cols);
            return 1;
        }
        // no run is so long that other CUs stand idle meanwhile
        if (cols > 2048 && n < kMaxSmallRuns - 1 && lp / kMaxSmallRuns > 2048 + kPad && n * 2 < kMaxSmallRuns) return 2;
    }
    puts("ok");
    return 0;
}
"""


def test_partial_gram_matrices_have_their_room(tmp_path):
    src = tmp_path / "runs.cpp"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-I", os.path.join(ROOT, "include"), "-I", CSRC, str(src), "-o",
                    str(tmp_path / "runs")], check=True)
    out = subprocess.run([str(tmp_path / "runs")], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout == "ok\n", out.stdout


MIXED = r"""
#include <stdio.h>
#include <algorithm>
#include <map>
#include <set>
#include "muon.hpp"
using namespace adamw;
#define CHECK(c) do { if (!(c)) { printf("line %d: %s\n", __LINE__, #c); return 1; } } while (0)

// Tiles of every launch, of matrices `from` to `to` of the table
static int check(const NsPlan& p, const NsBatch& b, std::set<uint32_t>& seen, int64_t bytes)
{
    std::set<uint32_t> here;
    for (const NsLaunch* l : {&b.moments, &b.normalise, &b.square, &b.apply}) {
        std::set<uint32_t> in;
        for (int64_t i = 0; i < l->count; ++i) {
            const DevTile& t = p.tiles[(size_t)(l->first + i)];
            CHECK(t.mat < p.mats.size() && t.parts.base == p.mats[t.mat].parts.base);
            CHECK((p.mats[t.mat].parts.sp == (uint32_t)kPad) == b.small);
            in.insert(t.mat);
        }
        if (l == &b.moments) here = in;
        CHECK(in == here);
    }
    for (uint32_t m : here) {
        CHECK(seen.insert(m).second);
        CHECK((int64_t)p.mats[m].partials + 8 * (int64_t)p.mats[m].n_partials <= bytes);
    }
    return 0;
}

int main()
{
    const int64_t sides[][2] = {{16, 48}, {300, 520}, {64, 64}, {65, 66}, {700, 30}, {1, 9}, {128, 128}, {0, 5}};
    for (int pick = 1; pick < 256; ++pick)
        for (int least = 0; least < 2; ++least) {
            std::vector<int64_t> numel, cols;
            std::vector<void*> a, b;
            uint64_t at = 0x7f0000000000ull;
            int n_small = 0, n_large = 0;
            for (int i = 0; i < 8; ++i) {
                if (!(pick >> i & 1)) continue;
                const int64_t r = sides[i][0], c = sides[i][1];
                numel.push_back(r * c);
                cols.push_back(c);
                a.push_back((void*)at);
                b.push_back((void*)(at + (1 << 20)));
                at += 1 << 22;
                if (r) ++(std::min(r, c) <= kPad ? n_small : n_large);
            }
            adamw_tensor_list l{};
            l.n_tensors = (int64_t)numel.size();
            l.numel = numel.data();
            l.ptr[0] = a.data();
            l.ptr[1] = b.data();
            l.shard_end = -1;
            NsKind kind{};
            kind.end = kEndOrtho;
            kind.in = ADAMW_F32;
            kind.esz[0] = 2;
            kind.esz[1] = 4;
            std::string err;
            int64_t bytes = 0;
            CHECK(ns_workspace_bytes(&l, cols.data(), least != 0, &bytes, err) == ADAMW_OK);
            NsPlan p;
            CHECK(build_ns_plan(kind, &l, cols.data(), 0, 0x600000000000ull, bytes, &p, err) == ADAMW_OK);
            CHECK((p.small != nullptr) == (n_small && n_large));
            const size_t own = p.batches.size();
            if (!least) CHECK(own <= 1 && (!p.small || p.small->batches.size() == 1));
            p.flatten();
            CHECK(!p.small && (int)p.mats.size() == n_small + n_large);
            std::set<uint32_t> seen;
            for (const NsBatch& x : p.batches)
                if (check(p, x, seen, bytes)) return 1;
            CHECK(seen.size() == p.mats.size());
        }
    puts("mixed ok 0");
    return 0;
}
"""


def test_small_matrices_have_batches_of_their_own(tmp_path):
    src = tmp_path / "mixed.cpp"
    src.write_text(MIXED)
    base = ["g++", "-std=c++17", "-Wall", "-Wextra", "-I", os.path.join(ROOT, "include"), "-I", CSRC] + SAN
    _build_and_run(base + [str(src)] + [os.path.join(CSRC, f) for f in ("muon_plan.cpp", "plan.cpp", "validate.cpp")],
                   str(tmp_path / "mixed"), "mixed")
