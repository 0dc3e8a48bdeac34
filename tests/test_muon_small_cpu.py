"""The runs of columns of small gram, on the CPU."""
import os
import subprocess

from test_sanitizers import CSRC, ROOT

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
