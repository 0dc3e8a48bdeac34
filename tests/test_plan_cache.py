"""The plan-cache policy of a stream (CPU): tests/native/cache_check.cpp simulates training
loops over up to 32 parameter groups with a norm, a clipping, a check and a step each, lists
that come once, captured lists and long keys, under AddressSanitizer and
UndefinedBehaviorSanitizer."""
import os

from test_sanitizers import CSRC, NATIVE, ROOT, SAN, _build_and_run


def test_cache_policy(tmp_path):
    srcs = [os.path.join(NATIVE, "cache_check.cpp"), os.path.join(CSRC, "plan.cpp")]
    _build_and_run(["g++", "-std=c++17", "-Wall", "-Wextra", "-I", os.path.join(ROOT, "include"), "-I", CSRC, *SAN, *srcs],
                   str(tmp_path / "cache_check"), "cache_check")
