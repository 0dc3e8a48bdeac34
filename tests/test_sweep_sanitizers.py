"""The planner of the gradient norms and of clipping, and the update kernels' tables,
under AddressSanitizer and UndefinedBehaviorSanitizer (CPU only):
tests/native/sweep_check.cpp over 5,000 random lists, built with and without the sanitizers; both print the same checksum."""
import os

from test_sanitizers import CSRC, NATIVE, ROOT, SAN, _build_and_run


def test_sweep_planner_under_sanitizers(tmp_path):
    srcs = [os.path.join(NATIVE, "sweep_check.cpp"), os.path.join(CSRC, "plan.cpp"), os.path.join(CSRC, "validate.cpp")]
    base = ["g++", "-std=c++17", "-Wall", "-Wextra", "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    with_san = _build_and_run(base + SAN + srcs, str(tmp_path / "sweep_check_san"), "sweep_check")
    plain = _build_and_run(base + ["-O3"] + srcs, str(tmp_path / "sweep_check"), "sweep_check")
    assert with_san == plain
