"""The tables that the update kernels receive and the maps from workgroup and lane to
elements (CPU): tests/native/launch_check.cpp walks every workgroup and lane of 240 random
lists in five launch forms each, built with and without the sanitizers."""
import os

from test_sanitizers import CSRC, NATIVE, ROOT, SAN, _build_and_run


def test_every_element_is_taken_once(tmp_path):
    srcs = [os.path.join(NATIVE, "launch_check.cpp"), os.path.join(CSRC, "plan.cpp")]
    base = ["g++", "-std=c++17", "-Wall", "-Wextra", "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    with_san = _build_and_run(base + SAN + srcs, str(tmp_path / "launch_check_san"), "launch_check")
    plain = _build_and_run(base + ["-O3"] + srcs, str(tmp_path / "launch_check"), "launch_check")
    assert with_san == plain
