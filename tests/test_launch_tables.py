"""The tables that the update kernels receive and the maps from workgroup and lane to
elements (CPU): tests/native/launch_check.cpp walks every workgroup and lane of 240 random
lists in five launch forms each, built with and without the sanitizers; and the table itself
(adamw_plan_inspect_bytes, for_check 4) is held against the caller's buffers for the bench's
own layouts and random lists."""
import os

import numpy as np
import pytest

import adamw_optimizer_step_apply_amd as A
import test_plan_bounds as bounds
import workloads
from test_sanitizers import CSRC, NATIVE, ROOT, SAN, _build_and_run


def test_every_element_is_taken_once(tmp_path):
    srcs = [os.path.join(NATIVE, "launch_check.cpp"), os.path.join(CSRC, "plan.cpp")]
    base = ["g++", "-std=c++17", "-Wall", "-Wextra", "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    with_san = _build_and_run(base + SAN + srcs, str(tmp_path / "launch_check_san"), "launch_check")
    plain = _build_and_run(base + ["-O3"] + srcs, str(tmp_path / "launch_check"), "launch_check")
    assert with_san == plain


def check_launch(spec, code, dt, prec=None):
    """The items that the step's workgroups take (for_check 4) against every element's
    address in the layout the caller handed in, as check_plan does for the plan's chunks."""
    rows, rng = A.adamw_plan_inspect_bytes(code, dt, spec.tensor_list(), 4, prec)
    rng = rng.astype(np.int64)
    t, off, cnt, kind, flat = rows[:, 0], rows[:, 1], rows[:, 2], rows[:, 3], rows[:, 4]
    vec, head, parts = (kind & 1).astype(bool), kind >> 4 & 7, kind >> 8
    body = np.where(vec, (cnt - head) // 8 * 8, 0)
    assert np.all(cnt > 0) and np.all(body[vec] > 0) and np.all(cnt - body - np.where(vec, head, 0) < np.where(vec, 8, 4097))
    assert np.array_equal(flat, spec.start[t] + off)
    # 8 workgroups for the first items, one for the short ones after them
    assert np.all(np.isin(parts, (1, 8))) and np.all(np.diff(parts) <= 0)
    assert np.all(cnt[parts == 1] <= 4096)
    t_own, lo_own, hi_own = spec.owned_intervals()
    for s in range(5):
        e = spec.esz[s]
        lo, hi = rng[:, s, 0], rng[:, s, 1]
        if e == 0:
            assert not lo.any() and not hi.any()
            continue
        assert np.array_equal(lo, spec.addr(s, t, flat)) and np.array_equal(hi - lo, cnt * e)
        assert np.all((lo + head * e)[vec] % 16 == 0), f"stream {s}: vector part not 16-byte aligned"
        if spec.kind(s) == "blocked":
            assert np.all((flat - spec.b) % bounds.B + cnt <= bounds.B), f"stream {s}: item crosses a state block"
        got = bounds.merge(lo, hi)
        start = spec.addr(s, t_own, lo_own)
        want = bounds.merge(start, start + (hi_own - lo_own) * e)
        assert all(np.array_equal(a, b) for a, b in zip(got, want)), f"stream {s}: bytes differ from the owned elements'"
    return rows


@pytest.mark.parametrize("mode", ["mixed-blocked", "mixed"])
def test_ragged_10k_as_the_bench_lays_it_out(mode):
    wl = workloads.get("ragged_10k")
    rows = check_launch(bounds.bench_spec(mode, wl.numels, bounds.ESZ[("mixed", "f16")]), A.MIXED, A.F16)
    assert (rows[:, 3] >> 8 == 1).sum() > 5000


@pytest.mark.parametrize("mode", ["mixed", "kahan", "split"])
@pytest.mark.parametrize("blocked", [True, False])
def test_opt_1_3b_as_the_bench_lays_it_out(mode, blocked):
    wl = workloads.get("opt_1_3b")
    spec = bounds.bench_spec(mode + ("-blocked" if blocked else ""), wl.numels, bounds.ESZ[(mode, "bf16")])
    check_launch(spec, bounds.CODE[mode], A.BF16)


def test_random_lists():
    rng = np.random.default_rng(np.random.SeedSequence([9, 200]))
    shared = 0
    for _ in range(200):
        spec, kind, dt, prec = bounds._random_spec(rng)
        if kind == "check":
            continue
        rows = check_launch(spec, bounds.CODE.get(kind, A.MIXED), bounds.DT[dt], prec)
        plan, _ = A.adamw_plan_inspect_bytes(bounds.CODE.get(kind, A.MIXED), bounds.DT[dt], spec.tensor_list(), False, prec)
        wide = kind == "mixed" or (prec is not None and spec.esz[2:] == (4, 4, 4))
        if 8 * len(plan) <= (512 if wide else 1024):     # the card holds the list whole: taken as planned
            shared += len(plan) > 0
            assert np.all(rows[:, 3] >> 8 == 8) and np.array_equal(rows[:, [0, 1, 2, 4, 5]], plan[:, [0, 1, 2, 4, 5]])
        else:
            assert len(rows) <= len(plan)
    assert shared > 20


def test_introspection_of_the_launch_belongs_to_the_byte_form():
    tl = A.TensorList([10], [[4096 + (s << 20)] for s in range(5)])
    with pytest.raises(A.AdamWError, match="inspect_bytes"):
        A.adamw_plan_inspect(A.MIXED, A.BF16, tl, 4)
    rows, _ = A.adamw_plan_inspect_bytes(A.MIXED, A.BF16, tl, 4)
    assert rows[:, :4].tolist() == [[0, 0, 8, 8 * 256 + 1], [0, 8, 2, 8 * 256]]
