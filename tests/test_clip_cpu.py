"""Clipping without a GPU: bad calls are refused before any HIP call."""
import ctypes

import pytest

import adamw_optimizer_step_apply_amd as A
from test_grad_norm_cpu import FAKE, grads


def clip(**kw):
    return A.GradClip(**{"d_sumsq": FAKE, **kw})


@pytest.mark.parametrize("call,needle", [
    (lambda: A.adamw_clip_grads(7, grads([10]), clip(), stream=0), "g_dtype"),
    (lambda: A.adamw_clip_grads(A.BF16, grads([10]), clip(d_sumsq=0), stream=0), "d_sumsq"),
    (lambda: A.adamw_clip_grads(A.BF16, grads([10]), clip(d_sumsq=FAKE + 4), stream=0), "8-byte"),
    (lambda: A.adamw_clip_grads(A.BF16, grads([10]), clip(max_norm=-1.0), stream=0), "max_norm"),
    (lambda: A.adamw_clip_grads(A.BF16, grads([10]), clip(max_norm=float("inf")), stream=0), "max_norm"),
    (lambda: A.adamw_clip_grads(A.BF16, grads([10]), clip(max_norm=float("nan")), stream=0), "max_norm"),
    (lambda: A.adamw_clip_grads(A.BF16, grads([10]), clip(eps=-1e-6), stream=0), "eps"),
    (lambda: A.adamw_clip_grads(A.BF16, grads([10]), clip(eps=float("nan")), stream=0), "eps"),
    (lambda: A.adamw_clip_grads(A.BF16, grads([10]), clip(), 0.0, stream=0), "inv_loss_scale"),
    (lambda: A.adamw_clip_grads(A.BF16, grads([10]), clip(), float("inf"), stream=0), "inv_loss_scale"),
    (lambda: A.adamw_clip_grads(A.BF16, grads([10]), clip(), d_scale=FAKE + 2, stream=0), "d_scale"),
    (lambda: A.adamw_clip_grads(A.BF16, grads([10], base=FAKE + 1), clip(), stream=0), "aligned"),
    (lambda: A.adamw_clip_grads(A.BF16, grads([10, 3], shard_begin=0, shard_end=14), clip(), stream=0), "shard"),
    (lambda: A.adamw_clip_grads(A.BF16, grads([10, -3]), clip(), stream=0), "numel"),
])
def test_rejected_before_any_hip_call(call, needle):
    with pytest.raises(A.AdamWError) as ei:
        call()
    assert ei.value.status in (A.E_INVALID, A.E_UNSUPPORTED)
    assert needle.lower() in str(ei.value).lower(), str(ei.value)


def test_null_clip_is_refused():
    tl = grads([10])
    assert A._lib.adamw_clip_grads(A.BF16, ctypes.byref(tl.c), None, 1.0, None, None) == A.E_INVALID
    assert "clip" in A.adamw_last_error()


@pytest.mark.parametrize("call", [lambda: A.adamw_clip_grads(A.F32, grads([10, 20], esz=4), clip(max_norm=0.0), stream=0),
                                  lambda: A.adamw_clip_grads(A.F16, grads([10]), clip(), 0.0, FAKE, stream=0)])
def test_valid_call_reaches_hip(call):
    with pytest.raises(A.AdamWError) as ei:
        call()
    assert ei.value.status == A.E_HIP


def test_binding_struct_matches_the_c_layout(tmp_path):
    import os
    import subprocess
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "adamw.h"\n'
                   'int main(void) { printf("%zu %zu %zu %zu\\n", sizeof(adamw_grad_clip), '
                   'offsetof(adamw_grad_clip, d_sumsq), offsetof(adamw_grad_clip, max_norm), '
                   'offsetof(adamw_grad_clip, eps)); return 0; }\n')
    exe = tmp_path / "layout"
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-I", inc, str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    s = A.adamw_grad_clip
    assert got == [ctypes.sizeof(s), s.d_sumsq.offset, s.max_norm.offset, s.eps.offset]


def _tl(numels, base=FAKE, esz=(2, 2, 4, 4, 4)):
    import numpy as np
    offs = np.concatenate([[0], np.cumsum(numels)[:-1]])
    return A.TensorList(numels, [[base + s * (1 << 36) + int(o) * esz[s] for o in offs] for s in range(5)])


def step(mode=A.MIXED, dt=A.BF16, tl=None, hp=None, c=None, d_step=FAKE, **kw):
    A.adamw_multi_tensor_step_clipped(mode, dt, tl or _tl([10]), hp or A.HParams(), c or clip(), d_step, stream=0, **kw)


@pytest.mark.parametrize("call,needle", [
    (lambda: step(dt=A.F32), "p_dtype"),
    (lambda: step(mode=9), "mode"),
    (lambda: step(c=clip(d_sumsq=0)), "d_sumsq"),
    (lambda: step(c=clip(d_sumsq=FAKE + 4)), "8-byte"),
    (lambda: step(c=clip(max_norm=-0.5)), "max_norm"),
    (lambda: step(c=clip(max_norm=float("inf"))), "max_norm"),
    (lambda: step(c=clip(eps=float("inf"))), "eps"),
    (lambda: step(hp=A.HParams(beta1=1.0)), "beta"),
    (lambda: step(d_step=0), "d_step"),
    (lambda: step(d_step=FAKE + 2), "aligned"),
    (lambda: step(d_found_inf=FAKE + 1), "aligned"),
    (lambda: step(d_scale=FAKE + 2), "d_scale"),
    (lambda: step(d_scale=FAKE, scaler=A.LossScaler(0.5, 0.5, 10)), "growth_factor"),
    (lambda: step(d_scale=FAKE, scaler=A.LossScaler(2.0, 0.5, 0)), "growth_interval"),
    (lambda: step(prec=A.PurePrecision(A.F16, A.BF16, 1)), "exp_avg"),
    (lambda: step(tl=_tl([10], base=FAKE + 1)), "aligned"),
    (lambda: step(tl=A.TensorList([10], [[FAKE], None, [FAKE], [FAKE], [FAKE]])), "grad"),
])
def test_step_rejected_before_any_hip_call(call, needle):
    with pytest.raises(A.AdamWError) as ei:
        call()
    assert ei.value.status in (A.E_INVALID, A.E_UNSUPPORTED)
    assert needle.lower() in str(ei.value).lower(), str(ei.value)


@pytest.mark.parametrize("kw", [{}, {"mode": A.PURE_KAHAN, "tl": _tl([10], esz=(2,) * 5)}, {"d_scale": FAKE, "dt": A.F16},
                                {"d_scale": FAKE, "advance_scale": False, "scaler": A.LossScaler(2.0, 0.5, 0)}])
def test_valid_step_reaches_hip(kw):
    with pytest.raises(A.AdamWError) as ei:
        step(**kw)
    assert ei.value.status == A.E_HIP


@pytest.mark.parametrize("dt,esz", [(A.BF16, 2), (A.F32, 4)])
@pytest.mark.parametrize("phase", [0, 1, 3])
def test_plan_covers_the_list(dt, esz, phase):
    """Chunks of 128 KiB, each but a piece's first starting at a 16-byte edge."""
    chunk = 131072 // esz
    numels = [0, 1, 7, chunk - 1, chunk, chunk + 1, 5, 3 * chunk + 17, 2 ** 32 + 5]
    tl = grads(numels, FAKE + phase * esz, esz)
    rows, ranges = A.adamw_plan_inspect_bytes(A.MIXED, dt, tl, for_check=3)
    pos = {}
    for (t, off, n, kind, _, _), r in zip(rows[:, :6].tolist(), ranges.tolist()):
        assert kind == 2 and off == pos.get(t, 0) and 0 < n <= chunk + 16 // esz - 1
        lo, hi = r[1]
        assert hi - lo == n * esz and lo == tl.c.ptr[1][t] + off * esz and (off == 0 or lo % 16 == 0)
        pos[t] = off + n
    assert pos == {t: n for t, n in enumerate(numels) if n}


def test_plan_beyond_the_grid_limit_is_refused():
    """A chunk shared by 8 workgroups: at most (2^32 - 1) / 256 / 8 chunks."""
    n = 2_097_151 * 65536
    assert len(A.adamw_plan_inspect_bytes(A.MIXED, A.BF16, grads([n]), for_check=3)[0]) == 2_097_151
    with pytest.raises(A.AdamWError, match="chunks"):
        A.adamw_clip_grads(A.BF16, grads([n + 1]), clip(), stream=0)


@pytest.mark.parametrize("tl", [
    A.TensorList([10, 10], [None, [FAKE, FAKE]]),
    A.TensorList([10, 4, 10], [None, [FAKE, FAKE + 4096, FAKE + 18]]),
    A.TensorList([10, 4, 10], [None, [FAKE + 2, FAKE + 4096, FAKE]], 0, 17),
], ids=["twice", "by one", "inside the shard"])
def test_overlapping_buffers_are_refused(tl):
    with pytest.raises(A.AdamWError, match="overlap"):
        A.adamw_clip_grads(A.BF16, tl, clip(), stream=0)
    with pytest.raises(A.AdamWError) as ei:          # the norm only reads: an element listed twice counts twice
        A.adamw_grad_norm(A.BF16, tl, FAKE, stream=0)
    assert ei.value.status == A.E_HIP


@pytest.mark.parametrize("tl", [
    A.TensorList([10, 10], [None, [FAKE + 20, FAKE]]),
    A.TensorList([0, 10, 0], [None, [FAKE, FAKE, FAKE + 2]]),
    A.TensorList([10, 10], [None, [FAKE, FAKE]], 0, 10),
    A.TensorList([10, 10], [None, [FAKE, FAKE]], 5, 15),
    A.TensorList([10, 10], [None, [FAKE]], 0, 20, 2),
], ids=["touching", "empty", "outside the shard", "split", "flat"])
def test_disjoint_buffers_are_not(tl):
    with pytest.raises(A.AdamWError) as ei:
        A.adamw_clip_grads(A.BF16, tl, clip(), stream=0)
    assert ei.value.status == A.E_HIP


def test_no_exception_leaves_the_c_entries():
    """A count of tensors that no host array can have comes back as a status."""
    tl = grads([10])
    tl.c.n_tensors = 2 ** 61
    c, h, sc = clip().c(), A.HParams().c(), A.LossScaler().c()
    lib = A._lib
    assert lib.adamw_grad_norm(A.BF16, ctypes.byref(tl.c), 0, FAKE, None, None, None) == A.E_NOMEM
    assert lib.adamw_tensor_norms(A.BF16, ctypes.byref(tl.c), None, FAKE, None, None) in (A.E_NOMEM, A.E_INVALID)
    assert lib.adamw_clip_grads(A.BF16, ctypes.byref(tl.c), ctypes.byref(c), 1.0, None, None) == A.E_NOMEM
    assert lib.adamw_multi_tensor_step_clipped(A.MIXED, A.BF16, None, ctypes.byref(tl.c), ctypes.byref(h), ctypes.byref(c),
                                               FAKE, None, None, ctypes.byref(sc), None) == A.E_NOMEM


def test_results_of_another_type_or_place_are_refused():
    """The binding hands the library no buffer that it would write past."""
    import torch
    d, f, i = torch.float64, torch.float32, torch.int32
    for call in (lambda: A.adamw_grad_norm(A.BF16, grads([10]), torch.zeros(1, dtype=d), stream=0),
                 lambda: A.adamw_grad_norm(A.BF16, grads([10]), torch.zeros(1, dtype=f, device="meta"), stream=0),
                 lambda: A.adamw_grad_norm(A.BF16, grads([10]), FAKE, torch.zeros(1, dtype=f), stream=0),
                 lambda: A.adamw_grad_norm(A.BF16, grads([10]), FAKE, None, torch.zeros(1, dtype=i), stream=0),
                 lambda: A.adamw_tensor_norms(A.BF16, grads([10, 2]), torch.zeros(2, dtype=f), stream=0),
                 lambda: A.adamw_clip_grads(A.BF16, grads([10]), clip(d_sumsq=torch.zeros(1, dtype=f)), stream=0),
                 lambda: step(c=clip(d_sumsq=torch.zeros(1, dtype=d)))):
        with pytest.raises(ValueError, match="is needed, got"):
            call()
