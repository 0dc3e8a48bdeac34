"""The Newton-Schulz products and the Muon step without a GPU: what is refused before any HIP call, the binding's
structures, workspace sizes, and the planner under the sanitizers (tests/native/muon_check.cpp over 1,500 random lists)."""
import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

import adamw_optimizer_step_apply_amd as A
from test_sanitizers import CSRC, NATIVE, ROOT, SAN, _build_and_run

FAKE, WS = 0x7f0000000000, (0x600000000000, 1 << 34)     # never dereferenced
HEADER = os.path.join(ROOT, "include", "adamw.h")


def test_planner_under_sanitizers(tmp_path):
    srcs = [os.path.join(NATIVE, "muon_check.cpp")] + [os.path.join(CSRC, f) for f in ("muon_plan.cpp", "plan.cpp", "validate.cpp")]
    base = ["g++", "-std=c++17", "-Wall", "-Wextra", "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    with_san = _build_and_run(base + SAN + srcs, str(tmp_path / "muon_check_san"), "muon_check")
    plain = _build_and_run(base + ["-O3"] + srcs, str(tmp_path / "muon_check"), "muon_check")
    assert with_san == plain


def test_structures_and_constants_match_the_header(tmp_path):
    src = tmp_path / "layout.c"
    fields = [f"adamw_newton_schulz, {n}" for n, _ in A.adamw_newton_schulz._fields_]
    fields += [f"adamw_muon_hparams, {n}" for n, _ in A.adamw_muon_hparams._fields_]
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "adamw.h"\nint main(void)\n{\n' +
                   "".join(f'    printf("%zu\\n", offsetof({f}));\n' for f in fields) +
                   '    printf("%zu\\n%zu\\n", sizeof(adamw_newton_schulz), sizeof(adamw_muon_hparams));\n' +
                   '    printf("%d %d %d %d\\n", ADAMW_MUON_SCALE_NONE, ADAMW_MUON_SCALE_SPECTRAL, ADAMW_MUON_SCALE_RMS, '
                   'ADAMW_NS_MAX_STEPS);\n    return 0;\n}\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-I", os.path.dirname(HEADER), str(src), "-o", str(tmp_path / "l")], check=True)
    out = subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout.split()
    want = [getattr(A.adamw_newton_schulz, n).offset for n, _ in A.adamw_newton_schulz._fields_]
    want += [getattr(A.adamw_muon_hparams, n).offset for n, _ in A.adamw_muon_hparams._fields_]
    want += [ctypes.sizeof(A.adamw_newton_schulz), ctypes.sizeof(A.adamw_muon_hparams), A.MUON_SCALE_NONE,
             A.MUON_SCALE_SPECTRAL, A.MUON_SCALE_RMS, A.NS_MAX_STEPS]
    assert [int(x) for x in out] == want
    assert re.search(r"ADAMW_NS_MAX_STEPS = (\d+)", open(HEADER).read()).group(1) == str(A.NS_MAX_STEPS)


def mats(shapes, streams=(2, 2, 4, 0, 4), base=FAKE, **kw):
    rows, at = [], base
    for esz in streams:
        row = []
        for r, c in shapes:
            row.append(at)
            at += -(-r * c * esz // 256) * 256
        rows.append(row if esz else None)
    return A.MatrixList(shapes, rows, **kw)


SHAPES = [(64, 100), (100, 64), (7, 9)]


def ortho(m=None, dtype=A.BF16, ws=WS, ns=None):
    A.adamw_orthogonalize(dtype, m or mats(SHAPES, (2, 2, 0, 0, 0)), ws, ns, stream=0)


def step(m=None, mode=A.MIXED, p_dtype=A.BF16, hp=None, d_step=FAKE - 4096, ws=WS, **kw):
    A.adamw_muon_multi_tensor_step(mode, p_dtype, m or mats(SHAPES), hp, d_step, ws, stream=0, **kw)


def cols_of(m, i, c):
    m.cols[i] = c
    return m


NS, HP = A.NewtonSchulz, A.MuonHParams
REFUSED = [
    (lambda: ortho(dtype=7), "u_dtype"),
    (lambda: ortho(ns=NS(steps=0)), "steps"),
    (lambda: ortho(ns=NS(steps=17)), "steps"),
    (lambda: ortho(ns=NS(eps=-1.0)), "eps"),
    (lambda: ortho(ns=NS(eps=math.inf)), "finite"),
    (lambda: ortho(ns=NS(a=math.nan)), "finite"),
    (lambda: ortho(ns=NS(a=100.0)), "past 64"),
    (lambda: ortho(ns=NS(2.0, 1.0, 1.0, steps=5)), "past 64"),
    (lambda: ortho(ws=(0, 1 << 30)), "workspace is null"),
    (lambda: ortho(ws=(WS[0] + 128, 1 << 30)), "256-byte"),
    (lambda: ortho(ws=(WS[0], 4096)), "largest matrix needs"),
    (lambda: ortho(ws=(WS[0], -1)), "largest matrix needs"),
    (lambda: ortho(ws=(FAKE - (FAKE % 256), 1 << 30)), "overlap"),
    (lambda: ortho(cols_of(mats(SHAPES, (2, 2, 0, 0, 0)), 1, 63)), "does not divide"),
    (lambda: ortho(cols_of(mats(SHAPES, (2, 2, 0, 0, 0)), 1, 0)), "does not divide"),
    (lambda: ortho(cols_of(mats(SHAPES, (2, 2, 0, 0, 0)), 1, -64)), "does not divide"),
    (lambda: ortho(A.MatrixList([(8, 8)], [None, [FAKE]])), "param"),
    (lambda: ortho(A.MatrixList([(8, 8)], [[FAKE], None])), "grad"),
    (lambda: ortho(A.MatrixList([(8, 8)], [[FAKE + 1], [FAKE + 4096]])), "aligned"),
    (lambda: ortho(A.MatrixList([(8, 8)], [[FAKE], [FAKE + 4098]]), A.F32), "aligned"),
    (lambda: ortho(A.MatrixList([(8, 8)], [[FAKE], [FAKE + 64]])), "overlap"),
    (lambda: ortho(A.MatrixList([(8, 8)], [[FAKE], [FAKE]]), A.F32), "overlap"),
    (lambda: ortho(A.MatrixList([(8, 8)], [[FAKE], [FAKE]]), A.F16), "overlap"),
    (lambda: ortho(A.MatrixList([(8, 8), (8, 8)], [[FAKE, FAKE], [FAKE + 4096, FAKE + 8192]])), "overlap"),
    (lambda: ortho(A.MatrixList([(8, 8), (8, 8)], [[FAKE, FAKE + 4096], [FAKE + 4096, FAKE]])), "overlap"),
    (lambda: ortho(A.MatrixList([(1 << 31, 1)], [[FAKE], [FAKE + (1 << 40)]]), ws=(WS[0], 1 << 44)), "larger than"),
    (lambda: ortho(A.MatrixList([((1 << 20) + 1, (1 << 20) + 1)], [[FAKE], [FAKE + (1 << 44)]]), ws=(WS[0], 1 << 46)), "larger than"),
    (lambda: ortho(A.MatrixList([(1 << 20, 1 << 20)], [[FAKE], [FAKE + (1 << 44)]]), ws=(1 << 50, 1 << 47)), "tiles"),
    (lambda: ortho(mats(SHAPES, (2, 2, 0, 0, 0), shard_begin=1)), "in part"),
    (lambda: ortho(mats(SHAPES, (2, 2, 0, 0, 0), shard_end=6399)), "in part"),
    (lambda: ortho(mats(SHAPES, (2, 2, 0, 0, 0), shard_end=10 ** 6)), "shard range"),
    (lambda: ortho(mats(SHAPES, (2, 2, 0, 0, 0), flat_mask=A.BLOCKED_STATE)), "blocked"),
    (lambda: ortho(mats(SHAPES, (2, 2, 0, 0, 0), flat_mask=1 << 20)), "unknown bits"),
    (lambda: step(mode=9), "mode"),
    (lambda: step(p_dtype=A.F32), "p_dtype"),
    (lambda: step(mode=A.MIXED_SPLIT, p_dtype=A.F16), "p_dtype"),
    (lambda: step(mode=A.PURE_KAHAN, p_dtype=A.F16), "p_dtype"),
    (lambda: step(prec=A.PurePrecision(A.F16, A.BF16, 1)), "dtype"),
    (lambda: step(prec=A.PurePrecision(A.BF16, A.BF16, 3)), "kahan"),
    (lambda: step(hp=HP(lr=-1.0)), "lr"),
    (lambda: step(hp=HP(lr=math.inf)), "finite"),
    (lambda: step(hp=HP(momentum=1.0)), "momentum"),
    (lambda: step(hp=HP(momentum=-0.1)), "momentum"),
    (lambda: step(hp=HP(weight_decay=-0.1)), "weight_decay"),
    (lambda: step(hp=HP(inv_loss_scale=0.0)), "inv_loss_scale"),
    (lambda: step(hp=HP(nesterov=2)), "nesterov"),
    (lambda: step(hp=HP(scaling=3)), "scaling"),
    (lambda: step(hp=HP(ns=NS(steps=-1))), "steps"),
    (lambda: step(d_step=0), "d_step"),
    (lambda: step(d_step=FAKE + 2), "aligned"),
    (lambda: step(d_found_inf=FAKE + 2), "aligned"),
    (lambda: step(d_scale=FAKE + 2), "aligned"),
    (lambda: step(clip=A.GradClip(0)), "d_sumsq"),
    (lambda: step(clip=A.GradClip(FAKE + 4)), "d_sumsq"),
    (lambda: step(clip=A.GradClip(FAKE, max_norm=-1.0)), "max_norm"),
    (lambda: step(ws=(WS[0], 4096)), "largest matrix needs"),
    (lambda: step(A.MatrixList([(8, 8)], [[FAKE], [FAKE + 4096], [FAKE + 8192], None, None])), "aux"),
    (lambda: step(A.MatrixList([(8, 8)], [[FAKE], [FAKE + 4096], None, None, [FAKE + 8192]])), "exp_avg"),
    (lambda: step(A.MatrixList([(8, 8)], [[FAKE], [FAKE + 4096], [FAKE + 8192], None, [FAKE + 8192]])), "overlap"),
    (lambda: step(A.MatrixList([(8, 8)], [[FAKE], [FAKE], [FAKE + 8192], None, [FAKE + 16384]])), "overlap"),
]


@pytest.mark.parametrize("k", range(len(REFUSED)))
def test_refused_before_any_hip_call(k):
    call, needle = REFUSED[k]
    with pytest.raises(A.AdamWError) as e:
        call()
    assert e.value.status in (A.E_INVALID, A.E_UNSUPPORTED), str(e.value)
    assert needle in str(e.value), str(e.value)


@pytest.mark.parametrize("call", [ortho, step, lambda: ortho(A.MatrixList([(8, 8)], [[FAKE], [FAKE]])),
                                  lambda: step(mode=A.MIXED_SPLIT, m=mats(SHAPES, (2, 2, 4, 0, 2))),
                                  lambda: step(prec=A.PurePrecision(A.F32, A.F32, A.KAHAN_NONE), m=mats(SHAPES, (2, 2, 4, 0, 0)))])
def test_valid_calls_reach_hip(call):
    """Validation passes; only the first HIP call fails on a host without a GPU."""
    with pytest.raises(A.AdamWError) as e:
        call()
    assert e.value.status == A.E_HIP


def test_matrix_list_checks_its_tensors():
    t = torch.zeros(6, 8, dtype=torch.bfloat16)
    A.MatrixList([(6, 8)], [[t], [t]])
    with pytest.raises(ValueError, match="contiguous"):
        A.MatrixList([(8, 6)], [[t.T], [t]])
    with pytest.raises(ValueError, match="no matrix"):
        A.MatrixList([(6, 9)], [[t], [t]])
    with pytest.raises(ValueError, match="device="):
        A.make_orthogonalize_workspace(A.MatrixList([(6, 8)], [[FAKE], [FAKE]]))
    with pytest.raises(ValueError, match="contiguous"):
        A.adamw_orthogonalize(A.BF16, A.MatrixList([(6, 8)], [[t], [t]]), torch.zeros(64, 64, dtype=torch.uint8).T, stream=0)


def test_workspace_bytes():
    one = A.adamw_orthogonalize_workspace_bytes(mats([(2048, 2048)]))
    # three fp16 copies of the matrix and two squares, diagonals and partial sums
    assert 10 * 2048 ** 2 <= one <= 10.1 * 2048 ** 2
    many = A.adamw_orthogonalize_workspace_bytes(mats([(2048, 2048)] * 16))
    assert 15 * one < many <= 16 * one
    assert A.adamw_orthogonalize_workspace_bytes(mats([(2048, 2048)] * 16), least=True) == one
    assert A.adamw_orthogonalize_workspace_bytes(mats([(2048, 2048)] * 1000)) == (4 << 30) + 256
    assert A.adamw_orthogonalize_workspace_bytes(mats([(65536, 65536)])) > 10 * 65536 ** 2
    assert A.adamw_orthogonalize_workspace_bytes(A.MatrixList([], [[]])) >= 256
    with pytest.raises(A.AdamWError):
        A.adamw_orthogonalize_workspace_bytes(cols_of(mats(SHAPES), 0, 3))
