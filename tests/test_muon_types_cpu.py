"""Tensors of a type that a call on matrices would read as another one are refused by the binding, on the CPU: fp16 words
taken for bf16 are finite numbers, and nothing would show."""
import pytest
import torch

import adamw_optimizer_step_apply_amd as A

WS = (0x600000000000, 1 << 34)     # never dereferenced
STEP = 0x7f0000000000
F32, BF, F16, I16, I32 = torch.float32, torch.bfloat16, torch.float16, torch.int16, torch.int32


@pytest.fixture(autouse=True)
def as_if_on_the_gpu(monkeypatch):
    """The types are what is tested: places and sizes are looked at before, the library is called after."""
    check = A._check_types

    def seen(matrices, types):
        check(matrices, types)
        raise RuntimeError("passed")
    monkeypatch.setattr(A, "_check_streams", lambda matrices, sizes: None)
    monkeypatch.setattr(A, "_check_types", seen)


def of(*dtypes):
    return A.MatrixList([(6, 8)], [None if t is None else [torch.zeros(6, 8, dtype=t)] for t in dtypes])


def outcome(ok):
    return pytest.raises(RuntimeError if ok else ValueError, match="passed" if ok else "tensors are needed")


@pytest.mark.parametrize("dtypes,code,ok", [
    ((BF, F32), A.F32, True), ((BF, BF), A.BF16, True), ((BF, F16), A.F16, True), ((I16, I16), A.F16, True), ((BF, I32), A.F32, True),
    ((F16, F32), A.F32, False), ((BF, F16), A.BF16, False), ((BF, BF), A.F16, False)])
def test_orthogonalize(dtypes, code, ok):
    with outcome(ok):
        A.adamw_orthogonalize(code, of(*dtypes), WS, stream=0)


@pytest.mark.parametrize("mode,p_dtype,prec,dtypes,ok", [
    (A.MIXED, A.BF16, None, (BF, BF, F32, None, F32), True), (A.MIXED, A.F16, None, (F16, F16, F32, None, F32), True),
    (A.MIXED, A.BF16, None, (BF, F16, F32, None, F32), False), (A.MIXED, A.F16, None, (F16, BF, F32, None, F32), False),
    (A.MIXED, A.F16, None, (BF, F16, F32, None, F32), False), (A.MIXED, A.BF16, None, (I16, I16, I32, None, I32), True),
    (A.MIXED_SPLIT, A.BF16, None, (BF, BF, F32, None, I16), True), (A.MIXED_SPLIT, A.BF16, None, (BF, BF, F32, None, BF), False),
    (A.MIXED_SPLIT, A.BF16, None, (F16, BF, F32, None, I16), False), (A.PURE_KAHAN, A.BF16, None, (BF, BF, BF, None, BF), True),
    (A.PURE_KAHAN, A.BF16, None, (BF, BF, F16, None, BF), False), (A.PURE_KAHAN, A.BF16, None, (BF, BF, BF, None, F16), False),
    (A.MIXED, A.F16, A.PurePrecision(A.F32, A.BF16, A.KAHAN_F32), (BF, BF, F32, None, F32), True),
    (A.MIXED, A.F16, A.PurePrecision(A.BF16, A.BF16, A.KAHAN_NONE), (BF, BF, BF), True),
    (A.MIXED, A.F16, A.PurePrecision(A.BF16, A.BF16, A.KAHAN_NONE), (F16, F16, BF), False),
    (A.MIXED, A.F16, A.PurePrecision(A.BF16, A.BF16, A.KAHAN_BF16), (BF, BF, BF, None, F16), False)])
def test_step(mode, p_dtype, prec, dtypes, ok):
    with outcome(ok):
        A.adamw_muon_multi_tensor_step(mode, p_dtype, of(*dtypes), None, STEP, WS, prec=prec, stream=0)
