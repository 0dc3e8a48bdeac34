"""Tensors that would make a call on matrices read or write outside them are refused by the binding, on the CPU."""
import pytest
import torch

import adamw_optimizer_step_apply_amd as A

WS = (0x600000000000, 1 << 34)     # never dereferenced
STEP = 0x7f0000000000


def of(*dtypes):
    return A.MatrixList([(6, 8)], [None if t is None else [torch.zeros(6, 8, dtype=t)] for t in dtypes])


@pytest.fixture(autouse=True)
def as_if_on_the_gpu(request, monkeypatch):
    """The sizes are what is tested, so the device check sees what a GPU tensor would say."""
    if "host" in request.node.name:
        return
    check = A._check_streams

    def seen(matrices, sizes):
        matrices._kinds = [{(size, True) for size, _ in k} for k in matrices._kinds]
        check(matrices, sizes)
        raise RuntimeError("passed")
    monkeypatch.setattr(A, "_check_streams", seen)


F32, BF, F16, I16 = torch.float32, torch.bfloat16, torch.float16, torch.int16


@pytest.mark.parametrize("dtypes,code,ok", [((BF, F32), A.F32, True), ((BF, BF), A.BF16, True), ((BF, F16), A.F16, True),
                                            ((BF, BF), A.F32, False), ((BF, F32), A.BF16, False), ((F32, F32), A.F32, False)])
def test_orthogonalize(dtypes, code, ok):
    with pytest.raises(RuntimeError if ok else ValueError, match="passed" if ok else "bytes an element"):
        A.adamw_orthogonalize(code, of(*dtypes), WS, stream=0)


@pytest.mark.parametrize("mode,prec,dtypes,ok", [
    (A.MIXED, None, (BF, BF, F32, None, F32), True), (A.MIXED, None, (BF, BF, BF, None, F32), False),
    (A.MIXED, None, (BF, F32, F32, None, F32), False), (A.MIXED, None, (BF, BF, F32, None, BF), False),
    (A.MIXED_SPLIT, None, (BF, BF, F32, None, I16), True), (A.MIXED_SPLIT, None, (BF, BF, F32, None, F32), False),
    (A.PURE_KAHAN, None, (BF, BF, BF, None, BF), True), (A.PURE_KAHAN, None, (BF, BF, F32, None, BF), False),
    (A.MIXED, A.PurePrecision(A.F32, A.BF16, A.KAHAN_F32), (BF, BF, F32, None, F32), True),
    (A.MIXED, A.PurePrecision(A.BF16, A.BF16, A.KAHAN_F32), (BF, BF, BF, None, BF), False),
    (A.MIXED, A.PurePrecision(A.BF16, A.BF16, A.KAHAN_NONE), (BF, BF, BF), True),
])
def test_step(mode, prec, dtypes, ok):
    with pytest.raises(RuntimeError if ok else ValueError, match="passed" if ok else "bytes an element"):
        A.adamw_muon_multi_tensor_step(mode, A.BF16, of(*dtypes), None, STEP, WS, prec=prec, stream=0)


def test_host_tensors():
    with pytest.raises(ValueError, match="on the host"):
        A.adamw_orthogonalize(A.BF16, of(BF, BF), WS, stream=0)
    with pytest.raises(ValueError, match="on the host"):
        A.adamw_muon_multi_tensor_step(A.MIXED, A.BF16, of(BF, BF, F32, None, F32), None, STEP, WS, stream=0)
    there = A.MatrixList([(6, 8)], [[STEP], [STEP + 4096]])
    with pytest.raises(ValueError, match="workspace"):
        A.adamw_orthogonalize(A.BF16, there, torch.zeros(1 << 20, dtype=torch.uint8), stream=0)
    ml = A.MatrixList([(6, 8)], [[STEP + 4096], [STEP + 8192], [STEP + 12288], None, [STEP + 16384]])
    for kw, name in ((dict(d_step=torch.zeros(1, dtype=torch.int32)), "d_step"),
                     (dict(d_step=STEP, d_found_inf=torch.zeros(1)), "d_found_inf")):
        with pytest.raises(ValueError, match=name):
            A.adamw_muon_multi_tensor_step(A.MIXED, A.BF16, ml, None, workspace=WS, stream=0, **kw)
