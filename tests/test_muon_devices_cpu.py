"""Matrices, workspace and stream on different GPUs are refused by the binding: a kernel of one would read another's memory.
On the CPU, with lists that say where their tensors would be."""
import pytest
import torch

import adamw_optimizer_step_apply_amd as A

FAKE, WS = 0x7f0000000000, (0x600000000000, 1 << 34)     # never dereferenced


@pytest.fixture(autouse=True)
def as_if_on_a_gpu(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    check = A._check_devices

    def seen(*args):
        check(*args)
        raise RuntimeError("passed")
    monkeypatch.setattr(A, "_check_devices", seen)


def on(*devices):
    ml = A.MatrixList([(8, 8)], [[FAKE], [FAKE + 4096], [FAKE + 8192], None, [FAKE + 12288]])
    ml._devices = frozenset(devices)
    return ml


@pytest.mark.parametrize("devices,stream,ok", [((0,), None, True), ((), None, True), ((1,), None, False), ((0, 1), None, False),
                                               ((0, 1), 0, False), ((1,), 0, True)])
def test_devices(devices, stream, ok):
    for call in (lambda: A.adamw_orthogonalize(A.F32, on(*devices), WS, stream=stream),
                 lambda: A.adamw_muon_multi_tensor_step(A.MIXED, A.BF16, on(*devices), None, FAKE - 4096, WS, stream=stream)):
        with pytest.raises(RuntimeError if ok else ValueError, match="passed" if ok else "one is needed"):
            call()
