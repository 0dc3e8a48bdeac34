"""A loss-scale state that is no such state on the GPU is refused by the binding, on the CPU: a kernel would read, or write,
what is not there."""
import pytest
import torch

import adamw_optimizer_step_apply_amd as A

FAKE, WS = 0x7f0000000000, (0x600000000000, 1 << 34)     # never dereferenced


def calls(scale):
    shapes = [(8, 8)]
    ml = A.MatrixList(shapes, [[FAKE], [FAKE + 4096], [FAKE + 8192], None, [FAKE + 12288]])
    tl = A.TensorList([64], [[FAKE + (s << 16)] for s in range(5)])
    clip, step, found = A.GradClip(FAKE - 4096), FAKE - 8192, FAKE - 8188
    return {
        "muon": lambda: A.adamw_muon_multi_tensor_step(A.MIXED, A.F16, ml, None, step, WS, d_scale=scale, stream=0),
        "amp": lambda: A.adamw_multi_tensor_step_amp(A.MIXED, A.F16, tl, None, step, found, scale, stream=0),
        "clip": lambda: A.adamw_clip_grads(A.F16, tl, clip, d_scale=scale, stream=0),
        "clipped": lambda: A.adamw_multi_tensor_step_clipped(A.MIXED, A.F16, tl, None, clip, step, d_scale=scale, stream=0),
    }


@pytest.mark.parametrize("call", ["muon", "amp", "clip", "clipped"])
@pytest.mark.parametrize("scale", [A.loss_scale_state(1024.0, device="cpu"), torch.zeros(1), torch.zeros(2, 2)[:, 0]])
def test_host_and_short_states(call, scale):
    with pytest.raises(ValueError, match="d_scale"):
        calls(scale)[call]()


@pytest.mark.parametrize("call", ["muon", "amp", "clip", "clipped"])
def test_addresses_pass(call):
    if torch.cuda.is_available():
        pytest.skip("would run on made-up addresses")
    with pytest.raises(A.AdamWError) as e:
        calls(FAKE - 64)[call]()
    assert e.value.status == A.E_HIP
