"""GPU: edge calls of the gradient norms."""
import pytest
import torch

import adamw_optimizer_step_apply_amd as A
from gpu_util import free
from test_gpu_grad_norm import out64

pytestmark = pytest.mark.gpu


def test_tensor_norms_of_a_group_without_tensors():
    """Result tensors of no entries; the list's sum is 0, or not asked for."""
    tl, s = A.TensorList([], [None, []]), out64()
    empty32 = torch.empty(0, dtype=torch.float32, device="cuda")
    empty64 = torch.empty(0, dtype=torch.float64, device="cuda")
    A.adamw_tensor_norms(A.BF16, tl, empty32, empty64, s)
    assert s.item() == 0.0
    A.adamw_tensor_norms(A.BF16, tl, empty32)
    torch.cuda.synchronize()


@pytest.mark.parametrize("per_tensor", [False, True])
def test_joined_blocks_are_this_calls(per_tensor):
    """More than 4,096 partial sums: the blocks' sums pass between workgroups of the joining
    launch.  40 calls in a row without a synchronisation between them, the gradients scaled
    by another whole number each time: every sum is its own call's, exactly."""
    numels = [16384 * 4700 + 5, 16384 * 300 + 1, 7]
    gen = torch.Generator(device="cuda").manual_seed(8)
    base = torch.randint(-3, 4, (sum(numels),), device="cuda", generator=gen, dtype=torch.int8).to(torch.bfloat16)
    x = torch.empty_like(base)
    ts = list(x.split(numels))
    tl = A.TensorList(numels, [None, ts])
    assert len(A.adamw_plan_inspect(A.MIXED, A.BF16, tl, for_check=2)) % 16 != 0
    # whole numbers below 2^53 in any order of the sum
    want = [int((t.float() ** 2).sum(dtype=torch.float64)) for t in base.split(numels)]
    sums, per = out64().repeat(40), out64().repeat(40 * 3).view(40, 3)
    torch.cuda.synchronize()
    scales = [1 + (7 * k) % 11 for k in range(40)]
    for k, f in enumerate(scales):
        torch.mul(base, float(f), out=x)
        if per_tensor:
            A.adamw_tensor_norms(A.BF16, tl, None, per[k], sums[k:k + 1])
        else:
            A.adamw_grad_norm(A.BF16, tl, sums[k:k + 1])
    assert sums.tolist() == [sum(want) * f * f for f in scales]
    if per_tensor:
        assert per.tolist() == [[w * f * f for w in want] for f in scales]
    free()
