"""GPU: edge calls of the gradient norms."""
import pytest
import torch

import adamw_optimizer_step_apply_amd as A
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
