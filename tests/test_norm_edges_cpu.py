"""Edge calls of the gradient norms without a GPU."""
import pytest
import torch

import adamw_optimizer_step_apply_amd as A
from test_grad_norm_cpu import FAKE, grads


def test_an_empty_lists_norms_need_no_array():
    """A parameter group without tensors: torch's empty result tensors have a null address."""
    assert torch.empty(0).data_ptr() == 0
    with pytest.raises(A.AdamWError) as ei:
        A.adamw_tensor_norms(A.BF16, grads([]), None, None, FAKE, stream=0)
    assert ei.value.status == A.E_HIP, str(ei.value)      # accepted: only the GPU is missing
    with pytest.raises(A.AdamWError, match="both null"):
        A.adamw_tensor_norms(A.BF16, grads([0]), None, None, FAKE, stream=0)
