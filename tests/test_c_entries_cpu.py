"""No C++ exception leaves a C entry point (CPU): a count of tensors that no host array
can have comes back as a status from every call that takes a list."""
import ctypes

import pytest

import adamw_optimizer_step_apply_amd as A
from test_grad_norm_cpu import FAKE, grads


def huge():
    tl = grads([10])
    for s in range(5):
        tl.c.ptr[s] = tl.c.ptr[1]
    tl.c.n_tensors = 2 ** 61
    return tl


CALLS = {
    "step": lambda lib, l, h, sc, pc: lib.adamw_multi_tensor_step(A.MIXED, A.BF16, l, h, FAKE, None, None),
    "pure step": lambda lib, l, h, sc, pc: lib.adamw_pure_multi_tensor_step(pc, l, h, FAKE, None, None),
    "amp step": lambda lib, l, h, sc, pc: lib.adamw_multi_tensor_step_amp(A.MIXED, A.F16, l, h, FAKE, FAKE, FAKE, sc, None),
    "allocation-free step": lambda lib, l, h, sc, pc: lib.adamw_multi_tensor_step_noalloc(A.MIXED, A.BF16, l, h, FAKE, None,
                                                                                          None),
    "check": lambda lib, l, h, sc, pc: lib.adamw_check_finite(A.F16, l, FAKE, None),
}


@pytest.mark.parametrize("call", CALLS)
def test_no_exception_leaves(call):
    tl, h, sc, pc = huge(), A.HParams().c(), A.LossScaler().c(), A.PurePrecision(A.BF16, A.BF16, 1).c()
    assert CALLS[call](A._lib, ctypes.byref(tl.c), ctypes.byref(h), ctypes.byref(sc), ctypes.byref(pc)) == A.E_NOMEM
    assert A.adamw_last_error()
