"""The gradient norms without a GPU: bad calls are refused before any HIP call,
and the sweep plan (one workgroup per chunk of any elements) covers exactly the
list's elements, inside the caller's buffers, with every chunk but a piece's
first starting at a 16-byte edge."""
import numpy as np
import pytest

import adamw_optimizer_step_apply_amd as A

FAKE = 0x7f0000000000     # never dereferenced: validation fails before any HIP call
ESZ = {A.BF16: 2, A.F16: 2, A.F32: 4}


def grads(numels, base=FAKE, esz=2, gap=0, **kw):
    offs = np.concatenate([[0], np.cumsum([n * esz + gap for n in numels])[:-1]]) if numels else []
    return A.TensorList(numels, [None, [base + int(o) for o in offs]], **kw)


@pytest.mark.parametrize("call,needle", [
    (lambda: A.adamw_grad_norm(7, grads([10]), FAKE, stream=0), "g_dtype"),
    (lambda: A.adamw_grad_norm(A.BF16, grads([10]), 0, stream=0), "d_sumsq is null"),
    (lambda: A.adamw_grad_norm(A.BF16, grads([10]), FAKE + 4, stream=0), "8-byte"),
    (lambda: A.adamw_grad_norm(A.BF16, grads([10]), FAKE, FAKE + 2, stream=0), "4-byte"),
    (lambda: A.adamw_grad_norm(A.BF16, grads([10]), FAKE, 0, FAKE + 2, stream=0), "4-byte"),
    (lambda: A.adamw_grad_norm(A.BF16, grads([10], base=FAKE + 1), FAKE, stream=0), "aligned"),
    (lambda: A.adamw_grad_norm(A.F32, grads([10], base=FAKE + 2), FAKE, stream=0), "aligned"),
    (lambda: A.adamw_grad_norm(A.BF16, grads([10, -1]), FAKE, stream=0), "numel"),
    (lambda: A.adamw_grad_norm(A.BF16, A.TensorList([10], [[FAKE]]), FAKE, stream=0), "grad"),
    (lambda: A.adamw_grad_norm(A.BF16, A.TensorList([10], [None, [0]]), FAKE, stream=0), "grad"),
    (lambda: A.adamw_grad_norm(A.BF16, grads([10, 3], shard_begin=0, shard_end=14), FAKE, stream=0), "shard"),
    (lambda: A.adamw_grad_norm(A.BF16, grads([10], flat_mask=1 << 6), FAKE, stream=0), "flat_mask"),
    (lambda: A.adamw_tensor_norms(A.BF16, grads([10]), None, None, FAKE, stream=0), "both null"),
    (lambda: A.adamw_tensor_norms(7, grads([10]), FAKE, stream=0), "g_dtype"),
    (lambda: A.adamw_tensor_norms(A.BF16, grads([10]), FAKE + 2, stream=0), "4-byte"),
    (lambda: A.adamw_tensor_norms(A.BF16, grads([10]), None, FAKE + 4, stream=0), "8-byte"),
    (lambda: A.adamw_tensor_norms(A.BF16, grads([10]), FAKE, None, FAKE + 4, stream=0), "8-byte"),
])
def test_rejected_before_any_hip_call(call, needle):
    with pytest.raises(A.AdamWError) as ei:
        call()
    assert ei.value.status in (A.E_INVALID, A.E_UNSUPPORTED)
    assert needle.lower() in str(ei.value).lower(), str(ei.value)


@pytest.mark.parametrize("call", [lambda: A.adamw_grad_norm(A.F32, grads([10, 20], esz=4), FAKE, stream=0),
                                  lambda: A.adamw_tensor_norms(A.F16, grads([10, 0]), FAKE, stream=0)])
def test_valid_call_reaches_hip(call):
    with pytest.raises(A.AdamWError) as ei:
        call()
    assert ei.value.status == A.E_HIP


@pytest.mark.parametrize("seed", range(30))
def test_sweep_plan_covers_the_list(seed):
    rng = np.random.default_rng(seed)
    dt = (A.BF16, A.F16, A.F32)[seed % 3]
    esz = ESZ[dt]
    chunk = 32768 // esz
    nt = int(rng.integers(0, 25))
    numels = [int(x) for x in rng.choice([0, 1, 3, 7, 8, 9, 16, 100, 4097, 8191, 8192, 16384, 16391, 70000], size=nt)]
    pad8 = seed % 4 == 1
    step = [-(-n // 8) * 8 if pad8 else n for n in numels]
    total = sum(step)
    b = int(rng.integers(0, total + 1)) if seed % 2 else 0
    e = int(rng.integers(b, total + 1)) if seed % 2 else total
    base = FAKE + int(rng.integers(0, 16)) * esz
    tl = grads(numels, base, esz, gap=16 * int(rng.integers(0, 3)), shard_begin=b, shard_end=e,
               flat_mask=A.FLAT_PAD8 if pad8 else 0)
    rows, ranges = A.adamw_plan_inspect_bytes(A.MIXED, dt, tl, for_check=2)
    assert [tuple(r) for r in rows.tolist()] == A.adamw_plan_inspect(A.MIXED, dt, tl, for_check=2)
    starts = np.concatenate([[0], np.cumsum(step)])
    want = [(t, lo, hi) for t in range(nt)
            for lo, hi in [(max(b - int(starts[t]), 0), min(e - int(starts[t]), numels[t]))] if hi > lo]
    got, seen = {}, []
    for (t, off, n, kind, flat, seg), r in zip(rows.tolist(), ranges.tolist()):
        assert kind == 2 and 0 < n <= chunk + 16 // esz - 1 and flat == starts[t] + off
        assert [x for s in (0, 2, 3, 4) for x in r[s]] == [0] * 8
        lo, hi = r[1]
        assert hi - lo == n * esz and lo == tl.c.ptr[1][t] + off * esz
        if t in got:
            assert off == got[t][1] and lo % 16 == 0
            got[t] = (got[t][0], off + n)
        else:
            seen.append(t)
            got[t] = (off, off + n)
    assert [(t, *got[t]) for t in seen] == want


def test_sweep_plan_takes_one_chunk_per_short_tensor():
    """However a short tensor is aligned, it is one workgroup's work."""
    numels = [1, 7, 13, 100, 4099, 16384]
    rows = A.adamw_plan_inspect(A.MIXED, A.BF16, grads(numels, base=FAKE + 2), for_check=2)
    assert [r[0] for r in rows] == list(range(6))


def test_sweep_plan_beyond_32_bit_offsets():
    n = 2 ** 32 + 12345
    rows, ranges = A.adamw_plan_inspect_bytes(A.MIXED, A.F32, grads([n], base=FAKE + 4, esz=4), for_check=2)
    assert rows[-1][1] + rows[-1][2] == n and int(ranges[-1, 1, 1]) == FAKE + 4 + 4 * n
    assert rows[:, 2].sum() == n


def test_sweep_plan_honours_the_chunk_knob():
    try:
        A.adamw_set_chunk_elems(2048)
        assert len(A.adamw_plan_inspect(A.MIXED, A.F32, grads([8192], esz=4), for_check=2)) == 4
    finally:
        A.adamw_set_chunk_elems(0)
    assert len(A.adamw_plan_inspect(A.MIXED, A.F32, grads([8192], esz=4), for_check=2)) == 1
