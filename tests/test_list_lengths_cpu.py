"""Lists whose streams have too few entries, or too short a flat buffer, are refused before any HIP call: the library would
read past the array of addresses, or a kernel past the buffer."""
import pytest
import torch

import adamw_optimizer_step_apply_amd as A

FAKE, WS = 0x7f0000000000, (0x600000000000, 1 << 34)     # never dereferenced
COUNTER = FAKE - 4096


def entries(streams, short, given):
    """Three entries for each stream of `streams`, `given` for the stream `short`."""
    at = lambda s, i: FAKE + ((s * 8 + i) << 20)  # noqa: E731
    return [[at(s, i) for i in range(given if s == short else 3)] if s in streams else None for s in range(5)]


@pytest.mark.parametrize("given", [0, 1, 2])
def test_address_arrays_are_as_long_as_the_list(given):
    """What lies behind a shorter one may be null too, so that the refusals below do not show it."""
    tl = A.TensorList([64, 64, 64], entries(range(5), 3, given))
    assert [len(a) for a in tl._arrays] == [3] * 5
    assert list(tl._arrays[3])[given:] == [None] * (3 - given)


@pytest.mark.parametrize("given", [0, 1, 2])
@pytest.mark.parametrize("short", range(5))
def test_steps(short, given):
    tl = A.TensorList([64, 64, 64], entries(range(5), short, given))
    with pytest.raises(A.AdamWError, match="null") as e:
        A.adamw_multi_tensor_step(A.MIXED, A.BF16, tl, A.HParams(), COUNTER, stream=0)
    assert e.value.status == A.E_INVALID


@pytest.mark.parametrize("given", [0, 1, 2])
@pytest.mark.parametrize("call", ["check", "norm", "clip"])
def test_gradients(call, given):
    tl = A.TensorList([64, 64, 64], entries([1], 1, given))
    with pytest.raises(A.AdamWError, match="null") as e:
        if call == "check":
            A.adamw_check_finite(A.BF16, tl, COUNTER, stream=0)
        elif call == "norm":
            A.adamw_grad_norm(A.BF16, tl, COUNTER, stream=0)
        else:
            A.adamw_clip_grads(A.BF16, tl, A.GradClip(COUNTER), stream=0)
    assert e.value.status == A.E_INVALID


@pytest.mark.parametrize("given", [0, 1, 2])
@pytest.mark.parametrize("short", [0, 1, 2, 4])
def test_matrices(short, given):
    shapes = [(4, 16)] * 3
    with pytest.raises(A.AdamWError, match="null") as e:
        A.adamw_muon_multi_tensor_step(A.MIXED, A.BF16, A.MatrixList(shapes, entries([0, 1, 2, 4], short, given)), None,
                                       COUNTER, WS, stream=0)
    assert e.value.status == A.E_INVALID
    if short < 2:
        with pytest.raises(A.AdamWError, match="null"):
            A.adamw_orthogonalize(A.F32, A.MatrixList(shapes, entries([0, 1], short, given)), WS, stream=0)


def test_one_entry_is_enough_for_a_flat_or_blocked_stream():
    """Only the first HIP call fails, on a host without a GPU."""
    if torch.cuda.is_available():
        pytest.skip("would run on made-up addresses")
    for streams, mask in ([[[FAKE + (s << 20)] for s in range(5)], 0x1f],
                          [entries([0, 1], 9, 0)[:2] + [[FAKE], None, None], A.BLOCKED_STATE]):
        with pytest.raises(A.AdamWError) as e:
            A.adamw_multi_tensor_step(A.MIXED, A.BF16, A.TensorList([64, 64, 64], streams, flat_mask=mask), A.HParams(), COUNTER, stream=0)
        assert e.value.status == A.E_HIP


@pytest.mark.parametrize("mask,begin,end,length", [(0b10, 0, -1, 63 + 64 + 9), (0b10, 63, -1, 64 + 9), (0b10, 63, 127, 64),
                                                   (0b10 | A.FLAT_PAD8, 0, -1, 64 + 64 + 16)])
def test_a_flat_shard_buffer_of_matrices(mask, begin, end, length):
    shapes = [(7, 9), (8, 8), (3, 3)]
    for n, ok in ((length, True), (length + 5, True), (length - 1, False), (0, False)):
        streams = [[FAKE, FAKE + 4096, FAKE + 8192], [torch.zeros(n, dtype=torch.bfloat16)]]
        if ok:
            A.MatrixList(shapes, streams, begin, end, mask)
            continue
        with pytest.raises(ValueError, match="flat buffer"):
            A.MatrixList(shapes, streams, begin, end, mask)


def test_a_tensor_too_many():
    with pytest.raises(ValueError, match="no matrix"):
        A.MatrixList([(2, 3)], [[torch.zeros(2, 3)] * 2])
