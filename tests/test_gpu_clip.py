"""GPU: adamw_clip_grads against the formula in 64 bits.

f = min(1, max_norm / (sqrt(S) * inv + eps)) in binary64, rounded to binary32
(relative 2^-24, plus a few 2^-53); g * f is one binary32 product (2^-24) and one
rounding to the gradient's type: half a step, 2^-8 (bf16) or 2^-11 (fp16) of the
value where that is normal, else half the smallest subnormal."""
import math

import pytest
import torch

import adamw_optimizer_step_apply_amd as A
from gpu_util import free, same_bits
from test_gpu_grad_norm import DT, SIZES, make, out32, out64, sum_squares

pytestmark = pytest.mark.gpu

F_TOL = 2 * 2.0 ** -24 + 2.0 ** -48
TINY = {A.BF16: 2.0 ** -133, A.F16: 2.0 ** -24, A.F32: 2.0 ** -149}
HALF = {A.BF16: 2.0 ** -8, A.F16: 2.0 ** -11, A.F32: 0.0}


def sumsq_of(x):
    return torch.tensor([x], dtype=torch.float64, device="cuda")


def expect(g, dt, f):
    """|clipped - g * f| is at most this, element by element (both in 64 bits)."""
    want = g.double() * f
    return want, want.abs() * (F_TOL + HALF[dt] * (1 + F_TOL)) + TINY[dt] / 2 * (1 + F_TOL)


def same_but_for(buf, before, tensors):
    """Everything in `buf` outside `tensors` is as it was."""
    x, y = buf.clone(), before.clone()
    base = buf.data_ptr()
    for t in tensors:
        o = (t.data_ptr() - base) // buf.element_size()
        if t.numel():
            x[o:o + t.numel()] = 0
            y[o:o + t.numel()] = 0
    return same_bits(x, y)


@pytest.mark.parametrize("dt", [A.BF16, A.F16, A.F32])
@pytest.mark.parametrize("phase,align", [(0, 128), (1, 1), (3, 8), (5, 2)])
@pytest.mark.parametrize("max_norm", [0.25, 1e-4, 0.0])
def test_clips_a_ragged_list(dt, phase, align, max_norm):
    buf, ts = make(SIZES, dt, 41, phase=phase, align=align)
    before, old = buf.clone(), [t.clone() for t in ts]
    s = math.fsum(sum_squares(t) for t in ts)
    f = max_norm / (math.sqrt(s) + float(torch.tensor(1e-6)))
    assert f < 1
    A.adamw_clip_grads(dt, A.TensorList(SIZES, [None, ts]), A.GradClip(sumsq_of(s), max_norm))
    for t, o in zip(ts, old):
        want, tol = expect(o, dt, f)
        assert bool(((t.double() - want).abs() <= tol).all())
    assert same_but_for(buf, before, ts)


@pytest.mark.parametrize("dt", [A.BF16, A.F16, A.F32])
@pytest.mark.parametrize("s", [0.0, 0.9 ** 2, float("inf"), float("nan"), -1.0])
def test_nothing_to_clip_writes_nothing(dt, s):
    """A norm below the limit, and a sum that is not finite (or no sum of squares)."""
    buf, ts = make([100, 5000, 3], dt, 42, phase=1)
    before = buf.clone()
    A.adamw_clip_grads(dt, A.TensorList([100, 5000, 3], [None, ts]), A.GradClip(sumsq_of(s), 1.0))
    torch.cuda.synchronize()
    assert same_bits(buf, before)


def test_zero_norm_zero_limit_and_no_eps():
    x = torch.zeros(100, dtype=torch.bfloat16, device="cuda")
    A.adamw_clip_grads(A.BF16, A.TensorList([100], [None, [x]]), A.GradClip(sumsq_of(0.0), 0.0, 0.0))
    assert x.eq(0).all()


@pytest.mark.parametrize("on_device", [False, True])
def test_loss_scaled_gradients_stay_scaled(on_device):
    """The limit applies to the unscaled norm; the gradients keep their scale."""
    scale = 4096.0
    _, ts = make([3000, 77], A.F16, 43, std=1e-2 * scale)
    old = [t.clone() for t in ts]
    s = math.fsum(sum_squares(t) for t in ts)
    norm = math.sqrt(s) / scale
    f = 0.1 / (norm + float(torch.tensor(1e-6)))
    assert norm > 0.2
    kw = dict(d_scale=A.loss_scale_state(scale)) if on_device else dict(inv_loss_scale=1.0 / scale)
    A.adamw_clip_grads(A.F16, A.TensorList([3000, 77], [None, ts]), A.GradClip(sumsq_of(s), 0.1), **kw)
    for t, o in zip(ts, old):
        want, tol = expect(o, A.F16, f)
        assert bool(((t.double() - want).abs() <= tol).all())
    # a limit above the unscaled norm (and far below the scaled one) clips nothing
    kept = [t.clone() for t in ts]
    A.adamw_clip_grads(A.F16, A.TensorList([3000, 77], [None, ts]), A.GradClip(sumsq_of(s), 2 * norm), **kw)
    assert all(same_bits(a, b) for a, b in zip(ts, kept))


def test_subnormal_results_are_kept():
    x = torch.tensor([2.0 ** -14, 2.0 ** -20, -(2.0 ** -23), 2.0 ** -24], dtype=torch.float16, device="cuda")
    A.adamw_clip_grads(A.F16, A.TensorList([4], [None, [x]]), A.GradClip(sumsq_of(4.0), 1.0, 0.0))
    assert x.tolist() == [2.0 ** -15, 2.0 ** -21, -(2.0 ** -24), 0.0]     # ties to even


@pytest.mark.parametrize("pad8", [False, True])
@pytest.mark.parametrize("flat", [False, True])
def test_a_shard_is_clipped_and_nothing_else(pad8, flat):
    numels = [13, 5000, 8, 40_001]
    step = [-(-n // 8) * 8 if pad8 else n for n in numels]
    b, e = 9, sum(step) - 777
    mask = (2 if flat else 0) | (A.FLAT_PAD8 if pad8 else 0)
    if flat:
        buf = torch.full((e - b + 16,), 3.0, dtype=torch.float32, device="cuda")
        bufs = [buf[5:5 + e - b]]
        start = 0
        pieces = []
        for n, st_ in zip(numels, step):
            lo, hi = max(b, start), min(e, start + n)
            pieces.append(bufs[0][lo - b:hi - b])
            start += st_
    else:
        buf, bufs = make(numels, A.F32, 44, phase=1)
        pieces, start = [], 0
        for t, st_ in zip(bufs, step):
            lo, hi = max(b - start, 0), min(e - start, t.numel())
            pieces.append(t[lo:hi])
            start += st_
    before, old = buf.clone(), [p.clone() for p in pieces]
    A.adamw_clip_grads(A.F32, A.TensorList(numels, [None, bufs], b, e, mask), A.GradClip(sumsq_of(16.0), 1.0, 0.0))
    for p, o in zip(pieces, old):
        assert same_bits(p, o * 0.25)
    assert same_but_for(buf, before, pieces)


def test_the_factor_is_read_in_stream_order():
    """The norm and the clipping queued one after the other: the norm that follows is the limit."""
    _, ts = make([70_000, 11], A.F32, 45, phase=1)
    tl = A.TensorList([70_000, 11], [None, ts])
    s = out64()
    A.adamw_grad_norm(A.F32, tl, s)
    A.adamw_clip_grads(A.F32, tl, A.GradClip(s, 0.5))
    got = out32()
    A.adamw_grad_norm(A.F32, tl, s, got)
    # every element, and so the norm, is off by at most 2 * 2^-24 of itself; eps takes 1e-6 / norm off
    first = math.sqrt(s.item())
    assert abs(got.item() - 0.5) <= 0.5 * (4 * 2.0 ** -24 + 1e-6 / 2.0) and first > 0.49


def test_graph_replays_clip_again():
    st = torch.cuda.Stream()
    _, ts = make([9000, 5], A.F32, 46, phase=3)
    _, other = make([9000, 5], A.F32, 46, phase=3)
    s = sumsq_of(4.0)
    tl, tl2 = A.TensorList([9000, 5], [None, ts]), A.TensorList([9000, 5], [None, other])
    torch.cuda.synchronize()
    c = A.GradClip(s, 1.0, 0.0)
    A.adamw_clip_grads(A.F32, tl, c, stream=st)
    A.adamw_clip_grads(A.F32, tl2, c, stream=st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        A.adamw_clip_grads(A.F32, tl, c, stream=st)
    for v in (16.0, 0.5, 9.0, float("inf")):
        s.fill_(v)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            g.replay()
        A.adamw_clip_grads(A.F32, tl2, c, stream=st)
        torch.cuda.synchronize()
        _ = torch.ones(1 << 20, device="cuda").sum().item()
        assert all(same_bits(a, b) for a, b in zip(ts, other)), v
    del g
    free()


def test_beyond_32_bit_offsets():
    n = 2 ** 32 + 4_321
    x = torch.zeros(n + 3, dtype=torch.bfloat16, device="cuda")
    y = x[1:n + 1]
    places = [0, 1, 2 ** 31, 2 ** 32 - 1, 2 ** 32, n - 1]
    for p in places:
        y[p] = 8.0
    x[0], x[n + 1] = 8.0, 8.0
    A.adamw_clip_grads(A.BF16, A.TensorList([n], [None, [y]]), A.GradClip(sumsq_of(16.0), 2.0, 0.0))
    assert [y[p].item() for p in places] == [4.0] * len(places)
    assert x[0].item() == x[n + 1].item() == 8.0
    assert int((x[:2 ** 31] != 0).sum()) + int((x[2 ** 31:] != 0).sum()) == len(places) + 2
    del x, y
    free()


@pytest.mark.parametrize("elems", [2048, 1 << 22])
def test_chunk_knob(elems):
    """Chunks of the smallest and the largest size give the same clipping, and norms within the bound."""
    numels = [5, 9_000_001, 2048, 70_000]
    _, a = make(numels, A.BF16, 47, phase=3)
    _, b = make(numels, A.BF16, 47, phase=3)
    s = sumsq_of(9.0)
    A.adamw_clip_grads(A.BF16, A.TensorList(numels, [None, a]), A.GradClip(s, 1.0))
    want, got = out64(), out64()
    A.adamw_grad_norm(A.BF16, A.TensorList(numels, [None, a]), want)
    try:
        A.adamw_set_chunk_elems(elems)
        A.adamw_clip_grads(A.BF16, A.TensorList(numels, [None, b]), A.GradClip(s, 1.0))
        A.adamw_grad_norm(A.BF16, A.TensorList(numels, [None, b]), got)
    finally:
        A.adamw_set_chunk_elems(0)
    assert all(same_bits(x, y) for x, y in zip(a, b))
    # up to 4 M / 512 terms in a lane, each sum within that many roundings
    assert abs(got.item() - want.item()) <= want.item() * (8192 + 256) * 2.0 ** -53
    free()
