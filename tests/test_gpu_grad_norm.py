"""GPU: adamw_grad_norm and adamw_tensor_norms against sums in 64 bits.

The reference takes every element to binary64 on the host, where the square of
a 16-bit or fp32 value is exact, and adds the squares with math.fsum (one
rounding).  All terms are positive, so a kernel that adds in binary64 is off by
at most D * 2^-53 (relative), D the additions any one term passes through: at
most 64 in a lane, a few in the two reductions over lanes and waves, and one per
1,024 chunks.  D = 256 covers every list here.  The binary32 norm adds half an
ulp, 2^-24."""
import math

import numpy as np
import pytest
import torch

import adamw_optimizer_step_apply_amd as A
from gpu_util import free, same_bits

pytestmark = pytest.mark.gpu

SUM_TOL = 256 * 2.0 ** -53
NORM_TOL = 2.0 ** -24 + SUM_TOL
DT = {A.BF16: torch.bfloat16, A.F16: torch.float16, A.F32: torch.float32}
SIZES = [0, 1, 7, 8, 9, 31, 2047, 2049, 16384, 16385, 100_003, 3, 0, 40_000, 5]


def sum_squares(x) -> float:
    x = x.detach().double().cpu().numpy().ravel()
    return math.fsum((x * x).tolist())


def make(numels, dt, seed, *, std=1e-2, phase=0, align=1):
    """A list carved out of one buffer, and the buffer: tensors one after another, starts at multiples of `align`
    elements past `phase`; NaN between and around them, which nothing may read into a sum."""
    offs, pos = [], phase
    for n in numels:
        pos = phase + -(-(pos - phase) // align) * align
        offs.append(pos)
        pos += n
    gen = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((pos + 16,), float("nan"), dtype=DT[dt], device="cuda")
    tensors = [buf[o:o + n] for o, n in zip(offs, numels)]
    for t in tensors:
        t.copy_(torch.randn(t.numel(), device="cuda", generator=gen) * std)
    return buf, tensors


def out64(v=-1.0):
    return torch.full((1,), v, dtype=torch.float64, device="cuda")


def out32(v=-1.0):
    return torch.full((1,), v, dtype=torch.float32, device="cuda")


def flag(v=7):
    return torch.full((1,), v, dtype=torch.int32, device="cuda")


def norm(dt, tl, accumulate=False, start=-1.0):
    s, r, f = out64(start), out32(), flag()
    A.adamw_grad_norm(dt, tl, s, r, f, accumulate=accumulate)
    return s.item(), r.item(), f.item()


@pytest.mark.parametrize("dt", [A.BF16, A.F16, A.F32])
@pytest.mark.parametrize("phase,align", [(0, 128), (0, 1), (1, 1), (3, 8), (5, 2)])
def test_norm_of_a_ragged_list(dt, phase, align):
    _, ts = make(SIZES, dt, 11, phase=phase, align=align)
    want = math.fsum(sum_squares(t) for t in ts)
    s, r, f = norm(dt, A.TensorList(SIZES, [None, ts]))
    assert abs(s - want) <= SUM_TOL * want
    assert abs(r - math.sqrt(want)) <= NORM_TOL * math.sqrt(want)
    assert f == 0


@pytest.mark.parametrize("dt", [A.BF16, A.F16, A.F32])
def test_tensor_norms_of_a_ragged_list(dt):
    """Empty tensors get 0; the entries past the list's end stay as they were; the
    list's sum is adamw_grad_norm's, bit for bit."""
    _, ts = make(SIZES, dt, 12, phase=3)
    tl, n = A.TensorList(SIZES, [None, ts]), len(SIZES)
    r = torch.full((n + 2,), -5.0, dtype=torch.float32, device="cuda")
    q = torch.full((n + 2,), -5.0, dtype=torch.float64, device="cuda")
    s = out64()
    A.adamw_tensor_norms(dt, tl, r, q, s)
    for i, t in enumerate(ts):
        want = sum_squares(t)
        assert abs(q[i].item() - want) <= SUM_TOL * want, i
        assert abs(r[i].item() - math.sqrt(want)) <= NORM_TOL * math.sqrt(want), i
    assert r[n:].tolist() == [-5.0] * 2 and q[n:].tolist() == [-5.0] * 2
    assert s.item() == norm(dt, tl)[0]
    one = torch.full((n,), -5.0, dtype=torch.float32, device="cuda")
    A.adamw_tensor_norms(dt, tl, one)
    assert same_bits(one, r[:n])
    only64 = torch.full((n,), -5.0, dtype=torch.float64, device="cuda")
    A.adamw_tensor_norms(dt, tl, None, only64)
    assert same_bits(only64, q[:n])


@pytest.mark.parametrize("n", [1, 2, 63, 64, 255, 256, 257, 16383, 16384, 16385, 16384 * 1024, 16384 * 1025 + 1, 70_000_001])
def test_norm_of_one_tensor(n):
    x = torch.randn(n + 1, device="cuda", generator=torch.Generator(device="cuda").manual_seed(n)).to(torch.bfloat16)[1:]
    want = float(x.double().square().sum().cpu()) if n > 20_000_000 else sum_squares(x)
    # torch's own 64-bit sum of the largest is itself within a few hundred roundings
    tol = SUM_TOL * (4 if n > 20_000_000 else 1)
    s, _, f = norm(A.BF16, A.TensorList([n], [None, [x]]))
    assert abs(s - want) <= tol * want and f == 0
    free()


@pytest.mark.parametrize("dt,values", [
    (A.BF16, [3.3e38, -3.3e38, 1e-38, 1e-40, 2.0 ** -133, 1.0]),
    (A.BF16, [2.0 ** -133, -(2.0 ** -133)] * 7),
    (A.F16, [65504.0, -65504.0, 2.0 ** -24, 6.1e-5]),
    (A.F16, [2.0 ** -24] * 9),
    (A.F32, [3.4e38, -3.4e38, 1e-45, 1e-30]),
    (A.F32, [1e-45, -1e-45, 1e-40] * 3),
])
def test_range_of_the_inputs(dt, values):
    """The largest and the smallest (subnormal) values: no square overflows or vanishes."""
    x = torch.tensor(values, dtype=torch.float64).to(DT[dt]).cuda()
    assert torch.isfinite(x).all() and (x != 0).all()
    want = sum_squares(x)
    s, r, f = norm(dt, A.TensorList([len(values)], [None, [x]]))
    assert abs(s - want) <= SUM_TOL * want and f == 0
    root = math.sqrt(want)
    if root > 3.402824e38:      # beyond binary32
        assert r == math.inf
    else:      # below 2^-126 binary32 has steps of 2^-149, whose half is the rounding's bound
        assert abs(r - root) <= NORM_TOL * root + 2.0 ** -150


@pytest.mark.parametrize("dt", [A.BF16, A.F16, A.F32])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_found_inf_wherever_it_is(dt, bad):
    """One inf or NaN at a head, inside, at a tail, in a tensor of one element: the
    flag is set (as adamw_check_finite's), the sum is not finite, and only that
    tensor's norm is."""
    _, ts = make(SIZES, dt, 13, phase=3)
    tl = A.TensorList(SIZES, [None, ts])
    for i, j in ((1, 0), (10, 0), (10, 50_001), (10, 100_002), (9, 16384), (2, 6), (14, 4)):
        old = ts[i][j].clone()
        ts[i][j] = bad
        s, r, f = norm(dt, tl)
        assert f == 1 and not math.isfinite(s) and not math.isfinite(r)
        assert math.isnan(s) == math.isnan(bad)
        if dt != A.F32:
            g = flag()
            A.adamw_check_finite(dt, tl, g)
            assert g.item() == 1
        per = out64().repeat(len(SIZES))
        A.adamw_tensor_norms(dt, tl, None, per)
        assert [k for k, x in enumerate(per.tolist()) if not math.isfinite(x)] == [i]
        ts[i][j] = old
    assert norm(dt, tl)[2] == 0


def test_two_lists_of_two_types_and_an_empty_one():
    """Parameter groups: the first call starts the sum, the others add to it."""
    _, a = make([1000, 5, 30_000], A.BF16, 14)
    _, b = make([77, 4096], A.F32, 15, phase=1)
    s, r, f = out64(123.0), out32(), flag()
    A.adamw_grad_norm(A.BF16, A.TensorList([1000, 5, 30_000], [None, a]), s)
    A.adamw_grad_norm(A.F32, A.TensorList([77, 4096], [None, b]), s, accumulate=True)
    A.adamw_grad_norm(A.F32, A.TensorList([], [None, []]), s, r, f, accumulate=True)
    want = math.fsum(sum_squares(t) for t in a + b)
    assert abs(s.item() - want) <= SUM_TOL * want
    assert abs(r.item() - math.sqrt(want)) <= NORM_TOL * math.sqrt(want) and f.item() == 0
    b[0][3] = float("inf")
    A.adamw_grad_norm(A.F32, A.TensorList([77, 4096], [None, b]), s)
    A.adamw_grad_norm(A.BF16, A.TensorList([1000, 5, 30_000], [None, a]), s, r, f, accumulate=True)
    assert f.item() == 1 and s.item() == math.inf


@pytest.mark.parametrize("numels", [[], [0], [0, 0, 0]])
def test_nothing_to_sum(numels):
    ts = [torch.empty(1, dtype=torch.bfloat16, device="cuda") for _ in numels]
    tl = A.TensorList(numels, [None, ts])
    assert norm(A.BF16, tl) == (0.0, 0.0, 0)
    assert norm(A.BF16, tl, accumulate=True, start=9.0) == (9.0, 3.0, 0)
    r, s = out32().repeat(max(1, len(numels))), out64()
    A.adamw_tensor_norms(A.BF16, tl, r, None, s)
    assert s.item() == 0.0 and r.tolist() == ([0.0] * len(numels) or [-1.0])


@pytest.mark.parametrize("pad8", [False, True])
@pytest.mark.parametrize("flat", [False, True])
def test_shards(pad8, flat):
    """Each rank sums its own stretch; the ranks' sums add up to the list's; what is
    outside a rank's shard is never read (NaN there)."""
    numels = [13, 5000, 8, 40_001, 1, 16_384]
    _, ts = make(numels, A.BF16, 16, phase=3)
    step = [-(-n // 8) * 8 if pad8 else n for n in numels]
    starts = np.concatenate([[0], np.cumsum(step)])
    total = int(starts[-1])
    host = torch.zeros(total, dtype=torch.bfloat16, device="cuda")
    inside = torch.zeros(total, dtype=torch.bool, device="cuda")
    for t, s0 in zip(ts, starts):
        host[s0:s0 + t.numel()] = t
        inside[s0:s0 + t.numel()] = True
    mask = (2 if flat else 0) | (A.FLAT_PAD8 if pad8 else 0)
    sums, per = [], np.zeros(len(numels))
    for b, e in ((0, 7), (7, 7), (7, 20_001), (20_001, 61_000), (61_000, total)):
        if flat:
            x = torch.full((e - b + 8,), float("nan"), dtype=torch.bfloat16, device="cuda")
            x[3:3 + e - b] = torch.where(inside[b:e], host[b:e], torch.full_like(host[b:e], float("nan")))
            bufs = [x[3:3 + e - b]]
        else:
            bufs = []
            for t, s0 in zip(ts, starts):
                y = torch.full_like(t, float("nan"))
                lo, hi = max(b - int(s0), 0), min(e - int(s0), t.numel())
                if hi > lo:
                    y[lo:hi] = t[lo:hi]
                bufs.append(y)
        tl = A.TensorList(numels, [None, bufs], b, e, mask)
        want = sum_squares(torch.where(inside[b:e], host[b:e], torch.zeros_like(host[b:e])))
        s, _, f = norm(A.BF16, tl)
        assert abs(s - want) <= SUM_TOL * want and f == 0, (b, e)
        q = out64().repeat(len(numels))
        A.adamw_tensor_norms(A.BF16, tl, None, q)
        per += q.cpu().numpy()
        sums.append(s)
    whole = math.fsum(sum_squares(t) for t in ts)
    assert abs(math.fsum(sums) - whole) <= 2 * SUM_TOL * whole
    for i, t in enumerate(ts):
        assert abs(per[i] - sum_squares(t)) <= 2 * SUM_TOL * sum_squares(t), i


def test_same_call_same_bits():
    _, ts = make([3_000_001, 50_000, 7], A.F16, 17, phase=1)
    tl = A.TensorList([3_000_001, 50_000, 7], [None, ts])
    assert len({norm(A.F16, tl) for _ in range(20)}) == 1


def test_the_lists_are_only_read():
    buf, ts = make(SIZES, A.F16, 18, phase=5)
    before = buf.clone()
    tl = A.TensorList(SIZES, [None, ts])
    norm(A.F16, tl)
    A.adamw_tensor_norms(A.F16, tl, out32().repeat(len(SIZES)))
    torch.cuda.synchronize()
    assert same_bits(buf, before)


def test_many_small_tensors():
    rng = np.random.default_rng(19)
    numels = [int(x) for x in rng.integers(0, 300, 5000)]
    _, ts = make(numels, A.F32, 19, phase=1)
    tl = A.TensorList(numels, [None, ts])
    q, s = out64().repeat(5000), out64()
    A.adamw_tensor_norms(A.F32, tl, None, q, s)
    want = np.array([sum_squares(t) for t in ts])
    assert np.all(np.abs(q.cpu().numpy() - want) <= SUM_TOL * want)
    assert abs(s.item() - math.fsum(want)) <= SUM_TOL * math.fsum(want)
    assert norm(A.F32, tl)[0] == s.item()


def test_on_a_side_stream_and_two_streams_at_once():
    """Each stream has its own partial sums: two lists summed at once on two streams."""
    lists = []
    for k in range(2):
        _, ts = make([2_000_000 + k, 77], A.BF16, 20 + k, phase=k)
        lists.append((A.TensorList([2_000_000 + k, 77], [None, ts]), math.fsum(sum_squares(t) for t in ts)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [out64() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for (tl, _), st, o in zip(lists, streams, outs):
            A.adamw_grad_norm(A.BF16, tl, o, stream=st)
    torch.cuda.synchronize()
    for (_, want), o in zip(lists, outs):
        assert abs(o.item() - want) <= SUM_TOL * want


def test_graph_replays_follow_the_gradients():
    """Two lists' norms captured into two graphs on one stream and replayed 4 times
    with new gradients and eager work between, an eager call of a third list among it."""
    st = torch.cuda.Stream()
    cases = []
    for k, numels in enumerate(([300_000, 1, 50], [77, 9000])):
        _, ts = make(numels, A.BF16, 22 + k, phase=k)
        cases.append((numels, ts, A.TensorList(numels, [None, ts]), out64(), out32().repeat(len(numels)), out64()))
    _, other = make([500_000], A.BF16, 30)
    other_tl, other_out = A.TensorList([500_000], [None, other]), out64()
    want_other = sum_squares(other[0])

    def calls(c):
        A.adamw_grad_norm(A.BF16, c[2], c[3], stream=st)
        A.adamw_tensor_norms(A.BF16, c[2], c[4], None, c[5], stream=st)

    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for c in cases:
            calls(c)
    torch.cuda.synchronize()
    graphs = []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            calls(c)
        graphs.append(g)
    for r in range(4):
        for c in cases:
            for t in c[1]:
                t.mul_(1.5 if r % 2 else 0.5)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            for g in graphs:
                g.replay()
            A.adamw_grad_norm(A.BF16, other_tl, other_out, stream=st)
        torch.cuda.synchronize()
        _ = torch.ones(1 << 20, device="cuda").sum().item()
        assert abs(other_out.item() - want_other) <= SUM_TOL * want_other
        for numels, ts, _, s, per, s2 in cases:
            want = [sum_squares(t) for t in ts]
            assert abs(s.item() - math.fsum(want)) <= SUM_TOL * math.fsum(want), r
            assert s.item() == s2.item()
            for x, w in zip(per.tolist(), want):
                assert abs(x - math.sqrt(w)) <= NORM_TOL * math.sqrt(w)
    del graphs
    free()


def test_capture_of_an_unplanned_list_is_refused():
    st = torch.cuda.Stream()
    _, ts = make([5000], A.BF16, 31)
    tl, s = A.TensorList([5000], [None, ts]), out64()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        torch.ones(16, device="cuda")
        with pytest.raises(A.AdamWError):
            A.adamw_grad_norm(A.BF16, tl, s, stream=st)
    del g
    free()


def test_beyond_32_bit_offsets():
    """A tensor of more than 2^32 elements, zero but for planted values near its ends and around 2^32."""
    n = 2 ** 32 + 12_345
    x = torch.zeros(n + 1, dtype=torch.bfloat16, device="cuda")[1:]
    places = [0, 1, 6, 2 ** 31, 2 ** 32 - 1, 2 ** 32, 2 ** 32 + 1, n - 2, n - 1]
    for k, p in enumerate(places):
        x[p] = 2.0 ** k
    s, _, f = norm(A.BF16, A.TensorList([n], [None, [x]]))
    assert s == sum(4.0 ** k for k in range(len(places))) and f == 0
    del x
    free()


def test_workspace_release_between_calls():
    _, ts = make([10_000, 3], A.F16, 33)
    tl = A.TensorList([10_000, 3], [None, ts])
    a = norm(A.F16, tl)
    torch.cuda.synchronize()
    A.adamw_release_workspace()
    assert norm(A.F16, tl) == a


@pytest.fixture
def single_launch_limit():
    yield A.adamw_set_single_launch_max_workgroups
    A.adamw_set_single_launch_max_workgroups(-1)


@pytest.mark.parametrize("chunks", [1, 2, 31, 33, 700, 1024])
def test_one_launch_equals_two(chunks, single_launch_limit):
    """The single launch's last workgroup sees every other's partial of this call, not of
    an earlier one: 60 calls in a row with other gradients each, bit-identical to the
    two-launch form."""
    n = 16384 * (chunks - 1) + 5
    base = torch.randn(n + 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(chunks)).to(torch.bfloat16)
    x = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    tl = A.TensorList([n], [None, [x]])
    assert len(A.adamw_plan_inspect(A.MIXED, A.BF16, tl, for_check=2)) == chunks
    one, two = out64().repeat(60), out64().repeat(60)
    for k in range(60):
        x.copy_(base[k:k + n]).mul_(1.0 + k)
        single_launch_limit(-1)
        A.adamw_grad_norm(A.BF16, tl, one[k:k + 1])
        single_launch_limit(0)
        A.adamw_grad_norm(A.BF16, tl, two[k:k + 1])
    torch.cuda.synchronize()
    assert same_bits(one, two) and len(set(one.tolist())) == 60


def test_joins_of_several_levels():
    """More than 4,096 chunks (the partials are joined in blocks), and the whole-list sum
    beside per-tensor norms, of tensors of many chunks and of one."""
    numels = [16384 * 5000 + 3, 7, 0, 16384 * 300, 100, 16384 * 256, 16384 * 257]
    buf = torch.randint(-3, 4, (sum(numels) + 1,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5),
                        dtype=torch.int8).to(torch.bfloat16)[1:]
    ts, o = [], 0
    for n in numels:
        ts.append(buf[o:o + n])
        o += n
    want = [int((t.float() ** 2).sum(dtype=torch.float64)) for t in ts]      # whole numbers: every order is exact
    tl = A.TensorList(numels, [None, ts])
    assert norm(A.BF16, tl)[0] == sum(want)
    q, s = out64().repeat(len(numels)), out64()
    A.adamw_tensor_norms(A.BF16, tl, None, q, s)
    assert q.tolist() == want and s.item() == sum(want)
    free()


def test_results_too_short_or_of_another_type_are_refused():
    _, ts = make([100, 5], A.BF16, 34)
    tl = A.TensorList([100, 5], [None, ts])
    for bad in (out32(), out64().half(), torch.zeros(0, dtype=torch.float64, device="cuda")):
        with pytest.raises(ValueError):
            A.adamw_grad_norm(A.BF16, tl, bad)
        with pytest.raises(ValueError):
            A.adamw_clip_grads(A.BF16, tl, A.GradClip(bad))
    with pytest.raises(ValueError):
        A.adamw_tensor_norms(A.BF16, tl, out32())
    with pytest.raises(ValueError):
        A.adamw_tensor_norms(A.BF16, tl, torch.zeros(2, 2, device="cuda").t()[0])
    assert bool(torch.isfinite(torch.cat([t.float() for t in ts])).all())
