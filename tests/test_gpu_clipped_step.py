"""GPU: the clipped AdamW step against the CPU oracle, bit for bit, and the run of
norm, clipping and step together.

The oracle's step with the gradient multiplier round_f32(inv * f), f =
min(1, max_norm / (sqrt(S) * inv + eps)) formed here in binary64, is what the
clipped step computes: only the last bit of a binary64 square root lies between
the two multipliers before they are rounded to binary32."""
import math
import threading

import numpy as np
import pytest
import torch

import adamw_optimizer_step_apply_amd as A
from gpu_util import DT, MODE, Case, build_blocked, free, hp_pair, pure_precision, same_bits, to_np, unpack_blocked

pytestmark = pytest.mark.gpu

SIZES = [0, 1, 7, 8, 9, 2047, 2049, 16385, 100_003, 3, 40_000]
ALL = [("mixed", "bf16"), ("mixed", "f16"), ("kahan", "bf16"), ("split", "bf16"), ("pure-f32-f32-k", "bf16"),
       ("pure-bf16-f32-n", "bf16"), ("pure-bf16-bf16-k32", "bf16")]


@pytest.fixture
def single_launch_limit():
    yield A.adamw_set_single_launch_max_workgroups
    A.adamw_set_single_launch_max_workgroups(-1)


def multiplier(s, inv, max_norm, eps):
    inv, max_norm, eps = (float(np.float32(x)) for x in (inv, max_norm, eps))
    f = min(1.0, max_norm / (math.sqrt(s) * inv + eps))
    return float(np.float32(inv * f)), f


def clipped(case, hp, clip, found=None, tl=None, **kw):
    pure = case.mode.startswith("pure")
    A.adamw_multi_tensor_step_clipped(0 if pure else MODE[case.mode], DT[case.p_dtype], tl or case.tensor_list(), hp, clip,
                                      case.d_step, found, prec=pure_precision(case.mode) if pure else None, **kw)


def grads_of(case):
    return A.TensorList(case.numels, [None, [case.arena.view("g", i) for i in range(len(case.numels))]])


def snapshot(case):
    return {k: v.clone() for k, v in case.arena.bufs.items()}


def unchanged(case, snap):
    return all(same_bits(v, snap[k]) for k, v in case.arena.bufs.items())


@pytest.mark.parametrize("limit", [-1, 0])
@pytest.mark.parametrize("mode,p_dtype", ALL)
def test_steps_follow_the_oracle(mode, p_dtype, limit, single_launch_limit):
    """Norm and clipped step, 4 times, the limit above the norm once."""
    single_launch_limit(limit)
    scale = 65536.0 if p_dtype == "f16" else 1.0
    case = Case(mode, SIZES, seed=301, p_dtype=p_dtype, align_elems=3, loss_scale=scale, random_moments=True)
    dt = DT[p_dtype]
    s = torch.zeros(1, dtype=torch.float64, device="cuda")
    found = torch.zeros(1, dtype=torch.int32, device="cuda")
    for k in range(4):
        if k:
            case.refill_grads(k)
        max_norm = (0.1, 0.01, 1e6, 0.3)[k]
        A.adamw_grad_norm(dt, grads_of(case), s, None, found)
        clipped(case, hp_pair(inv_scale=1.0 / scale)[0], A.GradClip(s, max_norm), found)
        mult, f = multiplier(s.item(), 1.0 / scale, max_norm, 1e-6)
        assert (f == 1.0) == (k == 2)
        case.oracle_step(hp_pair(inv_scale=mult)[1])
    case.compare_all(f"clipped-{mode}-{p_dtype}-{limit}")
    free()


@pytest.mark.parametrize("limit", [-1, 0])
def test_first_moment_against_64_bits(limit, single_launch_limit):
    """From zero moments, exp_avg = (1 - beta1) * g * inv * f: two roundings of the
    multiplier and product, one of 1 - beta1's product and one of the sum with 0."""
    single_launch_limit(limit)
    case = Case("mixed", [5000, 3], seed=302, p_dtype="f16", loss_scale=1024.0)
    s = torch.zeros(1, dtype=torch.float64, device="cuda")
    A.adamw_grad_norm(A.F16, grads_of(case), s)
    clipped(case, hp_pair(inv_scale=1.0 / 1024)[0], A.GradClip(s, 0.02))
    gs = [case.arena.view("g", i).double() for i in range(2)]
    f = 0.02 / (math.sqrt(float(sum((g ** 2).sum() for g in gs))) / 1024 + 1e-6)
    for i, g in enumerate(gs):
        want = (1.0 - float(np.float32(0.9))) * g * (f / 1024)
        # 0.02 and 1e-6 are handed over in binary32: 2 more half steps
        assert bool(((case.arena.view("m", i).double() - want).abs() <= want.abs() * 6 * 2.0 ** -24 + 2.0 ** -149).all())


@pytest.mark.parametrize("limit", [-1, 0])
@pytest.mark.parametrize("mode", ["mixed", "kahan", "split"])
def test_without_clipping_it_is_the_plain_step(mode, limit, single_launch_limit):
    single_launch_limit(limit)
    a, b = (Case(mode, SIZES, seed=303, random_moments=True) for _ in range(2))
    hg, _ = hp_pair(inv_scale=0.37)
    s = torch.full((1,), 4.0, dtype=torch.float64, device="cuda")
    clipped(a, hg, A.GradClip(s, 1.0))      # norm 0.74 < 1
    b.gpu_step(hg)
    torch.cuda.synchronize()
    assert a.d_step.item() == b.d_step.item() == 1
    assert all(same_bits(a.arena.bufs[k], b.arena.bufs[k]) for k in a.keys)
    free()


@pytest.mark.parametrize("limit", [-1, 0])
@pytest.mark.parametrize("mode,p_dtype", ALL[:4])
@pytest.mark.parametrize("s,found", [(float("inf"), None), (float("nan"), 0), (-1.0, 0), (4.0, 1)])
def test_skipped_step_writes_nothing(mode, p_dtype, limit, s, found, single_launch_limit):
    single_launch_limit(limit)
    case = Case(mode, SIZES, seed=304, p_dtype=p_dtype, random_moments=True)
    case.d_step.fill_(5)
    snap = snapshot(case)
    flag = None if found is None else torch.full((1,), found, dtype=torch.int32, device="cuda")
    clipped(case, hp_pair()[0], A.GradClip(torch.tensor([s], dtype=torch.float64, device="cuda"), 1.0), flag)
    torch.cuda.synchronize()
    assert case.d_step.item() == 5 and unchanged(case, snap)
    free()


@pytest.mark.parametrize("limit", [-1, 0])
def test_dynamic_loss_scale(limit, single_launch_limit):
    """The scale is read, advanced once a step, backed off on an overflow that only the
    sum of squares tells, and left alone where the call is told to."""
    single_launch_limit(limit)
    case = Case("mixed", SIZES, seed=305, p_dtype="f16", loss_scale=4096.0, random_moments=True)
    scale, s = A.loss_scale_state(4096.0), torch.zeros(1, dtype=torch.float64, device="cuda")
    rule = A.LossScaler(2.0, 0.5, 3)
    want_scale, want_run = 4096.0, 0
    for k in range(6):
        case.refill_grads(k)
        if k == 4:
            case.arena.view("g", 8)[99_999] = float("inf")
            case.host["g"] = to_np(case.arena.bufs["g"])
        A.adamw_grad_norm(A.F16, grads_of(case), s)
        clipped(case, hp_pair(inv_scale=123.0)[0], A.GradClip(s, 0.05), d_scale=scale, scaler=rule, advance_scale=k != 1)
        if k != 4:
            inv = float(np.float32(1.0 / want_scale))
            case.oracle_step(hp_pair(inv_scale=multiplier(s.item(), inv, 0.05, 1e-6)[0])[1])
        if k == 4:
            want_scale, want_run = want_scale * 0.5, 0
        elif k != 1:
            want_run += 1
            if want_run == 3:
                want_scale, want_run = want_scale * 2.0, 0
        torch.cuda.synchronize()
        assert scale[0].item() == want_scale and scale.view(torch.int32)[1].item() == want_run, k
    case.compare_all(f"clipped-amp-{limit}")
    free()


@pytest.mark.parametrize("limit", [-1, 0])
def test_saturated_counter(limit, single_launch_limit):
    single_launch_limit(limit)
    case = Case("mixed", SIZES, seed=306, p_dtype="f16", random_moments=True)
    scale = A.loss_scale_state(8.0)
    for s in (4.0, float("nan")):
        case.d_step.fill_(2 ** 31 - 1)
        snap = snapshot(case)
        clipped(case, hp_pair()[0], A.GradClip(torch.tensor([s], dtype=torch.float64, device="cuda")), d_scale=scale)
        torch.cuda.synchronize()
        assert case.d_step.item() == 2 ** 31 - 1 and unchanged(case, snap)
        assert scale[0].item() == 8.0 and scale.view(torch.int32)[1].item() == 0
    free()


@pytest.mark.parametrize("limit", [-1, 0])
@pytest.mark.parametrize("mode", ["mixed", "kahan"])
def test_blocked_state_and_a_shard(mode, limit, single_launch_limit):
    single_launch_limit(limit)
    numels = [40_000, 24, 8, 70_000, 16]
    case = Case(mode, numels, seed=307, align_elems=1, random_moments=True)
    b, e = 8_000, sum(numels) - 4_000
    blocked = build_blocked(case, b, e)
    views = [[case.arena.view(k, i) for i in range(5)] for k in ("p", "g")]
    tl = A.TensorList(numels, views + [[blocked], None, None], b, e, A.BLOCKED_STATE)
    s = torch.tensor([9.0], dtype=torch.float64, device="cuda")
    clipped(case, hp_pair()[0], A.GradClip(s, 1.5), tl=tl)
    case.oracle_step(hp_pair(inv_scale=multiplier(9.0, 1.0, 1.5, 1e-6)[0])[1], shard=(b, e))
    torch.cuda.synchronize()
    assert case.d_step.item() == 1
    got = unpack_blocked(case, blocked, b, e)
    for k in case.keys[2:]:
        assert np.array_equal(got[k].view(np.uint8), case.host[k][b:e].view(np.uint8)), k
    assert np.array_equal(to_np(case.arena.bufs["p"]), case.host["p"])
    free()


@pytest.mark.parametrize("limit", [-1, 0])
def test_training_iteration_of_two_groups(limit, single_launch_limit):
    """A training run of 5 iterations: one norm over two parameter groups (of different
    weight decay), clipped steps of both under one dynamic loss scale, an overflow in
    the second iteration; captured into a graph on one stream and replayed, with eager
    work between; every value the oracle's."""
    single_launch_limit(limit)
    st = torch.cuda.Stream()
    groups = [Case("mixed", [30_000, 513], seed=308, p_dtype="f16", align_elems=1, loss_scale=1024.0),
              Case("mixed", [100, 7, 3000], seed=309, p_dtype="f16", align_elems=3, loss_scale=1024.0)]
    decay = (0.1, 0.0)
    tls, gls = [c.tensor_list() for c in groups], [grads_of(c) for c in groups]
    scale, rule = A.loss_scale_state(1024.0), A.LossScaler(2.0, 0.5, 2)
    s = torch.zeros(1, dtype=torch.float64, device="cuda")
    norm, found = torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    per = [torch.zeros(len(c.numels), device="cuda") for c in groups]

    def iteration():
        for k in range(2):
            A.adamw_grad_norm(A.F16, gls[k], s, norm if k else None, found if k else None, accumulate=k > 0, stream=st)
            A.adamw_tensor_norms(A.F16, gls[k], per[k], stream=st)
        for k, c in enumerate(groups):
            clipped(c, hp_pair(weight_decay=decay[k])[0], A.GradClip(s, 0.02), found, tl=tls[k], d_scale=scale, scaler=rule,
                    stream=st, advance_scale=k == 1)

    def expect(scale_before):
        total = math.fsum(float((c.arena.view("g", i).double() ** 2).sum()) for c in groups for i in range(len(c.numels)))
        if not math.isfinite(total):
            return None
        inv = float(np.float32(1.0 / scale_before))
        return multiplier(total, inv, 0.02, 1e-6)[0]

    torch.cuda.synchronize()
    graph, scales = None, []
    for k in range(5):
        for c in groups:
            c.refill_grads(k)
        if k == 1:
            groups[0].arena.view("g", 1)[512] = float("-inf")
            groups[0].host["g"] = to_np(groups[0].arena.bufs["g"])
        torch.cuda.synchronize()
        mult = expect(scale[0].item())
        with torch.cuda.stream(st):
            if k == 2:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=st):
                    iteration()
            if graph is None:
                iteration()
            else:
                graph.replay()
        torch.cuda.synchronize()
        _ = torch.ones(1 << 20, device="cuda").sum().item()
        assert (found.item() == 1) == (mult is None)
        assert norm.item() == float(np.float32(math.sqrt(s.item())))
        if mult is not None:
            sq = sum(float((p.double() ** 2).sum()) for p in per)
            assert abs(sq - s.item()) <= s.item() * 2 * (2.0 ** -24 + 2.0 ** -40)
            for c, wd in zip(groups, decay):
                c.oracle_step(hp_pair(inv_scale=mult, weight_decay=wd)[1])
        for c in groups:
            c.compare_all(f"two-groups-{limit}-{k}")
        scales.append(scale[0].item())
    # 1 clean, an overflow (512), 2 clean (back to 1024), 1 clean
    assert scales == [1024.0, 512.0, 512.0, 1024.0, 1024.0]
    del graph
    free()


def test_clipping_in_place_then_the_plain_step():
    """For a step that takes no clipping factor (the allocation-free one): clip in place, then step."""
    a, b = (Case("mixed", [30_000, 5], seed=310) for _ in range(2))
    s = torch.zeros(1, dtype=torch.float64, device="cuda")
    for c in (a, b):
        A.adamw_grad_norm(A.BF16, grads_of(c), s)
        A.adamw_clip_grads(A.BF16, grads_of(c), A.GradClip(s, 0.01))
    f = multiplier(s.item(), 1.0, 0.01, 1e-6)[1]
    g0 = torch.from_numpy(a.host["g"].view(np.int16).copy()).cuda().view(torch.bfloat16)
    for o, n in zip(a.arena.offsets, a.numels):
        assert same_bits(a.arena.bufs["g"][o:o + n], (g0[o:o + n].float() * float(np.float32(f))).bfloat16())
    a.host["g"] = to_np(a.arena.bufs["g"])
    hg, ho = hp_pair()
    a.gpu_step(hg)
    A.adamw_multi_tensor_step_noalloc(A.MIXED, A.BF16, b.tensor_list(), hg, b.d_step)
    a.oracle_step(ho)
    a.compare_all("clip-in-place")
    assert all(same_bits(a.arena.bufs[k], b.arena.bufs[k]) for k in a.keys)
    free()


@pytest.mark.parametrize("mode", ["mixed", "kahan"])
def test_one_list_with_blocked_state_for_norm_and_step(mode):
    """The norm and the clipped step on one list whose state is blocked on the padded flat
    index: the norm looks at the gradients alone."""
    case = Case(mode, SIZES, seed=311, align_elems=8, random_moments=True)
    n = range(len(SIZES))
    state = [[case.arena.view(k, i) for i in n] for k in case.keys[2:]]
    blocked, mask = A.make_blocked_state(MODE[mode], A.BF16, SIZES, *state)
    tl = A.TensorList(SIZES, [[case.arena.view(k, i) for i in n] for k in ("p", "g")] + [[blocked], None, None],
                      flat_mask=mask)
    s = torch.zeros(1, dtype=torch.float64, device="cuda")
    for _ in range(2):
        A.adamw_grad_norm(A.BF16, tl, s)
        clipped(case, hp_pair()[0], A.GradClip(s, 0.01), tl=tl)
        case.oracle_step(hp_pair(inv_scale=multiplier(s.item(), 1.0, 0.01, 1e-6)[0])[1])
    want = math.fsum(float((case.arena.view("g", i).double() ** 2).sum()) for i in n)
    # each of the two sums is within n * 2^-53 of the exact one
    assert abs(s.item() - want) <= 2 * sum(SIZES) * 2.0 ** -53 * want
    A.adamw_blocked_state_copy(MODE[mode], A.BF16, A.TensorList(SIZES, [None, None, *state], flat_mask=A.FLAT_PAD8), blocked,
                               to_blocked=False)
    case.compare_all(f"norm-and-step-blocked-{mode}")
    free()


def test_host_threads_each_on_their_stream():
    """Four host threads, each with lists and a stream of its own, run norm, clipping and step
    at once; each gets what it gets alone."""
    def work(k, out):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            case = Case("mixed", [20_000 + 7 * k, 5, 300], seed=320 + k, align_elems=1)
            s = torch.zeros(1, dtype=torch.float64, device="cuda")
            st.synchronize()
            for _ in range(5):
                A.adamw_grad_norm(A.BF16, grads_of(case), s)
                A.adamw_clip_grads(A.BF16, grads_of(case), A.GradClip(s, 0.05))
                clipped(case, hp_pair()[0], A.GradClip(s, 0.03))
            st.synchronize()
            out[k] = (case, s.item())

    alone, together = {}, {}
    for k in range(4):
        work(k, alone)
    threads = [threading.Thread(target=work, args=(k, together)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for k in range(4):
        (a, sa), (b, sb) = alone[k], together[k]
        assert sa == sb and b.d_step.item() == 5
        assert all(same_bits(a.arena.bufs[x], b.arena.bufs[x]) for x in a.keys), k
    free()
