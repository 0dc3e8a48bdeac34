"""GPU: an iteration over many parameter groups keeps every list's table on the device.

A call under capture is refused where its table is not there, so an iteration that was
made once and then captures whole shows that no group's norm, clipping or step has
pushed another's table out."""
import pytest
import torch

import adamw_optimizer_step_apply_amd as A
from gpu_util import Case, free, hp_pair, same_bits
from test_gpu_clipped_step import clipped, grads_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("groups", [5, 6, 12])
def test_an_iteration_over_many_groups_is_captured_after_one_call_each(groups):
    """Norm over all groups, clipping in place, clipped step: eager on one set of buffers,
    captured and replayed on an equal one, the same bits after each of 3 iterations."""
    st = torch.cuda.Stream()
    sets = [[Case("mixed", [4000 + 8 * g, 5, 900], seed=700 + g, align_elems=1) for g in range(groups)] for _ in range(2)]
    sums = [torch.zeros(1, dtype=torch.float64, device="cuda") for _ in range(2)]
    tls = [[c.tensor_list() for c in cases] for cases in sets]
    gls = [[grads_of(c) for c in cases] for cases in sets]

    def iteration(i):
        for k in range(groups):
            A.adamw_grad_norm(A.BF16, gls[i][k], sums[i], accumulate=k > 0, stream=st)
        for k, c in enumerate(sets[i]):
            A.adamw_clip_grads(A.BF16, gls[i][k], A.GradClip(sums[i], 0.03), stream=st)
            clipped(c, hp_pair()[0], A.GradClip(sums[i], 0.01), tl=tls[i][k], stream=st)

    torch.cuda.synchronize()
    iteration(0)
    iteration(1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        iteration(1)
    for _ in range(3):
        iteration(0)
        with torch.cuda.stream(st):
            graph.replay()
        torch.cuda.synchronize()
        _ = torch.ones(1 << 20, device="cuda").sum().item()
        assert sums[0].item() == sums[1].item()
        for a, b in zip(*sets):
            assert a.d_step.item() == b.d_step.item()
            assert all(same_bits(a.arena.bufs[x], b.arena.bufs[x]) for x in a.keys)
    del graph
    free()


def test_twelve_lists_of_steps_are_captured_after_one_call_each():
    """More lists than the least that is kept: small tables all stay."""
    st = torch.cuda.Stream()
    cases = [Case("kahan", [3000 + 16 * g, 7], seed=720 + g, align_elems=8) for g in range(12)]
    tls = [c.tensor_list() for c in cases]
    hg, ho = hp_pair()
    torch.cuda.synchronize()
    for c, tl in zip(cases, tls):
        A.adamw_multi_tensor_step(A.PURE_KAHAN, A.BF16, tl, hg, c.d_step, stream=st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        for c, tl in zip(cases, tls):
            A.adamw_multi_tensor_step(A.PURE_KAHAN, A.BF16, tl, hg, c.d_step, stream=st)
    for _ in range(2):
        with torch.cuda.stream(st):
            graph.replay()
        torch.cuda.synchronize()
        _ = torch.ones(1 << 20, device="cuda").sum().item()
    for c in cases:
        for _ in range(3):
            c.oracle_step(ho)
        c.compare_all("twelve-lists")
    del graph
    free()


def test_more_lists_than_are_kept():
    """40 lists through one stream twice, a captured one among them: every call uses its
    own list's table, the evicted ones planned again, and the captured table stays."""
    st = torch.cuda.Stream()
    graphed = Case("mixed", [5000, 3], seed=740, align_elems=1)
    cases = [Case("mixed", [200 + 1000 * (g % 5), 7, 40_000 if g == 20 else 9], seed=741 + g, align_elems=1) for g in range(40)]
    hg, ho = hp_pair()
    tl, tls = graphed.tensor_list(), [c.tensor_list() for c in cases]
    torch.cuda.synchronize()
    A.adamw_multi_tensor_step(A.MIXED, A.BF16, tl, hg, graphed.d_step, stream=st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        A.adamw_multi_tensor_step(A.MIXED, A.BF16, tl, hg, graphed.d_step, stream=st)
    for _ in range(2):
        for c, t in zip(cases, tls):
            A.adamw_multi_tensor_step(A.MIXED, A.BF16, t, hg, c.d_step, stream=st)
        with torch.cuda.stream(st):
            graph.replay()
        torch.cuda.synchronize()
    for c, n in [(graphed, 3)] + [(c, 2) for c in cases]:
        for _ in range(n):
            c.oracle_step(ho)
        c.compare_all("forty-lists")
    del graph
    free()
