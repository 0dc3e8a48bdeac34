"""The Muon step's rarer calls: skips over several batches and over nothing, many steps of small matrices, and small lists in
graphs and on two streams at once.  Compared with the eager call of the same list, bit for bit, and with the
definition in 64 bits at the tolerance of test_gpu_muon_step.py."""
import pytest
import torch

import adamw_optimizer_step_apply_amd as A
from muon_util import Arena, far, gradient, ns64
from test_gpu_muon_step import LISTS, TOL_NS, hparams, momentum, state, step, update_of

pytestmark = pytest.mark.gpu
SMALL = LISTS["small"] + [(64, 900)]


@pytest.mark.parametrize("shapes", [SMALL, LISTS["larger"] + LISTS["odd"]])
@pytest.mark.parametrize("skip", [False, True])
def test_batches_of_one_matrix_each_under_the_flag(shapes, skip):
    hp = hparams()
    g, m, w = state(shapes, torch.bfloat16, torch.float32, 50)
    p = [x.bfloat16() for x in w]
    n = A.adamw_orthogonalize_workspace_bytes(A.MatrixList(shapes, [[]] * 5), least=True)
    found = torch.tensor([int(skip)], dtype=torch.int32, device="cuda")
    arenas, t = step(shapes, [p, g, m, w], A.MIXED, A.BF16, hp, found=found,
                     workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))
    assert t == 4 + (not skip)
    for i, v in enumerate(arenas[2].views()):
        assert torch.equal(v.cpu(), m[i] if skip else momentum(g[i], m[i], hp, 1.0)[0])
    for v, x in zip(arenas[3].views(), w):
        assert torch.equal(v.cpu(), x) == skip


@pytest.mark.parametrize("counter,flag,after", [(7, 1, 7), (7, 0, 8), (2 ** 31 - 1, 0, 2 ** 31 - 1), (-3, 0, -3)])
def test_lists_without_elements(counter, flag, after):
    d_step = torch.tensor([counter], dtype=torch.int32, device="cuda")
    found = torch.tensor([flag], dtype=torch.int32, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    none = [torch.empty(0, 5, dtype=t, device="cuda") for t in (torch.bfloat16, torch.bfloat16, torch.float32, torch.float32)]
    mats = A.MatrixList([(0, 5)], [[none[0]], [none[1]], [none[2]], None, [none[3]]])
    A.adamw_muon_multi_tensor_step(A.MIXED, A.BF16, mats, hparams(), d_step, ws, d_found_inf=found)
    torch.cuda.synchronize()
    assert int(d_step) == after


@pytest.mark.parametrize("steps", [7, 8, 12])
def test_many_steps_of_small_matrices(steps):
    hp = hparams(ns=A.NewtonSchulz(steps=steps))
    g, m, _ = state(SMALL, torch.bfloat16, torch.float32, 51)
    for i, o in enumerate(update_of(SMALL, g, m, hp, A.BF16)):
        assert far(o, ns64(momentum(g[i], m[i], hp, 1.0)[1], hp.ns)) <= TOL_NS, SMALL[i]


def made(shapes, seed):
    g, m, w = state(shapes, torch.bfloat16, torch.float32, seed)
    arenas = [Arena(x, x[0].dtype) for x in ([x.bfloat16() for x in w], g, m, w)]
    mats = A.MatrixList(shapes, [arenas[0].views(), arenas[1].views(), arenas[2].views(), None, arenas[3].views()])
    return arenas, mats, A.make_orthogonalize_workspace(mats), torch.zeros(1, dtype=torch.int32, device="cuda")


def call(x, stream=None):
    A.adamw_muon_multi_tensor_step(A.MIXED, A.BF16, x[1], hparams(), x[3], x[2], stream=stream)


def test_a_small_list_captured_and_replayed():
    eager, cap = made(SMALL, 52), made(SMALL, 52)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call(cap)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            call(cap)
    call(eager)
    torch.cuda.synchronize()
    gen = torch.Generator().manual_seed(53)
    for k in range(3):
        for v, x in zip(eager[0][1].views(), cap[0][1].views()):
            new = gradient(*v.shape, gen).bfloat16()
            v.copy_(new)
            x.copy_(new)
        torch.cuda.synchronize()
        graph.replay()
        call(eager)
        torch.cuda.synchronize()
        assert int(eager[3]) == int(cap[3]) == k + 2
        assert all(torch.equal(x.buf, y.buf) for x, y in zip(eager[0], cap[0])), k


def test_two_lists_on_two_streams_at_once():
    here = [made(SMALL, 54), made(LISTS["odd"], 55)]
    there = [made(SMALL, 54), made(LISTS["odd"], 55)]
    torch.cuda.synchronize()
    for _ in range(5):
        for x in here:
            call(x)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in there]
    for _ in range(5):
        for x, st in zip(there, streams):
            call(x, st)
    torch.cuda.synchronize()
    for x, y in zip(here, there):
        assert int(x[3]) == int(y[3]) == 5
        assert all(torch.equal(a.buf, b.buf) for a, b in zip(x[0], y[0]))
