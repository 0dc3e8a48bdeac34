"""Newton-Schulz products where their error grows: matrices of low rank and many steps, for matrices of at most 64
on the shorter side by themselves and in other company; and the calls of such lists in graphs and on two streams.

The tolerance of full-rank matrices is that of test_gpu_orthogonalize.py.  Of a matrix of rank one, a step multiplies what
rounding left in the other directions by a = 3.4445.  Small matrices by themselves hold at most three symmetric products a step
in 22 bits, each rounded by at most 2^-23 of its elements, so by 2^-23 sqrt(64) of their largest eigenvalue in the
Frobenius norm: with K steps 3 K 8 a^K 2^-23 together.
"""
import pytest
import torch

import adamw_optimizer_step_apply_amd as A
from muon_util import Arena, far, gradient, ns64
from test_gpu_orthogonalize import TOL_BF16, TOL_NS, run

pytestmark = pytest.mark.gpu
SMALL = [(16, 64), (64, 700), (700, 40), (9, 9)]


def rank_one(r, c, gen):
    return torch.randn(r, 1, generator=gen, dtype=torch.float64) @ torch.randn(1, c, generator=gen, dtype=torch.float64)


@pytest.mark.parametrize("company", [[], [(65, 66)]])
@pytest.mark.parametrize("steps", [6, 7, 8, 9, 12, 16])
def test_many_steps_of_small_matrices(steps, company):
    gen = torch.Generator().manual_seed(30)
    ns = A.NewtonSchulz(steps=steps)
    outs, ins = run([gradient(r, c, gen) for r, c in SMALL + company], "f32", ns)
    for o, u in zip(outs, ins):
        assert far(o, ns64(u, ns)) <= TOL_NS + TOL_BF16, (tuple(u.shape), far(o, ns64(u, ns)))


@pytest.mark.parametrize("steps", [1, 3, 5, 7])
def test_small_matrices_of_rank_one(steps):
    gen = torch.Generator().manual_seed(31)
    ns = A.NewtonSchulz(steps=steps)
    outs, ins = run([rank_one(r, c, gen) for r, c in SMALL], "f32", ns)
    for o, u in zip(outs, ins):
        # what the inputs' own rounding to fp32 put there is the definition's too
        assert far(o, ns64(u, ns)) <= 3 * steps * 8 * ns.a ** steps * 2.0 ** -23 + TOL_BF16, tuple(u.shape)


@pytest.mark.parametrize("shapes", [SMALL, SMALL + [(65, 65)], [(65, 65), (300, 200)]])
@pytest.mark.parametrize("steps", [8, 9, 12, 16])
def test_rank_one_and_many_steps_keep_to_the_map_s_range(steps, shapes):
    """Rounding may fill the absent directions, but like singular values: none passes the map's largest value 1.21."""
    gen = torch.Generator().manual_seed(32)
    outs, _ = run([rank_one(r, c, gen) for r, c in shapes], "f32", A.NewtonSchulz(steps=steps))
    for o in outs:
        assert bool(torch.isfinite(o).all()), tuple(o.shape)
        assert float(torch.linalg.svdvals(o.double().cpu())[0]) <= 1.3, tuple(o.shape)


def test_small_lists_captured_and_replayed():
    gen = torch.Generator().manual_seed(33)
    us = [gradient(r, c, gen) for r, c in SMALL]
    a_in, a_out = Arena(us, torch.bfloat16), Arena([0 * u for u in us], torch.bfloat16)
    mats = A.MatrixList(SMALL, [a_out.views(), a_in.views()])
    ws = A.make_orthogonalize_workspace(mats)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        A.adamw_orthogonalize(A.BF16, mats, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            A.adamw_orthogonalize(A.BF16, mats, ws)
    for k in range(4):
        new = [gradient(r, c, gen) for r, c in SMALL]
        for v, u in zip(a_in.views(), new):
            v.copy_(u.bfloat16())
        ws.fill_(255)   # what other work may leave there
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        replayed = [v.clone() for v in a_out.views()]
        eager, _ = run(new, "bf16")
        assert all(torch.equal(x, y) for x, y in zip(replayed, eager)), k


def test_two_graphs_share_a_workspace_in_turn():
    """Replays that do not overlap in time may share one: every part is written before it is read."""
    gen = torch.Generator().manual_seed(34)
    lists = [SMALL, [(100, 200), (64, 64)]]
    st = torch.cuda.Stream()
    made = []
    for shapes in lists:
        us = [gradient(r, c, gen) for r, c in shapes]
        a_in, a_out = Arena(us, torch.float32), Arena([0 * u for u in us], torch.bfloat16)
        made.append((us, a_in, a_out, A.MatrixList(shapes, [a_out.views(), a_in.views()])))
    ws = torch.empty(max(A.adamw_orthogonalize_workspace_bytes(m[3]) for m in made), dtype=torch.uint8, device="cuda")
    st.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(st):
        for m in made:
            A.adamw_orthogonalize(A.F32, m[3], ws)
        torch.cuda.synchronize()
        for m in made:
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=st):
                A.adamw_orthogonalize(A.F32, m[3], ws)
    for _ in range(3):
        for m in made:
            for v in m[2].views():
                v.zero_()
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
            torch.cuda.synchronize()
        for us, _, a_out, _ in made:
            eager, _ = run(us, "f32")
            assert all(torch.equal(x, y) for x, y in zip(a_out.views(), eager))


def test_one_matrix_read_twice():
    """An input may be in a list more than once; its results are each one's own."""
    gen = torch.Generator().manual_seed(35)
    u = gradient(70, 90, gen).float().cuda()
    outs = [torch.zeros(70, 90, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    mats = A.MatrixList([(70, 90)] * 2, [outs, [u, u]])
    A.adamw_orthogonalize(A.F32, mats, A.make_orthogonalize_workspace(mats))
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and far(outs[0], ns64(u)) <= TOL_NS + TOL_BF16


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gap,phase", [(8, 0), (1, 3)])
def test_runs_of_steps_of_long_and_unaligned_matrices(dtype, gap, phase):
    """Nine steps go in two runs, with X in the workspace between them; workgroups of one and of several tiles."""
    gen = torch.Generator().manual_seed(36)
    ns = A.NewtonSchulz(steps=9)
    outs, ins = run([gradient(r, c, gen) for r, c in [(9, 20001), (5000, 33), (64, 64), (1, 4097), (63, 130)]], dtype, ns, gap, phase)
    for o, u in zip(outs, ins):
        assert far(o, ns64(u, ns)) <= TOL_NS + TOL_BF16, (tuple(u.shape), far(o, ns64(u, ns)))


def test_runs_of_steps_in_place_with_zeros_and_nan():
    gen = torch.Generator().manual_seed(37)
    ns = A.NewtonSchulz(steps=12)
    us = [gradient(30, 500, gen), torch.zeros(40, 70, dtype=torch.float64), gradient(20, 20, gen), gradient(50, 90, gen)]
    us[2][3, 4] = float("nan")
    outs, ins = run(us, "bf16", ns, inplace=True)
    assert far(outs[0], ns64(ins[0], ns)) <= TOL_NS + TOL_BF16 and far(outs[3], ns64(ins[3], ns)) <= TOL_NS + TOL_BF16
    assert bool((outs[1] == 0).all()) and bool(torch.isnan(outs[2]).all())


def test_runs_of_steps_captured_and_replayed():
    gen = torch.Generator().manual_seed(38)
    ns = A.NewtonSchulz(steps=16)
    us = [gradient(r, c, gen) for r, c in SMALL]
    a_in, a_out = Arena(us, torch.float16), Arena([0 * u for u in us], torch.bfloat16)
    mats = A.MatrixList(SMALL, [a_out.views(), a_in.views()])
    ws = A.make_orthogonalize_workspace(mats)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        A.adamw_orthogonalize(A.F16, mats, ws, ns)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            A.adamw_orthogonalize(A.F16, mats, ws, ns)
    eager, _ = run(us, "f16", ns)
    for k in range(3):
        for v in a_out.views():
            v.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a_out.views(), eager)), k
