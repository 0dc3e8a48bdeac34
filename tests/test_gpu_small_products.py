"""Matrices of at most 64 on the shorter side against their definition in 64 bits, through the update that a step makes of
them: a mixed step from master weights of zero with lr 1 and no decay leaves w = -O, O as the step uses it, in fp32 and
without a 16-bit rounding.  With no gradient and a momentum of 1/2, u is half of the momentum given, exactly."""
import pytest
import torch

import adamw_optimizer_step_apply_amd as A
from muon_util import f32

pytestmark = pytest.mark.gpu


def updates(us, ns, company=()):
    """O of each matrix of `us` (fp32 on the GPU), with the matrices of `company` in the same list."""
    every = list(us) + list(company)
    shapes = [tuple(u.shape) for u in every]
    p, g = ([torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in shapes] for _ in range(2))
    m, w = [2.0 * u for u in every], [torch.zeros(s, device="cuda") for s in shapes]
    mats = A.MatrixList(shapes, [p, g, m, None, w])
    ws = A.make_orthogonalize_workspace(mats)
    hp = A.MuonHParams(lr=1.0, momentum=0.5, weight_decay=0.0, nesterov=False, scaling=A.MUON_SCALE_NONE, ns=ns)
    A.adamw_muon_multi_tensor_step(A.MIXED, A.BF16, mats, hp, torch.zeros(1, dtype=torch.int32, device="cuda"), ws)
    torch.cuda.synchronize()
    assert all(torch.equal(x, u) for x, u in zip(m, every))
    return [-x for x in w[:len(us)]]


def polynomial(x, ns):
    for _ in range(ns.steps):
        x = f32(ns.a) * x + f32(ns.b) * x ** 3 + f32(ns.c) * x ** 5
    return x


def far_from_rank_one(o, left, right, ns):
    """Relative distance of o from the products of left (outer) right, whose one singular value goes through the
    polynomial."""
    n = float(left.double().norm() * right.double().norm())
    want = torch.outer(left.double(), right.double() * (polynomial(n / (n + f32(ns.eps)), ns) / n))
    return float((o.double() - want).norm() / want.norm())


LONG = [(16, 4194304, 5), (16, 524288, 6), (16, 152064, 7), (64, 1048576, 7), (5, 2097152, 7), (500000, 16, 7)]


@pytest.mark.parametrize("signs", [False, True])
@pytest.mark.parametrize("rows,cols,steps", LONG)
def test_long_matrices_of_rank_one(rows, cols, steps, signs):
    """Rows that are constant (or constant but for the sign of a column) add up like terms, whose roundings add up too.
    The tolerance is that of short matrices of rank one (test_gpu_orthogonalize_edges.py): the length is no reason for
    more."""
    gen = torch.Generator(device="cuda").manual_seed(60)
    short, long = min(rows, cols), max(rows, cols)
    left = torch.randn(short, device="cuda", generator=gen) * 1e-3
    right = torch.ones(long, device="cuda")
    if signs:
        right = torch.where(torch.rand(long, device="cuda", generator=gen) < 0.5, -right, right)
    u = torch.outer(left, right) if rows < cols else torch.outer(right, left)
    ns = A.NewtonSchulz(steps=steps)
    o = updates([u], ns)[0]
    assert bool(torch.isfinite(o).all())
    assert far_from_rank_one(o if rows < cols else o.T, left, right, ns) <= 3 * steps * 8 * ns.a ** steps * 2.0 ** -23
