"""Matrices of at most 64 on the shorter side against their definition in 64 bits, through the update that a step makes of
them: a mixed step from master weights of zero with lr 1 and no decay leaves w = -O, O as the step uses it, in fp32 and
without a 16-bit rounding.  With no gradient and a momentum of 1/2, u is half of the momentum given, exactly.

Tolerances, relative in the Frobenius norm.  Everything but u and O is in 64 bits.  A run of at most 7 steps goes on
polynomials of one Gram matrix: at most three symmetric products a step, each rounded by at most 2^-53 of its elements,
so by 2^-53 sqrt(64) of their largest eigenvalue; and a step multiplies what is wrong in the Gram matrix by at most a^2:
3 K 8 a^(2 K) 2^-53 after K steps.  Between two runs X is rounded to fp32, by 2^-24, and every step after that multiplies that by a
at most; the result's norm is at least 0.68 that of X.  O's own rounding is 2^-24.
"""
import pytest
import torch

import adamw_optimizer_step_apply_amd as A
from muon_util import f32, far, ns64

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


def tolerance(ns):
    runs = -(-ns.steps // 7)
    run = -(-ns.steps // runs)
    held = 3 * run * 8 * ns.a ** (2 * run) * 2.0 ** -53
    return 2.0 ** -24 + held + sum((held + 1.5 * 2.0 ** -24) * ns.a ** (ns.steps - k * run) for k in range(1, runs))


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


SHAPES = [(64, 64), (64, 2048), (16, 768), (768, 16), (17, 33), (48, 100), (33, 5000), (20001, 49), (4, 64), (1, 300),
          (300, 1), (1, 1)]
KINDS = {"full": None, "rank_one": 0.0, "noise_1e-1": 1e-1, "noise_1e-2": 1e-2, "noise_3e-3": 3e-3, "noise_1e-4": 1e-4}


def matrices(kind, gen, shapes=SHAPES):
    """Normal matrices, or one direction and so much noise."""
    rand = lambda *s: torch.randn(s, device="cuda", generator=gen, dtype=torch.float64)  # noqa: E731
    noise = KINDS[kind]
    return [(rand(r, c) if noise is None else rand(r, 1) * rand(1, c) + noise * rand(r, c)).float() * 1e-3
            for r, c in shapes]


@pytest.mark.parametrize("steps", [1, 3, 5, 7, 8, 12, 16])
@pytest.mark.parametrize("kind", list(KINDS))
def test_update_of_spectra(kind, steps):
    gen = torch.Generator(device="cuda").manual_seed(61)
    us, ns = matrices(kind, gen), A.NewtonSchulz(steps=steps)
    for o, u in zip(updates(us, ns), us):
        assert far(o, ns64(u, ns)) <= tolerance(ns), (tuple(u.shape), far(o, ns64(u, ns)), tolerance(ns))


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["full", "noise_1e-2"])
def test_results_are_the_definition_s_rounded_once(name, kind):
    """An element is off by half a step of bf16, 2^-8 of it, and the tolerance above."""
    code, dtype = {"f32": (A.F32, torch.float32), "bf16": (A.BF16, torch.bfloat16), "f16": (A.F16, torch.float16)}[name]
    gen = torch.Generator(device="cuda").manual_seed(62)
    us = [u.to(dtype) for u in matrices(kind, gen)]
    outs = [torch.zeros(u.shape, dtype=torch.bfloat16, device="cuda") for u in us]
    ml = A.MatrixList(SHAPES, [outs, us])
    A.adamw_orthogonalize(code, ml, A.make_orthogonalize_workspace(ml))
    torch.cuda.synchronize()
    for o, u in zip(outs, us):
        want = ns64(u)
        most = 2.0 ** -8 * want.abs() + tolerance(A.NewtonSchulz()) * want.norm()
        assert bool(((o.double() - want).abs() <= most).all()), tuple(u.shape)


@pytest.mark.parametrize("magnitude", [1e-35, 1e-12, 1e12, 1e35])
def test_magnitudes(magnitude):
    gen = torch.Generator(device="cuda").manual_seed(63)
    ns = A.NewtonSchulz(eps=0.0)
    us = [(u.double() * 1e3 * magnitude).float() for u in matrices("full", gen)]
    for o, u in zip(updates(us, ns), us):
        assert far(o, ns64(u.double() / magnitude, ns)) <= tolerance(ns), tuple(u.shape)


def test_a_norm_far_below_eps():
    """X is then as small as that, and what the steps make of it is a^5 X."""
    gen = torch.Generator(device="cuda").manual_seed(64)
    us = [u * 1e-20 for u in matrices("full", gen)]
    for o, u in zip(updates(us, A.NewtonSchulz()), us):
        assert far(o, ns64(u)) <= tolerance(A.NewtonSchulz()), tuple(u.shape)


COMPANY = [(16, 48), (300, 520), (64, 64), (65, 66), (700, 30), (1, 9), (520, 260), (33, 5000)]


def results(us, least=False):
    outs = [torch.zeros(u.shape, dtype=torch.bfloat16, device="cuda") for u in us]
    ml = A.MatrixList([tuple(u.shape) for u in us], [outs, us])
    n = A.adamw_orthogonalize_workspace_bytes(ml, least=least)
    A.adamw_orthogonalize(A.F32, ml, torch.full((n,), 0x7e, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    return outs


def test_a_matrix_has_the_same_bits_alone_in_company_and_batch_by_batch():
    gen = torch.Generator(device="cuda").manual_seed(65)
    us = matrices("noise_1e-2", gen, COMPANY)
    alone = [results([u])[0] for u in us]
    for got in (results(us), results(us, least=True), results(us + matrices("full", gen, [(768, 768)] * 24))):
        assert all(torch.equal(x, y) for x, y in zip(alone, got))
    ns, one = A.NewtonSchulz(), [updates([u], A.NewtonSchulz())[0] for u in us]
    assert all(torch.equal(x, y) for x, y in zip(one, updates(us, ns)))
    assert all(torch.equal(x, y) for x, y in zip(one, updates(us, ns, matrices("full", gen, [(768, 768)] * 24))))
    for o, u in zip(one, us):
        if min(u.shape) <= 64:
            assert far(o, ns64(u)) <= tolerance(ns)


@pytest.mark.parametrize("flag", [0, 1])
def test_a_skipped_step_of_both_sorts(flag):
    """The counter goes on once for all batches, small matrices' or others', and not at all under the flag."""
    gen = torch.Generator(device="cuda").manual_seed(66)
    ms = matrices("full", gen, COMPANY)
    p, g = ([torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in COMPANY] for _ in range(2))
    kept, w = [m.clone() for m in ms], [torch.zeros(s, device="cuda") for s in COMPANY]
    ml = A.MatrixList(COMPANY, [p, g, ms, None, w])
    ws = torch.empty(A.adamw_orthogonalize_workspace_bytes(ml, least=True), dtype=torch.uint8, device="cuda")
    d_step, found = (torch.tensor([v], dtype=torch.int32, device="cuda") for v in (6, flag))
    A.adamw_muon_multi_tensor_step(A.MIXED, A.BF16, ml, A.MuonHParams(), d_step, ws, d_found_inf=found)
    torch.cuda.synchronize()
    assert int(d_step) == 7 - flag
    for m, k, x in zip(ms, kept, w):
        assert torch.equal(m, k) == bool(flag) and bool((x == 0).all()) == bool(flag)
