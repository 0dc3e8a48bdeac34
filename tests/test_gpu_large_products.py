"""Matrices of more than 64 rows and columns against their definition in 64 bits, through the update that a step makes of
them (test_gpu_small_products.py), on spectra where single roundings count: low rank, one direction and weak noise, one
step and many.

The tolerance is the distance of the documented roundings, modelled in 64 bits, from the definition, and a quarter of it
more: where an fp32 sum differs in its last bits an element of A, B or X may be rounded the other way, which moves it as
much as rounding did, but the same number of elements is rounded by steps of the same size.  2^-13 is for models that
hardly round at all, of one step, where the fp32 sums' own roundings show.  And where X has no singular value those
roundings grow like any other: an element of the next X is a sum of s / 16 matrix instructions, the linear term and lo's
part (s: the shorter side), rounded to fp32 after each, by 0.41 2^-24 of the partial sum in the root mean square, at
random.  Partial sums are a X and a part of B X, or a part of B X before a X joins it, and B lies in [-2.75, 0]: at most
a |X|.  So 0.41 a sqrt(s / 16 + 2) 2^-24 of |X| together, which every later step multiplies by a at most.
"""
import math

import pytest
import torch

import adamw_optimizer_step_apply_amd as A
from muon_util import f32, far, gradient, ns64
import test_gpu_orthogonalize
from test_gpu_small_products import far_from_rank_one, results, tolerance, updates

pytestmark = pytest.mark.gpu
SHAPES = [(65, 65), (128, 512), (512, 100), (300, 300), (768, 768), (66, 4000)]
KINDS = ["normal", "decay", "rank 1", "rank 8", "rank 60", "rank 1 + 1e-1", "rank 1 + 1e-2", "rank 1 + 1e-3", "rank 8 + 1e-3"]


def documented(u, ns, diagonal_steps=3):
    """The products with the roundings that the header documents, every sum in 64 bits."""
    h = lambda x: x.to(torch.float16).double()  # noqa: E731
    a, b, c = f32(ns.a), f32(ns.b), f32(ns.c)
    x = u.double()
    x = x / (x.norm() + f32(ns.eps)) * 2.0 ** 14
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for k in range(ns.steps):
        hi = h(x)
        lo = h((x - hi) * 2048.0) / 2048.0
        g = hi @ hi.T * 2.0 ** -14
        gh = h(g)
        e = (g - gh).diagonal()
        p = (b * (gh + torch.diag(e)) + c * (gh @ gh + (e[:, None] + e[None, :]) * gh) * 2.0 ** -14) * 2.0 ** -2
        ph = h(p)
        rest = (p - ph).diagonal()[:, None] * 2.0 ** -12
        of_lo = a + (p.diagonal()[:, None] * 2.0 ** -12 if k + diagonal_steps >= ns.steps else 0.0)
        x = (a + rest) * hi + ph @ hi * 2.0 ** -12 + of_lo * lo
    return (x.T if tall else x) * 2.0 ** -14


def matrix(kind, shape, gen):
    rand = lambda *s: torch.randn(s, device="cuda", generator=gen, dtype=torch.float64)  # noqa: E731
    x = rand(*shape)
    if kind == "decay":
        u, _, v = torch.linalg.svd(x.cpu(), full_matrices=False)
        x = (u * torch.arange(1, min(shape) + 1, dtype=torch.float64) ** -1.0 @ v).cuda()
    elif kind != "normal":
        rank, _, noise = kind[5:].partition(" + ")
        k = int(rank)
        x = rand(shape[0], k) @ rand(k, shape[1]) / math.sqrt(k) + (float(noise) if noise else 0.0) * x
    return (x * 1e-3).float()


def sums(shape, ns):
    one = 0.41 * ns.a * math.sqrt(min(shape) / 16 + 2) * 2.0 ** -24
    return one * sum(ns.a ** k for k in range(ns.steps))


def check(us, ns, diagonal_steps=3):
    for o, u in zip(updates(us, ns), us):
        true = ns64(u, ns)
        model = far(documented(u, ns, diagonal_steps), true)
        assert far(o, true) <= 1.25 * model + 2.0 ** -13 + sums(u.shape, ns), (tuple(u.shape), far(o, true), model)


@pytest.mark.parametrize("steps", [1, 2, 3, 5, 8, 9])
@pytest.mark.parametrize("kind", KINDS)
def test_update_of_spectra(kind, steps):
    gen = torch.Generator(device="cuda").manual_seed(70)
    check([matrix(kind, s, gen) for s in SHAPES], A.NewtonSchulz(steps=steps))


# The bounds that the header states for these sizes, of any spectrum: a quarter more than the largest that the model
# gave over 20 matrices of each kind, and the sums' part at 768.
BOUNDS = [(1, 1e-3), (2, 1e-3), (3, 1.5e-3), (4, 2e-3), (5, 3.5e-3), (7, 5e-3), (8, 8e-3), (9, 2.5e-2)]


@pytest.mark.parametrize("steps,most", BOUNDS)
@pytest.mark.parametrize("kind", KINDS)
def test_documented_bounds(kind, steps, most):
    gen = torch.Generator(device="cuda").manual_seed(71)
    ns = A.NewtonSchulz(steps=steps)
    us = [matrix(kind, s, gen) for s in SHAPES + [(65, 65)] * 8]
    for o, u in zip(updates(us, ns), us):
        assert far(o, ns64(u, ns)) <= most, tuple(u.shape)


@pytest.mark.parametrize("coefficients,diagonal_steps", [((1.5, -0.5, 0.0), 7), ((1.875, -1.25, 0.375), 5)])
@pytest.mark.parametrize("kind", ["normal", "rank 8", "rank 1 + 1e-2"])
def test_other_coefficients(kind, coefficients, diagonal_steps):
    """Steps in which B's diagonal takes part with lo: those after which the others multiply by at most 16 together."""
    gen = torch.Generator(device="cuda").manual_seed(72)
    check([matrix(kind, s, gen) for s in SHAPES], A.NewtonSchulz(*coefficients, steps=8), diagonal_steps)


# long matrices, whose sums go in two levels, and one whose sums do not
LONG = [(65, 4194304), (8388609, 66), (130, 1048576), (300, 400000), (65, 262144)]


@pytest.mark.parametrize("signs", [False, True])
@pytest.mark.parametrize("shape", LONG)
def test_long_matrices_of_rank_one(shape, signs):
    """Equal columns (but for their sign) add up like terms, whose roundings in fp32 add up too.  The length is no reason
    for more than the header's bound of five steps."""
    gen = torch.Generator(device="cuda").manual_seed(73)
    short, long = min(shape), max(shape)
    left, right = torch.randn(short, device="cuda", generator=gen) * 1e-3, torch.ones(long, device="cuda")
    if signs:
        right = torch.where(torch.rand(long, device="cuda", generator=gen) < 0.5, -right, right)
    wide = shape[0] < shape[1]
    ns = A.NewtonSchulz()
    o = updates([torch.outer(left, right) if wide else torch.outer(right, left)], ns)[0]
    assert far_from_rank_one(o if wide else o.T, left, right, ns) <= 3.5e-3


def test_a_long_matrix_changes_no_other_s_bits():
    """Next to one, the others' squares go through the same launches, in one level as by themselves."""
    gen = torch.Generator(device="cuda").manual_seed(74)
    us = [matrix("normal", s, gen) for s in [(100, 200), (66, 200000), (768, 768), (66, 300001)]]
    ns = A.NewtonSchulz()
    alone = [updates([u], ns)[0] for u in us]
    assert all(torch.equal(x, y) for x, y in zip(alone, updates(us, ns)))
    for o, u in zip(alone, us):
        assert far(o, ns64(u, ns)) <= 3.5e-3


@pytest.mark.parametrize("name", list(test_gpu_orthogonalize.SHAPES))
def test_lists(name):
    """Every list that adamw_orthogonalize is tested on, at the tolerance of its sort; and what adamw_orthogonalize makes
    of it is the step's O rounded to bf16, bit for bit."""
    gen = torch.Generator().manual_seed(75)
    us = [gradient(r, c, gen).float().cuda() for r, c in test_gpu_orthogonalize.SHAPES[name]]
    ns = A.NewtonSchulz()
    for o, u, rounded in zip(updates(us, ns), us, results(us)):
        true = ns64(u, ns)
        most = tolerance(ns) if min(u.shape) <= 64 else 1.25 * far(documented(u, ns), true) + 2.0 ** -13 + sums(u.shape, ns)
        assert far(o, true) <= most, (tuple(u.shape), far(o, true), most)
        assert torch.equal(o.bfloat16(), rounded), tuple(u.shape)
