"""adamw_orthogonalize on the GPU against its definition in 64 bits.

Tolerances, relative in the Frobenius norm.  u = 2^-11 is fp16's half step.  A product step rounds five times to
fp16 (X on both sides of its Gram matrix, that matrix, the polynomial, X under it); as independent errors of the
elements each is at most 0.41 u in the root mean square (u / sqrt 3 over a binade of mantissas) times the
polynomial's largest value 2.8, together 2.6 u.  The singular values of the last steps lie in [0.68, 1.14], where the
map's slope is at most 1.6, so the last three steps give at most sqrt(1 + 1.6^2 + 2.6^2) = 3.2 times that: 8 u = 2^-8.
The result's rounding to bf16 adds at most 2^-8.
"""
import pytest
import torch

import adamw_optimizer_step_apply_amd as A
from muon_util import NS, Arena, far, gradient, ns64

pytestmark = pytest.mark.gpu
IN = {"f32": (A.F32, torch.float32), "bf16": (A.BF16, torch.bfloat16), "f16": (A.F16, torch.float16)}
TOL_NS, TOL_BF16 = 2.0 ** -8, 2.0 ** -8

SHAPES = {
    "one": [(1, 1)], "row": [(1, 300)], "column": [(257, 1)], "tiny": [(2, 3), (3, 2), (7, 7)],
    "wide_small": [(16, 768)], "tall_small": [(768, 16)], "square_64": [(64, 64)], "past_64": [(65, 63)],
    "odd": [(100, 37), (131, 257)], "edge_128": [(128, 129), (129, 128), (127, 128)],
    "wide": [(200, 1000)], "tall": [(1000, 200)], "long_sum": [(33, 20000)], "square_300": [(300, 300)],
    "edge_256": [(255, 257), (256, 256), (513, 256)], "mixed": [(64, 64), (1, 5), (700, 90), (90, 701), (320, 320)],
    "same": [(128, 256)] * 9, "large": [(1100, 1500)],
    # shorter sides of 64 at most throughout: several runs of columns, long runs, both orders
    "small_long": [(64, 2500), (3000, 50), (1, 5000), (7, 64)], "small_longer": [(9, 70001), (40000, 17)],
    # lists that take the larger tiles
    "many": [(768, 768)] * 24, "larger": [(2048, 4096), (4096, 2048)],
}


def run(us, dtype, ns=NS, gap=8, phase=0, workspace=None, inplace=False, stream=None):
    """The results of the matrices `us` (CPU, 64 bits), the inputs as the library read them, and the arenas."""
    code, t = IN[dtype]
    a_in = Arena(us, t, gap, phase)
    a_out = a_in if inplace else Arena([torch.zeros_like(u) for u in us], torch.bfloat16, gap, phase)
    inputs = [v.clone() for v in a_in.views()]
    mats = A.MatrixList([tuple(u.shape) for u in us], [a_out.views(), a_in.views()])
    ws = A.make_orthogonalize_workspace(mats) if workspace is None else workspace(mats)
    torch.cuda.synchronize()
    A.adamw_orthogonalize(code, mats, ws, ns, stream=stream)
    torch.cuda.synchronize()
    if not inplace:
        same = lambda x, y: torch.equal(x.view(torch.uint8), y.view(torch.uint8))  # noqa: E731  (a NaN equals itself)
        assert all(same(x, y) for x, y in zip(inputs, a_in.views())), "an input was written"
    assert a_in.guards_kept() and a_out.guards_kept(), "elements outside the matrices were written"
    return [v.clone() for v in a_out.views()], inputs


@pytest.mark.parametrize("dtype", list(IN))
@pytest.mark.parametrize("name", list(SHAPES))
def test_against_the_definition(name, dtype):
    gen = torch.Generator().manual_seed(len(name) * 7 + len(SHAPES[name]))
    outs, ins = run([gradient(r, c, gen) for r, c in SHAPES[name]], dtype)
    for o, u in zip(outs, ins):
        assert far(o, ns64(u)) <= TOL_NS + TOL_BF16, (tuple(u.shape), far(o, ns64(u)))


@pytest.mark.parametrize("shape", [(64, 67_200_001), (66_200_003, 65)])
def test_offsets_past_32_bits(shape):
    """More than 2^32 elements, bf16 in place, against polynomials of the Gram matrix in 64 bits at both ends."""
    r, c = shape
    gen = torch.Generator(device="cuda").manual_seed(25)
    u = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = u.view(-1)
    piece = 1 << 28
    for a in range(0, flat.numel(), piece):
        b = min(flat.numel(), a + piece)
        flat[a:b] = torch.randn(b - a, device="cuda", generator=gen)
    long = u if r < c else u.T                   # the short side first
    g = torch.zeros(min(shape), min(shape), dtype=torch.float64, device="cuda")
    for a in range(0, max(shape), 1 << 20):
        x = long[:, a:a + (1 << 20)].double().contiguous()
        g += x @ x.T.contiguous()
    norm = float(g.diagonal().sum().sqrt()) + 1e-7
    a, q = g / norm ** 2, torch.eye(min(shape), dtype=torch.float64, device="cuda")
    for _ in range(NS.steps):
        p = 3.4445 * torch.eye(min(shape), dtype=torch.float64, device="cuda") - 4.7750 * a + 2.0315 * a @ a
        q, a = p @ q, p @ a @ p
    ends = [(0, 5000), (max(shape) // 2, max(shape) // 2 + 5000), (max(shape) - 5000, max(shape))]
    want = [q @ long[:, b:e].double() / norm for b, e in ends]
    mats = A.MatrixList([shape], [[u], [u]])
    A.adamw_orthogonalize(A.BF16, mats, A.make_orthogonalize_workspace(mats))
    torch.cuda.synchronize()
    for (b, e), w in zip(ends, want):
        assert far(long[:, b:e], w) <= TOL_NS + TOL_BF16


@pytest.mark.parametrize("kind", ["normal", "decay", "momentum"])
@pytest.mark.parametrize("shape", [(64, 64), (200, 200), (96, 700), (520, 260)])
def test_spectra(shape, kind):
    gen = torch.Generator().manual_seed(11)
    outs, ins = run([gradient(*shape, gen, kind)], "f32")
    assert far(outs[0], ns64(ins[0])) <= TOL_NS + TOL_BF16


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1.0, 1e12, 1e30])
def test_any_magnitude(scale):
    """The norm is summed in binary64 and the quotient formed there: no overflow, no underflow."""
    gen = torch.Generator().manual_seed(12)
    ns = A.NewtonSchulz(eps=0.0)
    outs, ins = run([gradient(70, 90, gen) * scale * 1e3], "f32", ns)
    assert far(outs[0], ns64(ins[0].double() / scale, ns)) <= TOL_NS + TOL_BF16


def test_eps_dominates_a_small_matrix():
    gen = torch.Generator().manual_seed(13)
    ns = A.NewtonSchulz(eps=1.0, steps=1)
    outs, ins = run([gradient(40, 30, gen)], "f32", ns)
    assert far(outs[0], ns64(ins[0], ns)) <= TOL_NS + TOL_BF16


@pytest.mark.parametrize("gap,phase", [(0, 0), (1, 1), (3, 3), (8, 0), (5, 7)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_alignment(dtype, gap, phase):
    gen = torch.Generator().manual_seed(14)
    us = [gradient(r, c, gen) for r, c in [(33, 40), (40, 33), (8, 8), (129, 72)]]
    outs, ins = run(us, dtype, gap=gap, phase=phase if dtype == "bf16" else phase % 4)
    for o, u in zip(outs, ins):
        assert far(o, ns64(u)) <= TOL_NS + TOL_BF16


def test_in_place():
    gen = torch.Generator().manual_seed(15)
    us = [gradient(r, c, gen) for r, c in [(65, 130), (200, 30)]]
    apart, ins = run(us, "bf16")
    same, _ = run(us, "bf16", inplace=True)
    assert all(torch.equal(x, y) for x, y in zip(apart, same))


def test_zero_and_non_finite_matrices_keep_to_themselves():
    gen = torch.Generator().manual_seed(16)
    us = [gradient(r, c, gen) for r, c in [(80, 70), (64, 64), (70, 200), (30, 30), (96, 65), (5, 5)]]
    clean, _ = run(us, "f32")
    us[1] = us[1] * 0.0
    us[2][3, 150] = float("nan")
    us[3][7, 7] = float("inf")
    us[5][0, 0] = -float("inf")
    outs, _ = run(us, "f32")
    assert torch.equal(outs[0], clean[0]) and torch.equal(outs[4], clean[4])
    assert bool((outs[1] == 0).all())
    for i in (2, 3, 5):
        assert bool(torch.isnan(outs[i]).all()), i
    zero, _ = run([us[1]], "f32", A.NewtonSchulz(eps=0.0))
    assert bool((zero[0] == 0).all())


def test_empty_matrices_and_lists():
    gen = torch.Generator().manual_seed(17)
    us = [torch.zeros(0, 5, dtype=torch.float64), gradient(20, 30, gen), torch.zeros(0, 1, dtype=torch.float64)]
    outs, ins = run(us, "f32")
    assert far(outs[1], ns64(ins[1])) <= TOL_NS + TOL_BF16
    run([us[0]], "f32")
    mats = A.MatrixList([], [[], []])
    A.adamw_orthogonalize(A.F32, mats, torch.empty(512, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()


def test_batches_of_a_small_workspace_give_the_same_bits():
    gen = torch.Generator().manual_seed(18)
    shapes = [(300, 200), (64, 64), (200, 300), (128, 500), (1, 9), (310, 290)]
    us = [gradient(r, c, gen) for r, c in shapes]
    whole, _ = run(us, "bf16")

    def least(mats):
        n = A.adamw_orthogonalize_workspace_bytes(mats, least=True)
        assert n < A.adamw_orthogonalize_workspace_bytes(mats)
        ws = torch.full((n + 512,), 0x7e, dtype=torch.uint8, device="cuda")   # fp16 NaN bytes left by others
        return ws[:n]
    parts, _ = run(us, "bf16", workspace=least)
    for x, y in zip(whole, parts):
        assert far(x, y) <= 2 * TOL_NS + TOL_BF16   # another tile size sums in another order
    again, _ = run(us, "bf16", workspace=least)
    assert all(torch.equal(x, y) for x, y in zip(parts, again))


def test_workspace_contents_do_not_matter():
    gen = torch.Generator().manual_seed(19)
    us = [gradient(r, c, gen) for r, c in [(70, 130), (200, 64)]]
    filled = lambda v: lambda m: torch.full((A.adamw_orthogonalize_workspace_bytes(m),), v, dtype=torch.uint8, device="cuda")  # noqa: E731
    a, _ = run(us, "f16", workspace=filled(0))
    b, _ = run(us, "f16", workspace=filled(0xff))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("steps", [1, 2, 3, 6, 9])
def test_steps(steps):
    """Odd and even numbers of product steps end in different buffers."""
    gen = torch.Generator().manual_seed(20)
    ns = A.NewtonSchulz(steps=steps)
    outs, ins = run([gradient(r, c, gen) for r, c in [(90, 150), (150, 90)]], "f32", ns)
    for o, u in zip(outs, ins):
        assert far(o, ns64(u, ns)) <= TOL_NS + TOL_BF16


def test_other_coefficients():
    """The cubic iteration x (3 - x^2) / 2, whose values stay in [0, 1]."""
    gen = torch.Generator().manual_seed(21)
    ns = A.NewtonSchulz(1.5, -0.5, 0.0, steps=12)
    outs, ins = run([gradient(60, 200, gen, "normal")], "f32", ns)
    assert far(outs[0], ns64(ins[0], ns)) <= TOL_NS + TOL_BF16


def test_other_stream_and_two_streams_at_once():
    gen = torch.Generator().manual_seed(22)
    us = [gradient(r, c, gen) for r, c in [(256, 300), (100, 90)]]
    here, _ = run(us, "bf16")
    there, _ = run(us, "bf16", stream=torch.cuda.Stream())
    assert all(torch.equal(x, y) for x, y in zip(here, there))
    streams, made = [torch.cuda.Stream() for _ in range(2)], []
    for _ in streams:
        a_in, a_out = Arena(us, torch.bfloat16), Arena([0 * u for u in us], torch.bfloat16)
        mats = A.MatrixList([tuple(u.shape) for u in us], [a_out.views(), a_in.views()])
        made.append((a_in, a_out, mats, A.make_orthogonalize_workspace(mats)))
    torch.cuda.synchronize()
    for _ in range(3):
        for st, (_, _, mats, ws) in zip(streams, made):
            A.adamw_orthogonalize(A.BF16, mats, ws, stream=st)
    torch.cuda.synchronize()
    for _, a_out, _, _ in made:
        assert all(torch.equal(x, y) for x, y in zip(here, a_out.views()))


def test_captured_and_replayed():
    gen = torch.Generator().manual_seed(23)
    us = [gradient(r, c, gen) for r, c in [(130, 140), (64, 300), (300, 64)]]
    a_in, a_out = Arena(us, torch.float32), Arena([0 * u for u in us], torch.bfloat16)
    mats = A.MatrixList([tuple(u.shape) for u in us], [a_out.views(), a_in.views()])
    ws = A.make_orthogonalize_workspace(mats)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        with pytest.raises(A.AdamWError, match="capturing"):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                A.adamw_orthogonalize(A.F32, mats, ws)
        A.adamw_orthogonalize(A.F32, mats, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            A.adamw_orthogonalize(A.F32, mats, ws)
    for k in range(4):
        new = [gradient(r, c, gen) for r, c in a_in.shapes]
        for v, u in zip(a_in.views(), new):
            v.copy_(u.float())
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        replayed = [v.clone() for v in a_out.views()]
        eager, _ = run(new, "f32")
        assert all(torch.equal(x, y) for x, y in zip(replayed, eager)), k
        for v in a_out.views():
            v.zero_()


def test_shards_take_whole_matrices():
    """Two ranks, flat shard buffers on the padded index: together the whole list's result."""
    gen = torch.Generator().manual_seed(24)
    shapes = [(30, 50), (64, 21), (9, 11), (70, 70)]
    us = [gradient(r, c, gen) for r, c in shapes]
    whole, _ = run(us, "bf16")
    up8 = lambda n: -(-n // 8) * 8  # noqa: E731
    starts = [0]
    for r, c in shapes:
        starts.append(starts[-1] + up8(r * c))
    cut = starts[2]
    got = []
    for b, e in ((0, cut), (cut, starts[-1])):
        flat_in, flat_out = (torch.full((e - b,), 5.0, device="cuda").bfloat16() for _ in range(2))
        for u, s in zip(us, starts):
            if b <= s < e:
                flat_in[s - b:s - b + u.numel()] = u.flatten().cuda().bfloat16()
        mats = A.MatrixList(shapes, [[flat_out], [flat_in]], b, e, 0b11 | A.FLAT_PAD8)
        A.adamw_orthogonalize(A.BF16, mats, A.make_orthogonalize_workspace(mats))
        torch.cuda.synchronize()
        for u, s in zip(us, starts):
            if b <= s < e:
                got.append(flat_out[s - b:s - b + u.numel()].view(u.shape).clone())
                assert bool((flat_out[s - b + u.numel():s - b + up8(u.numel())] == 5.0).all())
    assert len(got) == len(whole)
    for x, y in zip(whole, got):
        assert far(x, y) <= 2 * TOL_NS + TOL_BF16
