"""adamw_muon_multi_tensor_step on the GPU.

Two kinds of check.  The orthogonalised update itself is read back exactly: a mixed step from master weights of zero
with lr 1 and no decay leaves w = -O, O the fp32 sums that the step uses, and is held against the definition in 64
bits (2^-8, see test_gpu_orthogonalize.py) and against the documented roundings in 64 bits, whose distance from the
definition it may pass by a quarter and 2^-13 (rounding an element the other way, where the fp32 sum differs, moves
it by as much as rounding it did).  Everything around O is one binary32 operation each: given that O, momentum, weights,
params, compensation and remainders of every mode are compared bit for bit with the formulas in torch on the CPU.
"""
import itertools

import numpy as np
import pytest
import torch

import adamw_optimizer_step_apply_amd as A
from muon_util import NS, Arena, f32, far, gradient, ns64, ns_rounded

pytestmark = pytest.mark.gpu
TOL_NS = 2.0 ** -8
LISTS = {
    "small": [(16, 48), (48, 16), (5, 7), (1, 1)],
    "odd": [(100, 37), (37, 100), (129, 65), (1, 77)],
    "aligned": [(64, 128), (256, 64), (200, 200)],
    "larger": [(520, 300), (300, 520)],
}


def state(shapes, p_dtype, m_dtype, seed, grad_scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    g = [(gradient(r, c, gen) * grad_scale).to(p_dtype) for r, c in shapes]
    m = [gradient(r, c, gen).to(m_dtype) for r, c in shapes]
    w = [(torch.randn(r, c, generator=gen, dtype=torch.float64) * 0.02).float() for r, c in shapes]
    return g, m, w


def hparams(**kw):
    return A.MuonHParams(**{**dict(lr=3e-3, weight_decay=0.1), **kw})


def momentum(g, m, hp, mult):
    """(m after the step before its rounding, u) of fp32 tensors, one operation a line."""
    beta, omb = f32(hp.momentum), float(np.float32(1) - np.float32(hp.momentum))
    og = (g.float() * mult) * omb
    m = m.float() * beta + og
    return m, (m * beta + og if hp.nesterov else m)


def scaling_of(hp, r, c):
    return {A.MUON_SCALE_NONE: 1.0, A.MUON_SCALE_SPECTRAL: max(1.0, r / c) ** 0.5,
            A.MUON_SCALE_RMS: 0.2 * max(r, c) ** 0.5}[hp.scaling]


def step(shapes, streams, mode, p_dtype, hp, gap=8, phase=0, counter=4, prec=None, clip=None, found=None, scale=None,
         stream=None, workspace=None):
    """One step on arenas of the CPU tensors `streams` (param, grad, exp_avg, aux or None); the arenas and the counter."""
    arenas = [None if x is None else Arena(x, x[0].dtype, gap, phase % (16 // x[0].element_size())) for x in streams]
    cut = lambda a: None if a is None else a.views()  # noqa: E731
    mats = A.MatrixList(shapes, [cut(arenas[0]), cut(arenas[1]), cut(arenas[2]), None, cut(arenas[3])])
    ws = A.make_orthogonalize_workspace(mats) if workspace is None else workspace
    d_step = torch.tensor([counter], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    A.adamw_muon_multi_tensor_step(mode, p_dtype, mats, hp, d_step, ws, d_found_inf=found, clip=clip, d_scale=scale,
                                   prec=prec, stream=stream)
    torch.cuda.synchronize()
    for a in arenas:
        assert a is None or a.guards_kept(), "elements outside the matrices were written"
    assert all(torch.equal(v.cpu().view(torch.int16), x.view(torch.int16)) for v, x in zip(arenas[1].views(), streams[1])), \
        "a gradient was written"
    return arenas, int(d_step)


def update_of(shapes, g, m, hp, p_code, **kw):
    """O of these gradients and momenta, as the step has it."""
    probe = A.MuonHParams(lr=1.0, momentum=hp.momentum, weight_decay=0.0, inv_loss_scale=hp.inv_loss_scale,
                          nesterov=hp.nesterov, scaling=A.MUON_SCALE_NONE, ns=hp.ns)
    zeros = [torch.zeros(s) for s in shapes]
    mode = A.MIXED
    arenas, _ = step(shapes, [[x.clone() for x in g], g, [x.float() for x in m], zeros], mode, p_code, probe, **kw)
    return [-v.cpu() for v in arenas[3].views()]


CODES = {torch.bfloat16: A.BF16, torch.float16: A.F16}


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("name", list(LISTS))
def test_update_against_the_definition(name, nesterov):
    shapes, hp = LISTS[name], hparams(nesterov=nesterov)
    g, m, _ = state(shapes, torch.bfloat16, torch.float32, 31)
    for o, gi, mi in zip(update_of(shapes, g, m, hp, A.BF16), g, m):
        u = momentum(gi, mi, hp, 1.0)[1]
        true, rounded = ns64(u), ns_rounded(u)
        assert far(o, true) <= TOL_NS
        assert far(o, true) <= 1.25 * far(rounded, true) + 2.0 ** -13, (tuple(u.shape), far(o, true), far(rounded, true))


@pytest.mark.parametrize("kind", ["normal", "decay"])
@pytest.mark.parametrize("shape", [(64, 64), (300, 300), (128, 900), (700, 260)])
def test_update_of_other_spectra(shape, kind):
    gen = torch.Generator().manual_seed(32)
    hp = hparams()
    g = [(gradient(*shape, gen, kind)).bfloat16()]
    m = [g[0].float() * 0.5]
    o = update_of([shape], g, m, hp, A.BF16)[0]
    u = momentum(g[0], m[0], hp, 1.0)[1]
    true, rounded = ns64(u), ns_rounded(u)
    assert far(o, true) <= min(TOL_NS, 1.25 * far(rounded, true) + 2.0 ** -13)


@pytest.mark.parametrize("name,gap,phase", [("small", 8, 0), ("odd", 3, 5), ("aligned", 8, 0), ("aligned", 1, 3), ("odd", 0, 0)])
@pytest.mark.parametrize("scaling", [A.MUON_SCALE_NONE, A.MUON_SCALE_SPECTRAL, A.MUON_SCALE_RMS])
@pytest.mark.parametrize("p_dtype", [torch.bfloat16, torch.float16])
def test_mixed(name, gap, phase, scaling, p_dtype):
    shapes, hp = LISTS[name], hparams(scaling=scaling)
    g, m, w = state(shapes, p_dtype, torch.float32, 33)
    p = [x.to(p_dtype) for x in w]
    o = update_of(shapes, g, m, hp, CODES[p_dtype])
    arenas, t = step(shapes, [p, g, m, w], A.MIXED, CODES[p_dtype], hp, gap, phase)
    assert t == 5
    decay = f32(1.0 - f32(hp.lr) * f32(hp.weight_decay))
    for i, (r, c) in enumerate(shapes):
        mm, _ = momentum(g[i], m[i], hp, 1.0)
        ww = w[i] * decay - o[i] * f32(f32(hp.lr) * scaling_of(hp, r, c))
        assert torch.equal(arenas[2].views()[i].cpu(), mm)
        assert torch.equal(arenas[3].views()[i].cpu(), ww)
        assert torch.equal(arenas[0].views()[i].cpu(), ww.to(p_dtype))


def bits(w):
    return w.contiguous().view(torch.int32)


@pytest.mark.parametrize("name,gap,phase", [("odd", 3, 5), ("aligned", 8, 0)])
def test_split_master(name, gap, phase):
    shapes, hp = LISTS[name], hparams(scaling=A.MUON_SCALE_SPECTRAL, nesterov=False)
    g, m, w = state(shapes, torch.bfloat16, torch.float32, 34)

    def split(x):
        b = bits(x)
        hi = (b >> 16) + ((b >> 15) & 1)
        return hi.short().view(torch.bfloat16), (b - (hi << 16)).short()
    o = update_of(shapes, g, m, hp, A.BF16)
    parts = [split(x) for x in w]
    arenas, _ = step(shapes, [[p for p, _ in parts], g, m, [r for _, r in parts]], A.MIXED_SPLIT, A.BF16, hp, gap, phase)
    decay = f32(1.0 - f32(hp.lr) * f32(hp.weight_decay))
    for i, (r, c) in enumerate(shapes):
        p, rest = split(w[i] * decay - o[i] * f32(f32(hp.lr) * scaling_of(hp, r, c)))
        assert torch.equal(arenas[0].views()[i].cpu().view(torch.int16), p.view(torch.int16))
        assert torch.equal(arenas[3].views()[i].cpu(), rest)


@pytest.mark.parametrize("name,gap,phase", [("odd", 3, 5), ("aligned", 8, 0), ("small", 1, 1)])
@pytest.mark.parametrize("m16,kahan", itertools.product([True, False], [A.KAHAN_NONE, A.KAHAN_BF16, A.KAHAN_F32]))
def test_pure(name, gap, phase, m16, kahan):
    shapes, hp = LISTS[name], hparams()
    m_dtype, c_dtype = torch.bfloat16 if m16 else torch.float32, torch.float32 if kahan == A.KAHAN_F32 else torch.bfloat16
    g, m, w = state(shapes, torch.bfloat16, m_dtype, 35)
    p, c = [x.bfloat16() for x in w], [(x * 1e-3).to(c_dtype) for x in w]
    o = update_of(shapes, g, m, hp, A.BF16)
    prec = A.PurePrecision(A.BF16 if m16 else A.F32, A.F32, kahan)
    arenas, _ = step(shapes, [p, g, m, c if kahan else None], A.MIXED, A.F16, hp, gap, phase, prec=prec)
    decay, lrwd = f32(1.0 - f32(hp.lr) * f32(hp.weight_decay)), f32(f32(hp.lr) * f32(hp.weight_decay))
    if m16 and kahan == A.KAHAN_BF16:      # the mode without a descriptor is this one
        plain, _ = step(shapes, [p, g, m, c], A.PURE_KAHAN, A.BF16, hp, gap, phase)
        assert all(torch.equal(x.buf, y.buf) for x, y in zip(plain, arenas) if x is not None)
    for i, (r, cc) in enumerate(shapes):
        inc = o[i] * f32(f32(hp.lr) * scaling_of(hp, r, cc))
        old = p[i].float()
        assert torch.equal(arenas[2].views()[i].cpu(), momentum(g[i], m[i], hp, 1.0)[0].to(m_dtype))
        if kahan == A.KAHAN_NONE:
            assert torch.equal(arenas[0].views()[i].cpu(), (old * decay - inc).bfloat16())
            continue
        s = c[i].float() + (-(old * lrwd) - inc)
        new = (old + s).bfloat16()
        assert torch.equal(arenas[0].views()[i].cpu(), new)
        assert torch.equal(arenas[3].views()[i].cpu(), (s - (new.float() - old)).to(c_dtype))


@pytest.mark.parametrize("use_scale", [True, False])
@pytest.mark.parametrize("use_clip", [True, False])
def test_loss_scale_and_clipping(use_scale, use_clip):
    shapes, scale = LISTS["aligned"], 1024.0
    hp = hparams(inv_loss_scale=1.0 if use_scale else 1.0 / scale)
    g, m, w = state(shapes, torch.float16, torch.float32, 36, grad_scale=scale)
    sumsq = torch.tensor([sum(float(x.double().square().sum()) for x in g)], dtype=torch.float64, device="cuda")
    d_scale = A.loss_scale_state(scale)
    clip = A.GradClip(sumsq, max_norm=0.01) if use_clip else None
    mult = f32(1.0 / scale)
    if use_clip:
        coef = f32(0.01) / (float(sumsq.sqrt()) * mult + f32(1e-6))
        assert coef < 1.0
        mult = f32(mult * coef)
    kw = dict(clip=clip, scale=d_scale if use_scale else None)
    o = update_of(shapes, g, m, hp, A.F16, **kw)
    arenas, t = step(shapes, [[x.half() for x in w], g, m, w], A.MIXED, A.F16, hp, **kw)
    assert t == 5 and float(d_scale[0]) == scale and int(d_scale.view(torch.int32)[1]) == 0
    decay = f32(1.0 - f32(hp.lr) * f32(hp.weight_decay))
    for i, (r, c) in enumerate(shapes):
        mm, u = momentum(g[i], m[i], hp, mult)
        assert torch.equal(arenas[2].views()[i].cpu(), mm)
        assert far(o[i], ns64(u)) <= TOL_NS
        ww = w[i] * decay - o[i] * f32(f32(hp.lr) * scaling_of(hp, r, c))
        assert torch.equal(arenas[3].views()[i].cpu(), ww)


@pytest.mark.parametrize("why", ["flag", "norm", "counter", "negative"])
def test_skipped_steps_write_nothing(why):
    shapes, hp = LISTS["odd"], hparams()
    g, m, w = state(shapes, torch.bfloat16, torch.float32, 37)
    if why == "norm":
        g[1][0, 0] = float("inf")
    found = torch.tensor([1 if why == "flag" else 0], dtype=torch.int32, device="cuda")
    sumsq = torch.tensor([float("inf") if why == "norm" else 1.0], dtype=torch.float64, device="cuda")
    counter = {"counter": 2 ** 31 - 1, "negative": -1}.get(why, 4)
    p = [x.bfloat16() for x in w]
    arenas, t = step(shapes, [p, g, m, w], A.MIXED, A.BF16, hp, counter=counter, found=found, clip=A.GradClip(sumsq))
    assert t == counter
    for a, x in zip(arenas, (p, g, m, w)):
        assert all(torch.equal(v.cpu().view(torch.uint8), y.view(torch.uint8)) for v, y in zip(a.views(), x))


def test_a_bad_gradient_spoils_its_own_matrix_only():
    shapes, hp = LISTS["odd"], hparams()
    g, m, w = state(shapes, torch.bfloat16, torch.float32, 38)
    good, _ = step(shapes, [[x.bfloat16() for x in w], g, m, w], A.MIXED, A.BF16, hp)
    bad = [x.clone() for x in g]
    bad[2][100, 3] = float("nan")
    arenas, _ = step(shapes, [[x.bfloat16() for x in w], bad, m, w], A.MIXED, A.BF16, hp)
    for i in range(len(shapes)):
        if i == 2:
            assert bool(torch.isnan(arenas[3].views()[i]).all())
        else:
            assert torch.equal(arenas[3].views()[i], good[3].views()[i])


def test_empty_list_advances_the_counter():
    d_step = torch.tensor([7], dtype=torch.int32, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    A.adamw_muon_multi_tensor_step(A.MIXED, A.BF16, A.MatrixList([], [[], [], [], None, []]), hparams(), d_step, ws)
    torch.cuda.synchronize()
    assert int(d_step) == 8


def test_captured_steps_replayed():
    """Three replays with new gradients, and eager steps of another list between them, against eager steps."""
    shapes, hp = LISTS["odd"], hparams()
    g, m, w = state(shapes, torch.bfloat16, torch.float32, 39)
    p = [x.bfloat16() for x in w]
    make = lambda: [Arena(x, x[0].dtype) for x in (p, g, m, w)]  # noqa: E731
    eager, cap = make(), make()
    lists = [A.MatrixList(shapes, [a[0].views(), a[1].views(), a[2].views(), None, a[3].views()]) for a in (eager, cap)]
    ws = [A.make_orthogonalize_workspace(x) for x in lists]
    steps = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        A.adamw_muon_multi_tensor_step(A.MIXED, A.BF16, lists[1], hp, steps[1], ws[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            A.adamw_muon_multi_tensor_step(A.MIXED, A.BF16, lists[1], hp, steps[1], ws[1])
    A.adamw_muon_multi_tensor_step(A.MIXED, A.BF16, lists[0], hp, steps[0], ws[0])
    torch.cuda.synchronize()
    gen = torch.Generator().manual_seed(40)
    for k in range(3):
        for v, x in zip(eager[1].views(), cap[1].views()):
            new = gradient(*v.shape, gen).bfloat16()
            v.copy_(new)
            x.copy_(new)
        torch.cuda.synchronize()
        graph.replay()
        A.adamw_muon_multi_tensor_step(A.MIXED, A.BF16, lists[0], hp, steps[0], ws[0])
        torch.cuda.synchronize()
        assert int(steps[0]) == int(steps[1]) == k + 2
        for x, y in zip(eager, cap):
            assert torch.equal(x.buf, y.buf), k


def test_workspace_of_one_matrix_at_a_time():
    shapes, hp = LISTS["larger"] + LISTS["odd"], hparams()
    g, m, w = state(shapes, torch.bfloat16, torch.float32, 41)
    p = [x.bfloat16() for x in w]
    whole, _ = step(shapes, [p, g, m, w], A.MIXED, A.BF16, hp)
    n = A.adamw_orthogonalize_workspace_bytes(A.MatrixList(shapes, [[]] * 5), least=True)
    parts, t = step(shapes, [p, g, m, w], A.MIXED, A.BF16, hp, workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))
    assert t == 5 and torch.equal(whole[2].buf, parts[2].buf)
    for i, (r, c) in enumerate(shapes):
        # the weights differ by two updates' errors at most
        most = 2 * TOL_NS * f32(hp.lr) * scaling_of(hp, r, c) * min(r, c) ** 0.5 * 1.14
        assert float((whole[3].views()[i] - parts[3].views()[i]).norm()) <= most + 1e-6 * float(w[i].norm())


def test_a_training_iteration():
    """As a program uses them: one global norm over matrices and vectors, a Muon step of the matrices and an AdamW step
    of the vectors, both clipped by it, under one loss scale that the last call advances."""
    shapes, vectors, scale = LISTS["aligned"], [64, 1000, 7], 512.0
    hp, ahp = hparams(), A.HParams()
    g, m, w = state(shapes, torch.float16, torch.float32, 42, grad_scale=scale)
    gen = torch.Generator().manual_seed(43)
    vg = [(torch.randn(n, generator=gen) * 1e-3 * scale).half() for n in vectors]
    arenas = [Arena(x, x[0].dtype) for x in ([x.half() for x in w], g, m, w)]
    mats = A.MatrixList(shapes, [arenas[0].views(), arenas[1].views(), arenas[2].views(), None, arenas[3].views()])
    vec = [[x.cuda() for x in vg]] + [[torch.zeros(n, device="cuda") for n in vectors] for _ in range(3)]
    vp = [torch.zeros(n, dtype=torch.float16, device="cuda") for n in vectors]
    tl = A.TensorList(vectors, [vp, *vec])
    sumsq, d_scale = torch.zeros(1, dtype=torch.float64, device="cuda"), A.loss_scale_state(scale)
    steps = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2)]
    ws = A.make_orthogonalize_workspace(mats)
    A.adamw_grad_norm(A.F16, mats, sumsq)
    A.adamw_grad_norm(A.F16, tl, sumsq, accumulate=True)
    clip = A.GradClip(sumsq, max_norm=0.05)
    A.adamw_muon_multi_tensor_step(A.MIXED, A.F16, mats, hp, steps[0], ws, clip=clip, d_scale=d_scale)
    A.adamw_multi_tensor_step_clipped(A.MIXED, A.F16, tl, ahp, clip, steps[1], d_scale=d_scale, scaler=A.LossScaler())
    torch.cuda.synchronize()
    total = sum(float(x.double().square().sum()) for x in g + vg)
    assert abs(float(sumsq) - total) <= 1e-12 * total
    assert int(steps[0]) == int(steps[1]) == 1 and int(d_scale.view(torch.int32)[1]) == 1
    coef = min(1.0, 0.05 / (total ** 0.5 / scale + 1e-6))
    assert coef < 1.0
    for i, (r, c) in enumerate(shapes):
        gg = g[i].double() / scale * coef
        mm = f32(hp.momentum) * m[i].double() + (1 - f32(hp.momentum)) * gg
        o = ns64(f32(hp.momentum) * mm + (1 - f32(hp.momentum)) * gg)
        ww = w[i].double() * (1 - f32(hp.lr) * f32(hp.weight_decay)) - f32(hp.lr) * scaling_of(hp, r, c) * o
        got = arenas[3].views()[i].cpu().double()
        assert float((got - ww).norm()) <= TOL_NS * f32(hp.lr) * scaling_of(hp, r, c) * float(o.norm()) + 1e-6 * float(w[i].norm())
    for x, y in zip(vec[3], vg):     # the AdamW step's first update has the sign of the gradient
        assert bool((torch.sign(x.cpu()) == -torch.sign(y.float())).all())
