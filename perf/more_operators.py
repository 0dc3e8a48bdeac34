"""Cases of the orthogonalised updates, with their plain forms.

``run`` computes an operator in elementary torch operations (``own`` false), or
by the calls that a training program makes of this library (``own`` true), on
the state that ``prepare`` makes:

* ``ortho``  every matrix of a list orthogonalised by Newton-Schulz products: from X = U / (|U| + eps), five
             times X <- a X + b (X X^T) X + c (X X^T)^2 X, rounded to bf16
* ``step``   the whole Muon step of a list of matrices: momentum, Newton-Schulz products of it, decoupled weight
             decay and the update of the weights, in the precisions of the AdamW step

A list's matrices lie one after another in one arena per stream, each start at a
multiple of ``align`` elements, with zeros between them; neighbours of one shape
form a group, which a plain form takes as one batch.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
NS = (3.4445, -4.7750, 2.0315)         # a, b, c, in 32 bits as the library has them
NS_A, NS_B, NS_C = (float(np.float32(x)) for x in NS)
NS_STEPS, NS_EPS = 5, float(np.float32(1e-7))
LR, MOMENTUM, DECAY = (float(np.float32(x)) for x in (2e-4, 0.95, 0.1))
OMB = float(np.float32(1) - np.float32(MOMENTUM))
MAX_NORM, CLIP_EPS = 1.0, 1e-6
PIECE = 1 << 26                        # elements taken to 64 bits at once


# ---------------------------------------------------------------------------
# Matrix lists: (matrices, rows, columns) of each group
# ---------------------------------------------------------------------------

def _groups(case):
    kind = case["list"]
    if kind == "same":                 # one matrix, or the experts of a layer
        return [(case["count"], case["rows"], case["cols"])]
    if kind == "adapters":             # the two factors of a low-rank adapter on every layer
        return [(case["count"], case["rank"], case["width"]), (case["count"], case["width"], case["rank"])]
    if kind == "layers":               # a transformer's matrices; each projection a matrix of its own, or fused
        d, n = case["width"], case["layers"]
        fan = [(n, 3 * d, d), (n, d, d)] if case["fused_qkv"] else [(4 * n, d, d)]
        return fan + ([(n, case["ffn"], d), (n, d, case["ffn"])] if case["ffn"] else [])
    r = random.Random(case["sizes_seed"])          # both sides log-uniform in [1, largest]
    side = lambda: max(1, min(case["largest"], int(math.exp(r.uniform(0.0, math.log(case["largest"] + 1))))))  # noqa: E731
    return [(1, side(), side()) for _ in range(case["count"])]


def _layout(case):
    """(groups as (first element, elements between matrices, matrices, rows, columns), arena length)."""
    groups, pos = [], 0
    for n, r, c in _groups(case):
        apart = -(-(r * c) // case["align"]) * case["align"]
        groups.append((pos, apart, n, r, c))
        pos += n * apart
    return groups, pos


def _case(name, op, dtype, list_, *, align=128, mode="", scaling="", nesterov=True, scale=0.0, clip=False, **sizes):
    return {"name": name, "op": op, "dtype": dtype, "list": list_, "align": align, "mode": mode, "scaling": scaling,
            "nesterov": nesterov, "scale": scale, "clip": clip, **sizes}


OPT_1_3B = dict(width=2048, ffn=8192, fused_qkv=False)
BERT_ATTENTION = dict(width=768, ffn=0, fused_qkv=True, layers=4)


def listed():
    return [
        # one factor of a low-rank adapter: a call that is all latency
        _case("ortho_adapter", "ortho", "bf16", "same", count=1, rows=16, cols=768),
        # the adapters of a whole model, from fp32 momentum
        _case("ortho_adapters_2048", "ortho", "f32", "adapters", count=24, rank=16, width=2048),
        # one projection alone, from fp32 momentum: too few products to fill the card
        _case("ortho_one_768", "ortho", "f32", "same", count=1, rows=768, cols=768),
        # matrices of any shape, odd sides, vectors among them, packed tightly
        _case("ortho_ragged_odd", "ortho", "f16", "ragged", align=1, count=60, largest=1500, sizes_seed=3),
        # the attention matrices of a BERT, its three input projections as one tall matrix
        _case("ortho_bert_attention", "ortho", "bf16", "layers", **BERT_ATTENTION),
        # one transformer layer
        _case("ortho_opt_1_3b_layer", "ortho", "bf16", "layers", layers=1, **OPT_1_3B),
        # a small model's one matrix
        _case("step_one_512", "step", "bf16", "same", mode="mixed", scaling="rms", count=1, rows=512, cols=512),
        # a layer's experts in pure bf16 with compensation, each orthogonalised by itself
        _case("step_experts_kahan", "step", "bf16", "same", mode="kahan", scaling="rms", count=64, rows=512, cols=1024),
        # fp16 gradients under a loss scale, clipped by the model's norm
        _case("step_bert_f16_clipped", "step", "f16", "layers", mode="mixed", scaling="spectral", scale=65536.0, clip=True,
              **BERT_ATTENTION),
        # odd shapes with the split master, momentum without its look ahead
        _case("step_ragged_split", "step", "bf16", "ragged", mode="split", scaling="none", nesterov=False, align=1,
              count=40, largest=1200, sizes_seed=4),
        # one of four ranks' share of a model whose matrices are dealt out whole
        _case("step_opt_1_3b_rank", "step", "bf16", "layers", mode="mixed", scaling="rms", layers=6, **OPT_1_3B),
        # every matrix of a whole model
        _case("step_opt_1_3b", "step", "bf16", "layers", mode="mixed", scaling="rms", layers=24, **OPT_1_3B),
    ]


def draw(rng):
    log = lambda lo, hi: int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))  # noqa: E731
    while True:
        op = rng.choice(("ortho", "step"))
        if op == "ortho":
            common = dict(dtype=rng.choice(("bf16", "f16", "f32")))
        else:
            mode = rng.choice(("mixed", "mixed", "kahan", "split"))
            dtype = rng.choice(("bf16", "f16")) if mode == "mixed" else "bf16"
            common = dict(dtype=dtype, mode=mode, scaling=rng.choice(("none", "spectral", "rms")),
                          nesterov=rng.random() < 0.7, clip=rng.random() < 0.4,
                          scale=2.0 ** rng.randrange(8, 17) if dtype == "f16" else 0.0)
        common["align"] = rng.choice((1, 2, 8, 128))
        kind = rng.choice(("same", "adapters", "layers", "ragged"))
        if kind == "same":
            sizes = dict(count=log(1, 100), rows=log(1, 4096), cols=log(1, 4096))
        elif kind == "adapters":
            sizes = dict(count=log(1, 100), rank=log(4, 128), width=log(64, 8192))
        elif kind == "layers":
            d = 64 * rng.randrange(2, 40)
            sizes = dict(width=d, ffn=rng.choice((0, 4 * d)), fused_qkv=rng.random() < 0.5, layers=log(1, 16))
        else:
            sizes = dict(count=log(1, 100), largest=log(8, 2048), sizes_seed=rng.randrange(1 << 30))
        case = _case("", op, common.pop("dtype"), kind, **common, **sizes)
        if work(case)["flops"] < 1e13 and _layout(case)[1] < 4e8:
            return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _views(arena, groups):
    """Each group of the arena as one tensor (matrices, rows, columns)."""
    return [arena[o:].as_strided((n, r, c), (apart, c, 1), arena.storage_offset() + o) for o, apart, n, r, c in groups]


def _gradients(length, groups, std, gen):
    """An fp32 arena of matrices as gradients and momenta are: a few strong directions, and noise in all the others."""
    out = torch.zeros(length, device="cuda")
    for x in _views(out, groups):
        n, r, c = x.shape
        k = max(1, min(r, c) // 16)
        x.copy_(torch.randn(n, r, c, device="cuda", generator=gen).mul_(0.3 * std))
        left, right = (torch.randn(n, *s, device="cuda", generator=gen) for s in ((r, k), (k, c)))
        x.add_(torch.matmul(left, right), alpha=std / math.sqrt(k))
    return out


def _weights(length, groups, std, gen):
    out = torch.zeros(length, device="cuda")
    for x in _views(out, groups):
        x.copy_(torch.randn(x.shape, device="cuda", generator=gen).mul_(std))
    return out


def prepare(case, seed):
    groups, length = _layout(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = TYPES[case["dtype"]]
    s = {"case": case, "groups": groups}
    if case["op"] == "ortho":
        s["u"] = _gradients(length, groups, 1e-3, gen).to(dtype)
        s["o"] = torch.zeros(length, dtype=torch.bfloat16, device="cuda")
    else:
        g = _gradients(length, groups, 1e-4, gen).mul_(case["scale"] or 1.0)
        s["g"] = g.to(dtype)
        if case["clip"]:               # the sum over the whole model, of which these matrices are a part
            s["sumsq"] = 1.25 * sum(s["g"][a:a + PIECE].double().square().sum() for a in range(0, length, PIECE)).reshape(1)
        if case["scale"]:
            s["scale"] = torch.tensor([case["scale"], 0.0], device="cuda")   # {fp32 scale, int32 growth tracker}
        del g
        m, w = _gradients(length, groups, 1e-4, gen), _weights(length, groups, 0.02, gen)
        if case["mode"] == "mixed":
            s.update(p=w.to(dtype), m=m, aux=w)
        elif case["mode"] == "split":
            p, rest = _split(w)
            s.update(p=p, m=m, aux=rest)
        else:
            aux = _weights(length, groups, 1e-6, gen)
            s.update(p=w.to(dtype), m=m.to(dtype), aux=aux.to(dtype))
        s["step"] = torch.full((1,), 99, dtype=torch.int32, device="cuda")
    if own:
        s.update(_handles(case, s))
    return s


def _handles(case, s):
    """The list and the workspace that a training program keeps from step to step."""
    import adamw_optimizer_step_apply_amd as A
    at = [(o + i * apart, r, c) for o, apart, n, r, c in s["groups"] for i in range(n)]
    cut = lambda x: [x[o:o + r * c] for o, r, c in at]  # noqa: E731
    if case["op"] == "ortho":
        mats = A.MatrixList([(r, c) for _, r, c in at], [cut(s["o"]), cut(s["u"])])
    else:
        mats = A.MatrixList([(r, c) for _, r, c in at], [cut(s["p"]), cut(s["g"]), cut(s["m"]), None, cut(s["aux"])])
    return {"mats": mats, "ws": A.make_orthogonalize_workspace(mats)}


def _join(p, rest):
    """The fp32 master of the split mode: its bits are (p << 16) + rest."""
    return ((p.view(torch.int16).int() << 16) + rest.int()).view(torch.float32)


def _split(w):
    bits = w.view(torch.int32)
    high = (bits >> 16) + ((bits >> 15) & 1)
    return high.short().view(torch.bfloat16), (bits - (high << 16)).short()


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    case = s["case"]
    if own:
        _run_own(case, s)
    elif case["op"] == "ortho":
        for u, o in zip(_views(s["u"], s["groups"]), _views(s["o"], s["groups"])):
            o.copy_(_newton_schulz(u.float()))
    else:
        _plain_step(case, s)
    if case["op"] == "ortho":
        return {"o": s["o"]}
    # The weights as the fp32 values that they stand for: a param with its compensation, or with its remainder, is
    # the sum of the two, and which of the two holds a last bit turns on the last bit of the sum.
    w = {"mixed": lambda: s["aux"], "split": lambda: _join(s["p"], s["aux"]),
         "kahan": lambda: s["p"].float() + s["aux"].float()}[case["mode"]]()
    return {"p": s["p"], "m": s["m"], "w": w, "step": s["step"]}


def _run_own(case, s):
    import adamw_optimizer_step_apply_amd as A
    dtypes = {"bf16": A.BF16, "f16": A.F16, "f32": A.F32}
    ns = A.NewtonSchulz(*NS, steps=NS_STEPS, eps=NS_EPS)
    if case["op"] == "ortho":
        A.adamw_orthogonalize(dtypes[case["dtype"]], s["mats"], s["ws"], ns)
        return
    mode = {"mixed": A.MIXED, "split": A.MIXED_SPLIT, "kahan": A.PURE_KAHAN}[case["mode"]]
    scaling = {"none": A.MUON_SCALE_NONE, "spectral": A.MUON_SCALE_SPECTRAL, "rms": A.MUON_SCALE_RMS}[case["scaling"]]
    hp = A.MuonHParams(lr=LR, momentum=MOMENTUM, weight_decay=DECAY, nesterov=case["nesterov"], scaling=scaling, ns=ns)
    A.adamw_muon_multi_tensor_step(mode, dtypes[case["dtype"]], s["mats"], hp, s["step"], s["ws"],
                                   clip=A.GradClip(s["sumsq"], MAX_NORM, CLIP_EPS) if case["clip"] else None,
                                   d_scale=s.get("scale"))


def _newton_schulz(u):
    """A batch of matrices in fp32, worked through on their shorter side."""
    x = u / (u.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    for _ in range(NS_STEPS):
        gram = torch.matmul(x, x.transpose(1, 2))
        x = NS_A * x + torch.matmul(NS_B * gram + NS_C * torch.matmul(gram, gram), x)
    return x.transpose(1, 2) if tall else x


def _scaling(case, r, c):
    return {"none": 1.0, "spectral": math.sqrt(max(1.0, r / c)), "rms": 0.2 * math.sqrt(max(r, c))}[case["scaling"]]


def _plain_step(case, s):
    g = s["g"].float()
    inv = (1.0 / s["scale"][:1].double()).float() if case["scale"] else torch.ones(1, device="cuda")
    if case["clip"]:
        coef = MAX_NORM / (s["sumsq"].sqrt() * inv.double() + CLIP_EPS)
        inv = (inv.double() * torch.where(coef < 1.0, coef, torch.ones_like(coef))).float()
    g.mul_(inv).mul_(OMB)
    m = s["m"].float().mul_(MOMENTUM).add_(g)
    u = m * MOMENTUM + g if case["nesterov"] else m.clone()
    s["m"].copy_(m)
    for x in _views(u, s["groups"]):
        x.copy_(_newton_schulz(x) * float(np.float32(LR * _scaling(case, *x.shape[1:]))))
    decay, lrwd = float(np.float32(1.0 - LR * DECAY)), float(np.float32(LR * DECAY))
    if case["mode"] == "mixed":
        s["aux"].mul_(decay).sub_(u)
        s["p"].copy_(s["aux"])
    elif case["mode"] == "split":
        p, rest = _split(_join(s["p"], s["aux"]).mul_(decay).sub_(u))
        s["p"].copy_(p)
        s["aux"].copy_(rest)
    else:
        old = s["p"].float()
        inc = s["aux"].float() + (-(old * lrwd) - u)
        s["p"].copy_(old + inc)
        s["aux"].copy_(inc - (s["p"].float() - old))
    s["step"] += 1


# ---------------------------------------------------------------------------
# What a pass has to move and compute, and its value in 64 bits
# ---------------------------------------------------------------------------

def _flops(r, c):
    """Products that the definition leaves no way round, a symmetric one counted once for each pair of elements: each
    step's Gram matrix, its square and the product with X; or, from one Gram matrix, polynomials of it (all
    symmetric: its square, the polynomial times it twice, and times the product so far), and one product with X."""
    s, l = min(r, c), max(r, c)
    by_steps = NS_STEPS * (s * s * l + s ** 3 + 2 * s * s * l)
    by_gram = s * s * l + (4 * NS_STEPS - 3) * s ** 3 + 2 * s * s * l
    return min(by_steps, by_gram)


def work(case):
    n = sum(k * r * c for k, r, c in _groups(case))
    flops = sum(k * _flops(r, c) for k, r, c in _groups(case))
    if case["op"] == "ortho":
        return {"bytes": n * (BYTES[case["dtype"]] + 2), "flops": flops}
    # mixed: gradient, momentum and master in, the last two and the param out; split: param and remainder in the
    # master's place; Kahan: four 2-byte streams in, three out
    per = {"mixed": 20, "split": 18, "kahan": 14}[case["mode"]]
    return {"bytes": n * per + 8, "flops": flops + 12 * n}


def _exact_newton_schulz(u):
    """One matrix: polynomials of its Gram matrix on the shorter side, and one product at the end."""
    x = u / (torch.dot(u.flatten(), u.flatten()).sqrt() + NS_EPS)
    gram = x @ x.T if x.shape[0] <= x.shape[1] else x.T @ x
    q = eye = torch.eye(gram.shape[0], dtype=torch.float64, device=u.device)
    for _ in range(NS_STEPS):
        p = NS_A * eye + gram @ (NS_B * eye + NS_C * gram)
        q, gram = p @ q, p @ gram @ p
    return q @ x if x.shape[0] <= x.shape[1] else x @ q


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    if case["op"] == "ortho":
        out = torch.zeros(s["u"].numel(), dtype=torch.float64, device="cuda")
        for x, y in zip(_views(s["u"], s["groups"]), _views(out, s["groups"])):
            for i in range(x.shape[0]):
                y[i] = _exact_newton_schulz(x[i].double())
        return {"o": out}
    f = 1.0 / (case["scale"] or 1.0)
    if case["clip"]:
        f *= min(1.0, MAX_NORM / (math.sqrt(float(s["sumsq"])) * f + CLIP_EPS))
    m = s["m"].double().mul_(MOMENTUM)
    w = {"mixed": lambda: s["aux"].double(), "split": lambda: _join(s["p"], s["aux"]).double(),
         "kahan": lambda: s["p"].double()}[case["mode"]]().mul_(1.0 - LR * DECAY)
    if case["mode"] == "kahan":
        w += s["aux"].double()
    for gs, ms, ws in zip(*(_views(x, s["groups"]) for x in (s["g"], m, w))):
        for i in range(gs.shape[0]):
            g = gs[i].double() * (f * (1.0 - MOMENTUM))
            ms[i] += g
            u = MOMENTUM * ms[i] + g if case["nesterov"] else ms[i]
            ws[i] -= LR * _scaling(case, *u.shape) * _exact_newton_schulz(u)
    return {"p": w, "m": m, "w": w, "step": torch.full((1,), 100, dtype=torch.int32, device="cuda")}
