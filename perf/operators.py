"""Cases of the gradient-norm and clipping operators, with their plain forms.

``run`` computes an operator in elementary torch operations (``own`` false), or
by the calls that a training program makes of this library (``own`` true), on
the state that ``prepare`` makes:

* ``grad_norm``     the global sum of squares and norm of a list's gradients, and whether one is inf or NaN
* ``tensor_norms``  the norm of every tensor of a list, and the list's sum of squares
* ``clip``          the gradients scaled in place to a largest global norm
* ``clipped_step``  an AdamW step that applies the clipping factor as it reads the gradients

A list's tensors lie one after another in one arena per stream, each start at a
multiple of ``align`` elements after ``phase`` elements, with zeros between
them, so a plain form may take a whole arena (or a shard's stretch of it) at once.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
PIECE = 1 << 26        # elements drawn, or taken to 64 bits, at once
CLIP_EPS = 1e-6        # what is added to the norm before the division
LR, BETA1, BETA2, EPS, DECAY = (float(np.float32(x)) for x in (2e-4, 0.9, 0.95, 1e-8, 0.1))
MAX_NORM = 1.0


# ---------------------------------------------------------------------------
# Tensor lists: (numel, whether it is a matrix) each
# ---------------------------------------------------------------------------

def _block(d, fused_qkv):
    """A transformer layer of width d: projections with their biases, a 4d feed-forward, two LayerNorms."""
    fan = [(d, 3 * d), (d, d)] if fused_qkv else [(d, d)] * 4
    sizes = []
    for a, b in fan + [(d, 4 * d), (4 * d, d)]:
        sizes += [(a * b, True), (b, False)]
    return sizes + [(d, False)] * 4


def _tensors(case):
    kind = case["list"]
    if kind == "flat":
        return [(case["n"], True)]
    if kind == "layers":
        d = case["width"]
        sizes = [(case["vocab"] * d, True), (case["positions"] * d, True)]
        for _ in range(case["layers"]):
            sizes += _block(d, case["fused_qkv"])
        return sizes + [(d, False)] * (2 if case["final_norm"] else 0)
    r = random.Random(case["sizes_seed"])      # log-uniform in [1, largest]
    top = math.log(case["largest"] + 1)
    return [(max(1, min(case["largest"], int(math.exp(r.uniform(0.0, top))))), True) for _ in range(case["count"])]


def _layout(case):
    """(numels, arena offsets, arena length, shard begin and end in the flat index, the shard's stretch of the arena)."""
    numels = [n for n, _ in _tensors(case)]
    offsets, pos = [], case["phase"]
    for n in numels:
        pos = case["phase"] + -(-(pos - case["phase"]) // case["align"]) * case["align"]
        offsets.append(pos)
        pos += n
    total = sum(numels)
    begin, end = case["rank"] * total // case["ranks"], (case["rank"] + 1) * total // case["ranks"]
    starts = np.concatenate([[0], np.cumsum(numels)])

    def place(x):
        i = int(np.searchsorted(starts, x, side="right")) - 1
        return offsets[i] + x - int(starts[i])

    return numels, offsets, pos, begin, end, (place(begin), place(end - 1) + 1)


def _case(name, op, dtype, list_, *, align=128, phase=0, rank=0, ranks=1, groups=1, scale=0.0, norm=2.0, mode="", **sizes):
    return {"name": name, "op": op, "dtype": dtype, "list": list_, "align": align, "phase": phase, "rank": rank,
            "ranks": ranks, "groups": groups, "scale": scale, "norm": norm, "mode": mode, **sizes}


OPT_125M = dict(width=768, layers=12, vocab=50272, positions=2050, fused_qkv=False, final_norm=True)
OPT_1_3B = dict(width=2048, layers=24, vocab=50272, positions=2050, fused_qkv=False, final_norm=False)
BERT_52M = dict(width=768, layers=4, vocab=30592, positions=512, fused_qkv=True, final_norm=False)


def listed():
    return [
        # a LoRA adapter's or a probing head's few gradients, a view that starts in the middle of a buffer
        _case("norm_small_odd", "grad_norm", "bf16", "flat", n=12289, phase=3),
        # one rank's share of a 4-way data-parallel job whose per-tensor gradients straddle its edges, loss-scaled fp16
        _case("norm_bert_shard", "grad_norm", "f16", "layers", rank=1, ranks=4, scale=65536.0, **BERT_52M),
        # a whole model in two parameter groups (matrices with weight decay, vectors without), one norm over both
        _case("norm_opt_1_3b_groups", "grad_norm", "bf16", "layers", groups=2, **OPT_1_3B),
        # ten thousand tensors of any length, packed tightly, loss-scaled fp16
        _case("norm_ragged_10k", "grad_norm", "f16", "ragged", count=10000, largest=1 << 22, sizes_seed=1, align=1,
              scale=65536.0),
        # every layer's gradient norm, as a training run logs it
        _case("norms_opt_125m", "tensor_norms", "bf16", "layers", **OPT_125M),
        # fp32 accumulated gradients of many small tensors
        _case("norms_ragged_f32", "tensor_norms", "f32", "ragged", count=2000, largest=1 << 20, sizes_seed=2, align=4),
        # the small adapter again, clipped in place at half its norm
        _case("clip_small_odd", "clip", "f16", "flat", n=12289, phase=5, scale=1024.0),
        # an fp32 gradient shard after its reduce-scatter
        _case("clip_bert_shard_f32", "clip", "f32", "flat", n=13059840, norm=3.0),
        # a whole model's gradients
        _case("clip_opt_1_3b", "clip", "bf16", "layers", norm=1.7, **OPT_1_3B),
        # a small model's step: one flat buffer of a million parameters
        _case("step_1m", "clipped_step", "bf16", "flat", n=1 << 20, mode="mixed"),
        # pure-bf16 training with Kahan compensation
        _case("step_opt_125m_kahan", "clipped_step", "bf16", "layers", mode="kahan", norm=5.0, **OPT_125M),
        # the mixed-precision step of a whole model
        _case("step_opt_1_3b", "clipped_step", "bf16", "layers", mode="mixed", norm=1.3, **OPT_1_3B),
    ]


def draw(rng):
    log = lambda lo, hi: int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))  # noqa: E731
    op = rng.choice(("grad_norm", "tensor_norms", "clip", "clipped_step"))
    step = op == "clipped_step"
    dtype = rng.choice(("bf16", "f16") if step else ("bf16", "f16", "f32"))
    mode = rng.choice(("mixed", "kahan") if dtype == "bf16" else ("mixed",)) if step else ""
    ranks = rng.choice((1, 1, 2, 4, 8))
    common = dict(align=rng.choice((1, 2, 8, 128)), phase=rng.choice((0, 0, 1, 3, 8)), ranks=ranks,
                  rank=rng.randrange(ranks), scale=2.0 ** rng.randrange(8, 17) if dtype == "f16" else 0.0,
                  norm=round(rng.uniform(1.2, 20.0), 3), mode=mode)
    if op == "tensor_norms":       # a list's norms are wanted whole
        common.update(ranks=1, rank=0)
    kind = rng.choice(("flat", "layers", "ragged"))
    if kind == "flat":
        return _case("", op, dtype, "flat", n=log(4096, 1 << 28), **common)
    if kind == "ragged":
        return _case("", op, dtype, "ragged", count=log(3, 4000), largest=log(500, 1 << 18),
                     sizes_seed=rng.randrange(1 << 30), **common)
    heads = rng.randrange(2, 25)
    return _case("", op, dtype, "layers", groups=rng.choice((1, 2)) if op == "grad_norm" else 1, width=64 * heads,
                 layers=rng.randrange(2, 17), vocab=log(1000, 32000), positions=rng.randrange(128, 2050),
                 fused_qkv=rng.random() < 0.5, final_norm=rng.random() < 0.5, **common)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _normal(n, std, dtype, gaps, gen):
    """An arena of n values drawn from N(0, std^2), zero in the gaps between tensors."""
    out = torch.empty(n, dtype=dtype, device="cuda")
    for a in range(0, n, PIECE):
        b = min(n, a + PIECE)
        out[a:b] = torch.randn(b - a, device="cuda", generator=gen).mul_(std)
    for a, b in gaps:
        out[a:b] = 0
    return out


def _sum_squares(x):
    return sum(x[a:a + PIECE].double().square().sum() for a in range(0, x.numel(), PIECE)).reshape(1)


def prepare(case, seed):
    numels, offsets, length, begin, end, stretch = _layout(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ends = [0] + [o + n for o, n in zip(offsets, numels)]
    gaps = [(a, b) for a, b in zip(ends, offsets) if b > a]
    dtype, op = TYPES[case["dtype"]], case["op"]
    std = case["norm"] / math.sqrt(sum(numels))                     # of the unscaled gradients
    s = {"case": case, "numels": numels, "offsets": offsets, "stretch": stretch,
         "g": _normal(length, std * (case["scale"] or 1.0), dtype, gaps, gen)}
    one = lambda t: torch.zeros(1, dtype=t, device="cuda")  # noqa: E731
    if op == "grad_norm":
        s.update(sumsq=one(torch.float64), norm=one(torch.float32), found=one(torch.int32))
    elif op == "tensor_norms":
        s.update(sumsq=one(torch.float64), norms=torch.zeros(len(numels), dtype=torch.float32, device="cuda"))
    else:
        s["sumsq"] = _sum_squares(s["g"])       # the global norm call's result, all-reduced over the ranks
    if case["scale"]:
        s["scale"] = torch.tensor([case["scale"], 0.0], device="cuda")   # {fp32 scale, int32 growth tracker}
    if op == "clipped_step":
        kahan = case["mode"] == "kahan"
        state = torch.bfloat16 if kahan else torch.float32
        w = _normal(length, 0.02, torch.bfloat16 if kahan else torch.float32, gaps, gen)
        s["p"] = w if kahan else w.to(dtype)
        s["aux"] = _normal(length, 1e-6, torch.bfloat16, gaps, gen) if kahan else w
        s["m"] = _normal(length, std, state, gaps, gen)
        s["v"] = _normal(length, std, torch.float32, gaps, gen).square_().to(state)
        s["step"] = torch.full((1,), 99, dtype=torch.int32, device="cuda")
    if own:
        s.update(_handles(case, s, begin, end))
    return s


def _handles(case, s, begin, end):
    """The tensor lists that a training program keeps from step to step."""
    import adamw_optimizer_step_apply_amd as A

    def tensor_list(which):
        views = [[x[s["offsets"][i]:s["offsets"][i] + s["numels"][i]] for i in which]
                 for x in (s.get("p"), s["g"], s.get("m"), s.get("v"), s.get("aux")) if x is not None]
        if len(views) == 1:
            views = [None, views[0]]
        return A.TensorList([s["numels"][i] for i in which], views, begin if case["ranks"] > 1 else 0,
                            end if case["ranks"] > 1 else -1)

    if case["groups"] == 1:
        return {"lists": [tensor_list(range(len(s["numels"])))]}
    matrix = [m for _, m in _tensors(case)]
    if case["ranks"] == 1:
        return {"lists": [tensor_list([i for i, m in enumerate(matrix) if m is group]) for group in (True, False)]}
    # the shard is one stretch of the whole list: each group's part of it is a stretch of the group
    starts, lists = np.concatenate([[0], np.cumsum(s["numels"])]), []
    for group in (True, False):
        which = [i for i, m in enumerate(matrix) if m is group]
        before = lambda x: sum(min(max(0, x - int(starts[i])), s["numels"][i]) for i in which)  # noqa: E731
        views = [s["g"][s["offsets"][i]:s["offsets"][i] + s["numels"][i]] for i in which]
        lists.append(A.TensorList([s["numels"][i] for i in which], [None, views], before(begin), before(end)))
    return {"lists": lists}


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    op = s["case"]["op"]
    if op == "grad_norm":
        return _plain_norm(s)
    if op == "tensor_norms":
        return _plain_norms(s)
    if op == "clip":
        return _plain_clip(s)
    return _plain_step(s)


def _run_own(s):
    import adamw_optimizer_step_apply_amd as A
    case, op = s["case"], s["case"]["op"]
    dt = {"bf16": A.BF16, "f16": A.F16, "f32": A.F32}[case["dtype"]]
    if op == "grad_norm":
        for k, grads in enumerate(s["lists"]):
            last = k == len(s["lists"]) - 1
            A.adamw_grad_norm(dt, grads, s["sumsq"], s["norm"] if last else None, s["found"] if last else None,
                              accumulate=k > 0)
        return {"sumsq": s["sumsq"], "norm": s["norm"], "found": s["found"]}
    if op == "tensor_norms":
        A.adamw_tensor_norms(dt, s["lists"][0], s["norms"], d_sumsq=s["sumsq"])
        return {"norms": s["norms"], "sumsq": s["sumsq"]}
    clip = A.GradClip(s["sumsq"], MAX_NORM, CLIP_EPS)
    if op == "clip":
        A.adamw_clip_grads(dt, s["lists"][0], clip, d_scale=s.get("scale"))
        return {"g": s["g"]}
    mode = A.PURE_KAHAN if case["mode"] == "kahan" else A.MIXED
    A.adamw_multi_tensor_step_clipped(mode, dt, s["lists"][0], A.HParams(LR, BETA1, BETA2, EPS, DECAY), clip, s["step"],
                                      d_scale=s.get("scale"))
    return _step_outputs(s)


def _step_outputs(s):
    out = {k: s[k] for k in ("p", "m", "v", "aux", "step")}
    if "scale" in s:
        out.update(scale=s["scale"][:1], tracker=s["scale"].view(torch.int32)[1:])
    return out


def _plain_norm(s):
    # 64 bits: the squares of a billion 16-bit values in 32 bits lose the small ones
    x = s["g"][s["stretch"][0]:s["stretch"][1]].double()
    sumsq = x.mul_(x).sum().reshape(1)
    return {"sumsq": sumsq, "norm": sumsq.sqrt().float(), "found": (~torch.isfinite(sumsq)).int()}


def _plain_norms(s):
    g = s["g"]
    sums = torch.stack([g[o:o + n].double().square_().sum() for o, n in zip(s["offsets"], s["numels"])])
    return {"norms": sums.sqrt().float(), "sumsq": sums.sum().reshape(1)}


def _plain_factor(s, inv):
    """The fp32 clipping factor and the fp32 multiplier of the gradients, unscaling included."""
    coef = MAX_NORM / (s["sumsq"].sqrt() * inv + CLIP_EPS)
    coef = torch.where(coef < 1.0, coef, torch.ones_like(coef))
    return coef.float(), (inv * coef).float()


def _plain_inverse(s):
    """1 / loss scale, rounded to fp32, as a 64-bit value."""
    return (1.0 / s["scale"][:1].double()).float().double() if "scale" in s else torch.ones_like(s["sumsq"])


def _plain_clip(s):
    g = s["g"][s["stretch"][0]:s["stretch"][1]]
    coef, _ = _plain_factor(s, _plain_inverse(s))
    g.copy_(g.float() * coef)
    return {"g": s["g"]}


def _plain_step(s):
    a, b = s["stretch"]
    p, m, v, aux = (s[k][a:b] for k in ("p", "m", "v", "aux"))
    _, mult = _plain_factor(s, _plain_inverse(s))
    g = s["g"][a:b].float() * mult
    t = (s["step"] + 1).double()
    step_size = (LR / (1.0 - torch.pow(torch.full_like(t, BETA1), t))).float()
    rbc2 = (1.0 / (1.0 - torch.pow(torch.full_like(t, BETA2), t))).float()
    kahan = s["case"]["mode"] == "kahan"
    m32 = m.float() if kahan else m
    v32 = v.float() if kahan else v
    m32.mul_(BETA1).add_(g * float(np.float32(1) - np.float32(BETA1)))
    v32.mul_(BETA2).add_((g * g).mul_(float(np.float32(1) - np.float32(BETA2))))
    u = m32 / (v32 * rbc2).sqrt_().add_(EPS)
    if kahan:
        m.copy_(m32)
        v.copy_(v32)
        old = p.float()
        inc = aux.float() + ((old * float(np.float32(LR * DECAY))).neg_() - u * step_size)
        p.copy_(old + inc)
        aux.copy_(inc - (p.float() - old))
    else:
        aux.mul_(float(np.float32(1.0 - LR * DECAY))).sub_(u * step_size)
        p.copy_(aux)
    s["step"] += 1
    if "scale" in s:
        s["scale"].view(torch.int32)[1:] += 1
    return _step_outputs(s)


# ---------------------------------------------------------------------------
# What a pass has to move and compute, and its value in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    numels, _, _, begin, end, _ = _layout(case)
    n, esz, op = end - begin, BYTES[case["dtype"]], case["op"]
    if op == "grad_norm":
        return {"bytes": n * esz + 16, "flops": 2 * n}
    if op == "tensor_norms":
        return {"bytes": n * esz + 4 * len(numels) + 8, "flops": 2 * n}
    if op == "clip":
        return {"bytes": 2 * n * esz + 8, "flops": n}
    # mixed: gradient, master and both moments in, those but the gradient and the param out; Kahan: five 2-byte
    # streams in, four out
    return {"bytes": n * (18 if case["mode"] == "kahan" else 28) + 16, "flops": 20 * n}


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    a, b = s["stretch"]
    op = case["op"]
    if op in ("grad_norm", "tensor_norms"):
        def total(x):
            parts = [x[k:k + PIECE].double() for k in range(0, x.numel(), PIECE)]
            return math.fsum(float(torch.dot(y, y)) for y in parts)
        if op == "grad_norm":
            ss = total(s["g"][a:b])
            return {"sumsq": np.array([ss]), "norm": np.array([math.sqrt(ss)]), "found": np.array([0], np.int32)}
        sums = [total(s["g"][o:o + n]) for o, n in zip(s["offsets"], s["numels"])]
        return {"norms": np.sqrt(np.array(sums)), "sumsq": np.array([math.fsum(sums)])}
    inv = 1.0 / (case["scale"] or 1.0)
    coef = min(1.0, MAX_NORM / (math.sqrt(float(s["sumsq"])) * inv + CLIP_EPS))
    if op == "clip":
        out = s["g"].double()
        out[a:b] *= coef
        return {"g": out}
    t = int(s["step"]) + 1
    p0, c0 = (s["p"], s["aux"]) if case["mode"] == "kahan" else (s["aux"], None)
    p, m, v = p0.double(), s["m"].double(), s["v"].double()
    for k in range(a, b, PIECE):
        e = min(b, k + PIECE)
        g = s["g"][k:e].double() * (inv * coef)
        m[k:e] = BETA1 * m[k:e] + (1.0 - BETA1) * g
        v[k:e] = BETA2 * v[k:e] + (1.0 - BETA2) * g * g
        mhat, vhat = m[k:e] / (1.0 - BETA1 ** t), v[k:e] / (1.0 - BETA2 ** t)
        p[k:e] -= LR * (mhat / (vhat.sqrt() + EPS) + DECAY * p[k:e])
        if c0 is not None:
            p[k:e] += c0[k:e].double()
    out = {"p": p, "m": m, "v": v, "aux": None if c0 is not None else p.clone(),
           "step": torch.full((1,), t, dtype=torch.int32, device="cuda")}
    if case["scale"]:
        out.update(scale=s["scale"][:1].double(), tracker=torch.ones(1, dtype=torch.int32, device="cuda"))
    return out
