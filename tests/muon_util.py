"""What the tests of the Newton-Schulz products and the Muon step share: the definition in 64 bits, the
library's roundings in 64 bits, and lists of matrices in arenas with guards between them."""
import math

import torch

import adamw_optimizer_step_apply_amd as A

NS = A.NewtonSchulz()
f32 = lambda x: float(torch.tensor(x, dtype=torch.float32))  # noqa: E731


def ns64(u, ns=NS):
    """The Newton-Schulz products of one matrix by their definition."""
    x = u.double()
    n = x.norm() + f32(ns.eps)
    x = x / n if n else x
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for _ in range(ns.steps):
        g = x @ x.T
        x = f32(ns.a) * x + (f32(ns.b) * g + f32(ns.c) * g @ g) @ x
    return x.T if tall else x


def ns_rounded(u, ns=NS):
    """The same with the roundings that the header documents (X as fp16 pairs, in the last step as one fp16, products of
    fp16 values, diagonals of the squares in full), every sum in 64 bits."""
    h = lambda x: x.to(torch.float16).double()  # noqa: E731
    x = u.double()
    x = x / (x.norm() + f32(ns.eps)) * 2.0 ** 14
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for k in range(ns.steps):
        hi = h(x)
        lo = h((x - hi) * 2048.0) / 2048.0 if k + 1 < ns.steps else torch.zeros_like(hi)
        g = hi @ hi.T * 2.0 ** -14
        gh = h(g)
        e = (g - gh).diagonal()
        sq = (gh @ gh + (e[:, None] + e[None, :]) * gh) * 2.0 ** -14
        p = (f32(ns.b) * (gh + torch.diag(e)) + f32(ns.c) * sq) * 2.0 ** -2
        ph = h(p)
        d, r = p.diagonal()[:, None] * 2.0 ** -12, (p - ph).diagonal()[:, None] * 2.0 ** -12
        x = (f32(ns.a) + r) * hi + ph @ hi * 2.0 ** -12 + (f32(ns.a) + d) * lo
    return (x.T if tall else x) * 2.0 ** -14


def far(x, y):
    """Relative distance of x from y in the Frobenius norm."""
    x, y = x.double(), y.double()
    return float((x - y).norm() / y.norm()) if y.norm() else float(x.norm())


def gradient(r, c, gen, kind="momentum"):
    """A matrix on the CPU: 'momentum' (some strong directions and noise), 'normal', or 'decay' (singular values 1/k)."""
    x = torch.randn(r, c, generator=gen, dtype=torch.float64)
    if kind == "momentum":
        k = max(1, min(r, c) // 16)
        x = 0.3 * x + torch.randn(r, k, generator=gen, dtype=torch.float64) @ torch.randn(
            k, c, generator=gen, dtype=torch.float64) / math.sqrt(k)
    elif kind == "decay":
        a, _, b = torch.linalg.svd(x, full_matrices=False)
        x = a * torch.arange(1, min(r, c) + 1, dtype=torch.float64) ** -1.0 @ b
    return x * 1e-3


class Arena:
    """One stream of a list: matrices in one buffer, `gap` guard elements before, between and behind them, the
    first at `phase` elements past a 16-byte edge."""

    def __init__(self, mats, dtype, gap=8, phase=0, guard=7.0):
        self.shapes, self.dtype, self.guard = [tuple(m.shape) for m in mats], dtype, guard
        per16 = 16 // torch.empty(0, dtype=dtype).element_size()
        self.at, pos = [], gap
        for m in mats:
            pos = -(-(pos - phase) // per16) * per16 + phase if gap else pos
            self.at.append(pos)
            pos += m.numel() + gap
        self.buf = torch.full((pos + gap,), guard, device="cuda").to(dtype)
        for m, v in zip(mats, self.views()):
            v.copy_(m.to(dtype) if dtype != torch.int16 else m)

    def views(self):
        return [self.buf[a:a + r * c].view(r, c) for a, (r, c) in zip(self.at, self.shapes)]

    def guards_kept(self):
        rest = torch.ones_like(self.buf, dtype=torch.bool)
        for a, (r, c) in zip(self.at, self.shapes):
            rest[a:a + r * c] = False
        return bool((self.buf[rest].float() == self.guard).all())
