"""Softmax cross entropy over a product and its gradients in 64 bits, with bounds
of the fp32 kernels' error, for the tests: torch's double operations."""
from __future__ import annotations

import math

import torch

IGNORE = -100
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


class Problem:
    """Operands of a product with a vocabulary, on the device they are made on."""

    def __init__(self, M, N, K, *, rowwise=True, a=E4M3, b=E4M3, bias=None, seed=0, spread=2.0, ignored=0.2,
                 device="cuda"):
        g = torch.Generator().manual_seed(1000 * seed + M + 3 * N + 7 * K)

        def randn(*shape):
            return torch.randn(*shape, generator=g)
        self.M, self.N, self.K, self.mode = M, N, K, int(rowwise)
        # codes of any size up to the type's largest, logits of standard deviation `spread`
        big = {E4M3: 60.0, E5M2: 3000.0}
        self.A = (randn(M, K) * big[a]).to(a).to(device)
        self.Bt = (randn(N, K) * big[b]).to(b).to(device)
        self.B = self.Bt.t()
        unit = spread / math.sqrt(K)
        if rowwise:
            self.sa = (torch.exp(0.5 * randn(M)) / big[a]).to(device)
            self.sb = (torch.exp(0.5 * randn(N)) * unit / big[b]).to(device)
        else:
            self.sa = torch.tensor([0.7 / big[a]]).to(device)
            self.sb = torch.tensor([1.3 * unit / big[b]]).to(device)
        self.bias = None if bias is None else (randn(N) * 0.5).to(bias).to(device)
        self.target = torch.randint(0, N, (M,), generator=g)
        self.target[torch.rand(M, generator=g) < ignored] = IGNORE
        self.target = self.target.to(device)
        self.dloss = torch.rand(M, generator=g).add_(0.1).div_(max(M, 1)).to(device)

    @property
    def operands(self):
        return self.A, self.B, self.sa, self.sb, self.mode

    def logits(self):
        """(z, bound of the fp32 kernel's error in z)."""
        a, b = self.A.double(), self.Bt.double()
        s = self.sa.double()[:, None] * self.sb.double()[None, :] if self.mode else self.sa.double() * self.sb.double()
        z = (a @ b.t()) * s
        # the sum: 2^-20 of its terms' magnitudes, as for every product; the product of the scales and the two operations
        # on the sum: one rounding each, 2^-24 of what they give
        err = 2.0 ** -20 * (a.abs() @ b.t().abs()) * s.abs() + 2.0 ** -23 * z.abs()
        if self.bias is not None:
            z = z + self.bias.double()
            err = err + torch.where(z.isfinite(), 2.0 ** -24 * z.abs(), 0.0)
        return z, err


def live(target, ignore=IGNORE):
    return target != ignore


def loss64(p: Problem, ignore=IGNORE):
    """(loss, lse, bound of loss, bound of lse) of rows with valid targets."""
    z, err = p.logits()
    lse = torch.logsumexp(z, dim=1)
    top = z.amax(dim=1)
    rest = lse - top
    # lse moves by at most the largest error of a z that counts. A term of the sum: the argument (z - top) log2(e) is
    # rounded twice, which changes exp by 2^-23 |z - top|, weighted by exp(z - top) at most 2^-23 / e; ex2 2^-22.
    # The sum itself: chains of 8 + 4 + ceil(N / 4096) + 32 joins, each join two products and a sum of positive terms
    # with two more ex2: 46 x 2^-24 of additions, at most (4 + N / 4096 + 32) x (2^-22 + 2 x 2^-24) of joins
    joins = 4 + p.N / 4096 + 32
    rel = 2.0 ** -22 + 2.0 ** -23 + (12 + joins) * 2.0 ** -24 + joins * (2.0 ** -22 + 2.0 ** -23 + 2.0 ** -23)
    # log: 2^-22 of its value at most; the last sum one rounding. The maximum that terms are relative to is one of the
    # z, `above` = 4 at most under the largest: a term grows with it as the sum does (rel stays), the log's value is
    # up to 4 larger and the maximum 4 smaller, which adds 4 x 2^-22 and, in the sums with them, 2 x 4 x 2^-24
    above = 4.0
    lse_tol = (err.masked_fill(z == -math.inf, 0).amax(dim=1) + rel + 2.0 ** -22 * (rest.abs() + above) + above * 2.0 ** -23
               + 2.0 ** -23 * lse.abs())
    at = torch.where(live(p.target, ignore), p.target, 0)[:, None]
    zt = z.gather(1, at)[:, 0]
    loss = torch.where(live(p.target, ignore), lse - zt, 0.0)
    loss_tol = lse_tol + err.gather(1, at)[:, 0] + 2.0 ** -23 * ((top - zt).abs() + loss.abs())
    return loss, lse, torch.where(live(p.target, ignore), loss_tol, 0.0), lse_tol


# The kernels keep dz as fp16, times the mantissas of the two scales (together in [1, 4)) and 2^12 / (a power of two at or
# below the largest |dloss|), and codes times their scales' powers of two and this / (the largest of these powers), which
# is exact down to fp16's smallest step.
CODE_SCALE = {E4M3: 2.0 ** 7, E5M2: 1.0}


def _pow2(x):
    return 2.0 ** math.floor(math.log2(float(x)))


def _half_tol(x, unit):
    """Bound of x's rounding to fp16 when kept as x / unit: 2^-11 of it (half a step of its 11 bits is 2^-12 to 2^-11), or
    half of 2^-24 units. Before it, five products in fp32: 5 x 2^-24."""
    return x.abs() * (2.0 ** -11 + 5 * 2.0 ** -24) + 2.0 ** -25 * unit


def grad64(p: Problem, lse, dloss=None, ignore=IGNORE):
    """((da, db, dbias), bounds of their errors before the output's rounding) for a given lse."""
    dloss = p.dloss if dloss is None else dloss
    z, err = p.logits()
    a = p.A.double() * (p.sa.double()[:, None] if p.mode else p.sa.double())
    w = p.Bt.double() * (p.sb.double()[:, None] if p.mode else p.sb.double())
    on = live(p.target, ignore)
    g = torch.where(on, dloss.double().expand(p.M), 0.0)
    d = z - lse.double()[:, None]
    prob = torch.where(on[:, None], d.exp(), 0.0)
    hot = torch.zeros_like(prob)
    hot[on, p.target[on]] = 1.0
    dz = torch.where(on[:, None], (prob - hot) * g[:, None], 0.0)
    # exp: the error of z, the argument's two roundings, ex2; the product with g; the difference with g at the target
    rel = err.masked_fill(z == -math.inf, 0) + 2.0 ** -23 * torch.where(d.isfinite(), d.abs(), 0.0) + 2.0 ** -22 + 2.0 ** -22
    dz_tol = torch.where(on[:, None], prob * g.abs()[:, None] * rel + hot * g.abs()[:, None] * 2.0 ** -23, 0.0)
    # (ex2 flushes what is under 2^-126)
    dz_tol = dz_tol + 2.0 ** -126 * g.abs()[:, None]
    g_most = dloss.abs().expand(p.M)[on].max() if bool(on.any()) else torch.tensor(2.0 ** -100)
    g_unit = max(_pow2(g_most) if float(g_most) > 0 else 0.0, 2.0 ** -100) / 2.0 ** 12
    a_unit = _pow2(p.sa.abs().max()) / CODE_SCALE[p.A.dtype]
    w_unit = _pow2(p.sb.abs().max()) / CODE_SCALE[p.Bt.dtype]
    half = dz_tol + _half_tol(dz.abs() + dz_tol, g_unit)

    def product(left, left_tol, right, right_tol, terms):
        """left @ right with a bound: operands off by their bounds, sums of 16 products at a time in fp32, joined in up
        to 76 parts, pieces and slices of each 2^-23 of the magnitudes, and four roundings of scales."""
        both = (left.abs() + left_tol) @ (right.abs() + right_tol)
        return left @ right, both - left.abs() @ right.abs() + ((terms / 16 + 80) * 2.0 ** -23) * both
    # (a mantissa of up to 2 is left with the code's error)
    da = product(dz, half, w, torch.full_like(w, 2 * 2.0 ** -25 * w_unit), p.N)
    db = product(dz.t(), half.t(), a, torch.full_like(a, 2 * 2.0 ** -25 * a_unit), p.M)
    # sums of 32 rows by halves, of parts in chains of M / 256 + 8; dz with a mantissa and without it: 4 roundings
    dbias = dz.sum(dim=0), dz_tol.sum(dim=0) + (5 + p.M / 256 + 8 + 4) * 2.0 ** -24 * (dz.abs() + dz_tol).sum(dim=0)
    return (da[0], db[0], dbias[0]), (da[1], db[1], dbias[1])


# unit roundoff and half of the smallest step
ROUND = {torch.bfloat16: (2.0 ** -8, 2.0 ** -134), torch.float16: (2.0 ** -11, 2.0 ** -25),
         torch.float32: (2.0 ** -24, 2.0 ** -150)}


def assert_close(got, want, tol, what=""):
    """|got - want| within tol and the rounding of got's type; NaN and infinities in the same places."""
    u, tiny = ROUND[got.dtype]
    g = got.double()
    assert g.shape == want.shape, (what, g.shape, want.shape)
    assert torch.equal(g.isnan(), want.isnan()), f"{what}: NaN in other places"
    inf = want.isinf()
    assert torch.equal(g[inf], want[inf]), f"{what}: infinities differ"
    fin = want.isfinite()
    err, lim = (g - want).abs()[fin], (u * (want.abs() + tol) + tol + tiny)[fin]
    bad = ~(err <= lim)
    if bool(bad.any()):
        i = int((err / lim.clamp_min(1e-300)).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; {float(g[fin][i])} for {float(want[fin][i])} "
                             f"(error {float(err[i]):.3g}, allowed {float(lim[i]):.3g})")
