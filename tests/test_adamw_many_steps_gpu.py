"""AdamW with states in 8 bits over many steps: where a gradient ends, or falls to
a millionth of its block's, the weights do as with states in 32 bits."""
from __future__ import annotations

import math
import warnings

import pytest
import torch

import fp8_scaled_gemm_gb300 as fm

pytestmark = pytest.mark.gpu

F32, E4M3 = torch.float32, torch.float8_e4m3fn
N = 2048


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class Run:
    """A tensor of N weights with states of zeros; every fourth one's gradient changes after 300 steps."""

    def __init__(self, **kw):
        self.kw = {"lr": 1e-3, "beta1": 0.9, "eps": 1e-12, "weight_decay": 0.0, **kw}
        self.w = torch.zeros(N, device="cuda")
        self.m, self.v = (torch.zeros(N, device="cuda").to(E4M3) for _ in range(2))
        self.ms, self.vs = (torch.zeros(N // 256, device="cuda") for _ in range(2))
        g = torch.Generator().manual_seed(3)
        self.sign = torch.sign(torch.randn(N, generator=g)).cuda()
        self.noise = [torch.randn(N, generator=g).cuda() for _ in range(16)]
        self.off = torch.arange(N, device="cuda") % 4 == 0
        self.t = 0

    def steps(self, count, factor=1.0):
        """`count` steps, the gradients of every fourth weight times `factor`, without noise where that is not 1."""
        for _ in range(count):
            self.t += 1
            g = self.sign + 0.3 * self.noise[self.t % 16]
            if factor != 1.0:
                g = torch.where(self.off, self.sign * factor, g)
            fm.fp8_adamw([self.w], [g], [self.m], [self.v], self.t, exp_avg_scales=[self.ms], exp_avg_sq_scales=[self.vs], **self.kw)


# With beta1 = 0.9 the mean of |m| in codes' units falls by a tenth a step: after 600 steps, 0.9^600 x 448 x 2^9, times how far
# the block's scale moves (a factor of 4 at most for these gradients): under 1e-21. A code is not zero with at most that
# probability. What is zero with a gradient of zero moves no weight. (beta1 = 0.95: 1500 steps, 1e-27.)
@pytest.mark.parametrize("beta1,beta2,wait", [(0.9, 0.95, 600), (0.9, 0.999, 600), (0.95, 0.99, 1500)])
@pytest.mark.parametrize("rounding", [None, "stochastic"])
def test_weights_rest_where_the_gradient_has_ended(beta1, beta2, wait, rounding):
    r = Run(beta1=beta1, beta2=beta2, **({"exp_avg_rounding": rounding} if rounding else {}))
    r.steps(300)
    r.steps(wait, 0.0)
    kept = r.w.clone()
    assert not bool(r.m.float()[r.off].any())
    r.steps(600, 0.0)
    assert torch.equal(r.w[r.off], kept[r.off]) and bool((r.w != kept)[~r.off].all())


@pytest.mark.parametrize("beta1,beta2,wait", [(0.9, 0.95, 600), (0.9, 0.99, 600), (0.95, 0.99, 1500)])
def test_weights_turn_with_a_gradient_that_is_small(beta1, beta2, wait):
    """The gradient falls to a millionth and turns: the mean of the codes follows it, so that a code that is not zero has the
    new sign, and the weights go back as with states in 32 bits."""
    r = Run(beta1=beta1, beta2=beta2, exp_avg_rounding="stochastic")
    r.steps(300)
    r.steps(wait, -1e-6)
    kept = r.w.clone()
    assert not bool((r.m.float() * -r.sign < 0)[r.off].any())
    r.steps(1000, -1e-6)
    moved = ((r.w - kept) * r.sign)[r.off]
    assert bool((moved >= 0).all()) and float(moved.mean()) > 0


def test_rounding_of_the_moment_keeps_its_mean():
    """m that goes from 0.3 towards 0.2 of the block's largest by a fiftieth a step: the nearest code would be the first one
    every time."""
    n = 256 * 400
    m, v = torch.full((n,), 0.3, device="cuda"), torch.full((n,), 0.5, device="cuda")
    m[::256], v[::256] = 1.0, 1.0
    m[1::2] *= -1.0
    g = torch.full((n,), 0.2, device="cuda")
    g[::256] = 1.0
    g[1::2] *= -1.0
    ms, vs = (torch.full((400,), 1.0 / 448, device="cuda") for _ in range(2))
    m, v, w = (m * 448).to(E4M3), (v * 448).to(E4M3), torch.zeros(n, device="cuda")
    start = float(m.float()[2]) / 448
    for step in range(1, 41):
        fm.fp8_adamw([w], [g], [m], [v], step, lr=0.0, beta1=0.98, exp_avg_scales=[ms], exp_avg_sq_scales=[vs],
                     exp_avg_rounding="stochastic")
    got = (m.double().reshape(-1, 256) * ms.double()[:, None])
    want = 0.2 + (start - 0.2) * 0.98 ** 40
    # each of 102000 values took 40 roundings between codes at most 16 / 448 apart, with a standard deviation of at most half
    # of that each: their mean's is under sqrt(40) x 8 / 448 / sqrt(102000) = 3.6e-4, six of which are allowed
    for sign, part in ((1.0, got[:, 2::2]), (-1.0, got[:, 1::2])):
        assert abs(float(part.mean()) * sign - want) < 6 * 3.6e-4 * math.sqrt(2)
    assert start - want > 4e-2


def chance(q, u):
    """q to a value that e4m3 holds, up or down by u (20 bits)."""
    a = q.abs()
    # codes are 2^-9 apart up to 2^-5, an eighth of the power of two above
    more = torch.where(a < 2.0 ** -6, 2.0 ** -6, 0.0)
    up = (((a + more).view(torch.int32) + u) & -(1 << 20)).view(F32) - more
    return torch.where(up == 0, 0.0, torch.copysign(up, q)).clamp(-448.0, 448.0)


@pytest.mark.parametrize("rounding", [None, "nearest", "stochastic"])
@pytest.mark.parametrize("shift", [0, 1])
def test_bits_of_the_moments_codes(rounding, shift):
    """Codes of m after a step: by the hash, or the nearest ones, and by the hash where the gradient is zero."""
    n, step, b1 = 70001, 11, 0.9
    gen = torch.Generator(device="cuda").manual_seed(5)
    g = torch.randn(n + shift, generator=gen, device="cuda")[shift:]
    g[::5] = 0.0
    m0 = torch.randn(n, generator=gen, device="cuda") * torch.exp(2 * torch.randn(n, generator=gen, device="cuda"))
    blocks = -(-n // 256)
    ms = torch.nn.functional.pad(m0, (0, blocks * 256 - n)).reshape(-1, 256).abs().amax(dim=1) / 448
    spread = ms.repeat_interleave(256)[:n]
    m = (m0 / spread).clamp(-448, 448).to(E4M3)
    v, vs, w = torch.zeros(n, device="cuda").to(E4M3), torch.zeros(blocks, device="cuda"), torch.zeros(n, device="cuda")
    new = (m.float() * spread) * b1 + g * (1.0 - b1)
    fm.fp8_adamw([w], [g], [m], [v], step, beta1=b1, exp_avg_scales=[ms], exp_avg_sq_scales=[vs],
                 **({} if rounding is None else {"exp_avg_rounding": rounding}))
    q = new / ms.repeat_interleave(256)[:n]
    x = (torch.arange(n, device="cuda") * 0x9E3779B1 + step * 0x85EBCA77) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x2C1B3C6D) & 0xFFFFFFFF
    x = ((x ^ (x >> 13)) * 0x297A2D39) & 0xFFFFFFFF
    x = x ^ (x >> 16)
    u = (((x * 0x9E3779B1) & 0xFFFFFFFF) >> 12).to(torch.int32)
    near = q.clamp(-448, 448).to(E4M3)
    by_chance = chance(q, u).to(E4M3)
    want = by_chance if rounding == "stochastic" else torch.where(g == 0, by_chance.float(), near.float()).to(E4M3)
    assert torch.equal(m.view(torch.uint8), want.view(torch.uint8))


def test_rounding_is_one_of_two_and_of_states_in_8_bits():
    x = [torch.zeros(8, device="cuda") for _ in range(4)]
    with pytest.raises(ValueError, match="exp_avg_rounding"):
        fm.fp8_adamw(x[:1], x[1:2], x[2:3], x[3:], 1, exp_avg_rounding="up")
    with pytest.raises(ValueError, match="exp_avg_rounding"):
        fm.fp8_adamw(x[:1], x[1:2], x[2:3], x[3:], 1, exp_avg_rounding="stochastic")
    fm.fp8_adamw(x[:1], x[1:2], x[2:3], x[3:], 1, exp_avg_rounding="nearest")


def test_special_values_with_chance():
    m, v = (torch.zeros(512, device="cuda").to(E4M3) for _ in range(2))
    ms, vs, w, g = torch.zeros(2, device="cuda"), torch.zeros(2, device="cuda"), torch.zeros(512, device="cuda"), torch.ones(512, device="cuda")
    g[300] = math.nan
    g[0] = 0.0
    fm.fp8_adamw([w], [g], [m], [v], 1, exp_avg_scales=[ms], exp_avg_sq_scales=[vs], exp_avg_rounding="stochastic")
    assert bool(m.float()[256:].isnan().all()) and not bool(m.float()[:256].isnan().any())
    assert float(m.float()[0]) == 0.0 and bool((m.float()[1:256] == 448.0).all())


def test_a_captured_step_rounds_as_an_eager_one():
    """The hash takes the step that the device holds when the graph runs."""
    a, b = Run(exp_avg_rounding="stochastic", beta2=0.99), Run(exp_avg_rounding="stochastic", beta2=0.99)
    step, g = torch.ones(1, dtype=torch.int64, device="cuda"), torch.zeros(N, device="cuda")

    def one():
        fm.fp8_adamw([a.w], [g], [a.m], [a.v], step, exp_avg_scales=[a.ms], exp_avg_sq_scales=[a.vs], **a.kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one()
    torch.cuda.current_stream().wait_stream(side)
    for t in (a.w, a.ms, a.vs, a.m.view(torch.uint8), a.v.view(torch.uint8), step):
        t.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step += 1
        one()
    for t in range(1, 20):
        g.copy_(a.sign + 0.3 * a.noise[t % 16])
        graph.replay()
        b.steps(1)
    for x, y in ((a.m, b.m), (a.v, b.v), (a.ms, b.ms), (a.vs, b.vs)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    # pow in double on either side: an ulp of double, which may turn an fp32 factor's rounding
    assert float((a.w - b.w).norm()) <= 1e-6 * float(b.w.norm())


def test_a_warning_where_the_rounding_is_not_chosen():
    x = [torch.zeros(8, device="cuda") for _ in range(2)]
    s = [torch.zeros(8, device="cuda").to(E4M3) for _ in range(2)]
    sc = [torch.zeros(1, device="cuda") for _ in range(2)]
    args = (x[:1], x[1:], s[:1], s[1:], 1)
    for rounding, warned in (("nearest", False), ("stochastic", False), (None, True), (None, False)):
        fm._warned_of_nearest = rounding is None and not warned
        with warnings.catch_warnings(record=True) as seen:
            warnings.simplefilter("always")
            fm.fp8_adamw(*args, exp_avg_scales=sc[:1], exp_avg_sq_scales=sc[1:], exp_avg_rounding=rounding)
        assert bool(seen) == warned and all("exp_avg_rounding" in str(w.message) for w in seen)
