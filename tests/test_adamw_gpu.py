"""fp8_adamw on the GPU: against the formula in 64 bits, against its single
operations in 32 bits (the same bits), and the rounding of its 8-bit states."""
from __future__ import annotations

import math

import pytest
import torch

import fp8_scaled_gemm_gb300 as fm

pytestmark = pytest.mark.gpu

BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-7, weight_decay=0.05)
U = 2.0 ** -24


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def blocks(x):
    x = x.reshape(-1)
    return torch.nn.functional.pad(x, (0, -x.numel() % 256)).reshape(-1, 256)


def spread(scales, n):
    """A block's scale beside each of its elements."""
    return scales.repeat_interleave(256)[:n]


class State:
    """Parameters with gradients and states for a call."""

    def __init__(self, sizes, param=F32, grad=None, bits=32, master=False, seed=0, shift=0):
        g = torch.Generator().manual_seed(seed)

        def place(x):
            buf = torch.zeros(x.numel() + shift, dtype=x.dtype, device="cuda")
            t = buf[shift:].view(x.shape)
            t.copy_(x)
            return t

        def randn(n):
            return torch.randn(n, generator=g)
        self.bits = bits
        self.p, self.g, self.w, self.m, self.v, self.ms, self.vs = ([] for _ in range(7))
        for n in sizes:
            w = randn(n)
            grad_values = randn(n) * torch.exp(2 * randn(n)) * 0.01
            m, v = 0.3 * grad_values + 0.003 * randn(n), grad_values.square() * 0.5 + 1e-6 * randn(n).square()
            self.p.append(place(w.to(param)))
            self.g.append(place(grad_values.to(grad or param)))
            if master:
                self.w.append(place(w))
            if bits == 32:
                self.m.append(place(m))
                self.v.append(place(v))
            else:
                for to, scales, x in ((self.m, self.ms, m), (self.v, self.vs, v.sqrt())):
                    s = blocks(x).abs().amax(dim=1) / 448
                    scales.append(place(s))
                    to.append(place((x / spread(s, n)).clamp(-448, 448).to(E4M3)))

    def call(self, step=7, **kw):
        fm.fp8_adamw(self.p, self.g, self.m, self.v, step, **{**HYPER, "masters": self.w or None,
                                                              "exp_avg_scales": self.ms or None,
                                                              "exp_avg_sq_scales": self.vs or None, **kw})

    def lists(self):
        return [self.p, self.w, self.m, self.v, self.ms, self.vs]

    def copy(self):
        c = object.__new__(State)
        c.bits = self.bits
        c.p, c.g, c.w, c.m, c.v, c.ms, c.vs = ([t.clone() for t in x] for x in
                                               (self.p, self.g, self.w, self.m, self.v, self.ms, self.vs))
        return c

    def same(self, other):
        def raw(t):
            return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])
        return all(torch.equal(raw(x), raw(y)) for a, b in zip(self.lists(), other.lists()) for x, y in zip(a, b))


def check(s: State, step=7, grad_scale=None, **kw):
    """One step of s against 64 bits, tensor by tensor."""
    old = s.copy()
    h = {**HYPER, **{k: v for k, v in kw.items() if k in HYPER}}
    lr = float(h["lr"])
    s.call(step, grad_scale=grad_scale, **kw)
    t = int(step)
    size, root = lr / (1 - h["beta1"] ** t), 1 / math.sqrt(1 - h["beta2"] ** t)
    for i in range(len(s.p)):
        n = s.p[i].numel()
        g = old.g[i].double() * (1.0 if grad_scale is None else float(grad_scale))
        w = (old.w if old.w else old.p)[i].double()
        m, v = old.m[i].double(), old.v[i].double()
        if s.bits == 8:
            m, v = m * spread(old.ms[i], n).double(), (v * spread(old.vs[i], n).double()) ** 2
        # every operation rounds its result by at most U of it: m is off by 4 U of its two terms (scale of a code or of g,
        # product, sum, the factor's own rounding), v by 6 U of itself, its root by 4 U
        m_new, v_new = h["beta1"] * m + (1 - h["beta1"]) * g, h["beta2"] * v + (1 - h["beta2"]) * g * g
        m_tol = 4 * U * (h["beta1"] * m.abs() + (1 - h["beta1"]) * g.abs()) + 2.0 ** -148
        v_tol, r = 6 * U * v_new + 2.0 ** -147, v_new.sqrt()
        r_tol = 4 * U * r + 2.0 ** -73
        denom = r * root + h["eps"]
        update = m_new / denom * size
        # the quotient: m's error, the root's, and 5 roundings; the product with size and size's own: 2; the decay 3, the
        # difference 1
        u_tol = size * m_tol / denom + update.abs() * (r_tol * root / denom + 8 * U) + 2.0 ** -148
        w_new = w * (1 - lr * h["weight_decay"]) - update
        w_tol = u_tol + 3 * U * w.abs() + U * w_new.abs()
        got = (s.w if s.w else s.p)[i].double()
        u = {F32: 0.0, BF16: 2.0 ** -8, F16: 2.0 ** -11}[F32 if s.w else s.p[i].dtype]
        assert bool(((got - w_new).abs() <= w_tol + u * w_new.abs() + 2.0 ** -25 * (u > 0)).all()), i
        if s.w:
            assert torch.equal(s.p[i], s.w[i].to(s.p[i].dtype))
        if s.bits == 32:
            assert bool(((s.m[i].double() - m_new).abs() <= m_tol).all())
            assert bool(((s.v[i].double() - v_new).abs() <= v_tol).all())
            continue
        for codes, scales, x, x_tol in ((s.m[i], s.ms[i], m_new, m_tol), (s.v[i], s.vs[i], r, r_tol)):
            want, want_tol = blocks(x).abs().amax(dim=1) / 448, blocks(x_tol).amax(dim=1) / 448
            assert bool(((scales.double() - want).abs() <= want_tol + 2 * U * want + 2.0 ** -149).all())
            c, q = codes.double(), x / spread(scales, n).double()
            q = torch.where(spread(scales, n) == 0, 0.0, q)
            off = torch.where(spread(scales, n) == 0, 0.0, x_tol / spread(scales, n).double()) + 2 * U * q.abs()
            if codes is s.m[i]:
                # to the nearest: half a step, 2^-4 relative, or half of 2^-9
                assert bool(((c - q).abs() <= 2.0 ** -4 * (q.abs() + off) + 2.0 ** -10 + off).all())
            else:
                # up or down: less than a step, 2^-3 of the power of two; what is not zero stays so
                gap = (2.0 ** torch.floor(torch.log2((q + off).clamp_min(2.0 ** -6)))) / 8
                assert bool(((c - q).abs() <= gap + off).all())
                assert torch.equal(c > 0, v_new > 0)


SIZES = [1, 2, 7, 8, 255, 256, 257, 511, 512, 2048, 5003, 70001]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad,master", [(F32, F32, False), (BF16, BF16, True), (F16, F32, True), (BF16, F32, False),
                                               (F16, F16, False), (F32, BF16, False), (F32, F16, True)])
def test_types(bits, param, grad, master):
    check(State(SIZES, param, grad, bits, master))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("shift", [1, 3, 4, 8])
def test_alignment(bits, shift):
    check(State(SIZES, BF16, BF16, bits, True, shift=shift))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [1, 31, 32, 33, 400, 401, 1000])
def test_many_tensors(bits, count):
    check(State([(37 * i) % 701 + 1 for i in range(count)], F32, F32, bits))


@pytest.mark.parametrize("bits", [32, 8])
def test_hyper_parameters(bits):
    for step, kw in ((1, {}), (100000, {}), (3, dict(weight_decay=0.0)), (2, dict(beta1=0.0)), (2, dict(beta1=0.0, beta2=0.0)),
                     (5, dict(lr=0.0)), (5, dict(lr=1.0, weight_decay=1.0)), (9, dict(eps=1.0))):
        check(State([300, 5000], bits=bits), step, **kw)
    check(State([300, 5000], bits=bits), grad_scale=torch.tensor([0.125], device="cuda"))
    check(State([300, 5000], BF16, BF16, bits, True), grad_scale=torch.tensor([3e-3], device="cuda"))


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_from_zero(bits):
    """States of zeros, several steps, with gradients that are zero in places."""
    s = State([1000, 256], bits=bits)
    for x in s.m + s.v + s.ms + s.vs:
        x.zero_()
    for step in range(1, 6):
        for g in s.g:
            g[::3] = 0.0
        s.g[1].zero_()
        check(s, step, eps=1e-8)
    assert not bool(s.m[1].float().any()) and not bool(s.v[1].float().any())


def single_operations(s: State, step, h, grad_scale=None):
    """The step in single fp32 operations."""
    size, root = h["lr"] / (1.0 - h["beta1"] ** step), 1.0 / math.sqrt(1.0 - h["beta2"] ** step)
    for i in range(len(s.p)):
        n = s.p[i].numel()
        w = s.w[i] if s.w else s.p[i].float()
        g = s.g[i].float()
        if grad_scale is not None:
            g = g * grad_scale
        m, v = s.m[i], s.v[i]
        if s.bits == 8:
            m, v = m.float() * spread(s.ms[i], n), v.float() * spread(s.vs[i], n)
            v = v * v
        m = m * h["beta1"] + g * (1.0 - h["beta1"])
        v = v * h["beta2"] + (g * g) * (1.0 - h["beta2"])
        r = torch.sqrt(v)
        w = w * (1.0 - h["lr"] * h["weight_decay"]) - (m / (r * root + h["eps"])) * size
        s.p[i].copy_(w)
        if s.w:
            s.w[i].copy_(w)
        if s.bits == 32:
            s.m[i].copy_(m)
            s.v[i].copy_(v)
            continue
        most = torch.full((1,), 448.0, device="cuda")
        s.ms[i].copy_(blocks(m).abs().amax(dim=1) / most)
        s.vs[i].copy_(blocks(r).amax(dim=1) / most)
        s.m[i].copy_(torch.where(spread(s.ms[i], n) == 0, 0.0, (m / spread(s.ms[i], n)).clamp(-448, 448)).to(E4M3))
        q = torch.where(spread(s.vs[i], n) == 0, 0.0, (r / spread(s.vs[i], n)).clamp(max=448.0))
        x = (torch.arange(n, device="cuda") * 0x9E3779B1 + step * 0x85EBCA77) & 0xFFFFFFFF
        x = ((x ^ (x >> 15)) * 0x2C1B3C6D) & 0xFFFFFFFF
        x = ((x ^ (x >> 13)) * 0x297A2D39) & 0xFFFFFFFF
        u = ((x ^ (x >> 16)) >> 12).to(torch.int32)
        up = ((q.view(torch.int32) + u) & -(1 << 20)).view(F32)
        low = torch.floor(q * 512.0 + u.float() * 2.0 ** -20) * 2.0 ** -9
        q = torch.where(q < 2.0 ** -6, torch.where(q > 0, low.clamp_min(2.0 ** -9), q), up)
        s.v[i].copy_(q.to(E4M3))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,master", [(F32, False), (BF16, True)])
def test_bits_of_single_operations(bits, param, master):
    """A step is its formula operation by operation: equal bits, over several steps."""
    s = State([70001, 4096, 3, 100000], param, param, bits, master)
    plain = s.copy()
    clip = torch.tensor([0.7], device="cuda")
    for step in range(5, 9):
        s.call(step, grad_scale=clip)
        single_operations(plain, step, HYPER, clip)
        assert s.same(plain)


@pytest.mark.parametrize("numerators", ["ones", "random"])
def test_roots_and_quotients_of_every_mantissa(numerators):
    """v over all fp32 values in [1, 4): with beta1 = beta2 = 1/2, no gradient, eps of 2^-60 and t so large that the
    corrections are 1, the new v and m are halves of the old and w becomes -m / sqrt(v), both correctly rounded."""
    n = 1 << 24
    v = (torch.arange(n, device="cuda", dtype=torch.int32) + 0x3F800000).view(F32)
    m = torch.ones(n, device="cuda")
    if numerators == "random":
        m = torch.randn(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    w, want = torch.zeros(n, device="cuda"), -(m / torch.sqrt(v))
    fm.fp8_adamw([w], [torch.zeros(n, device="cuda")], [2 * m], [2 * v], 200, lr=1.0, beta1=0.5, beta2=0.5, eps=2.0 ** -60,
                 weight_decay=0.0)
    assert torch.equal(w, want)


def test_rounding_of_the_root_keeps_its_mean():
    """Roots that decay by 0.05 % a step beside one that stays: the nearest code would be the old one every time."""
    n = 256 * 400
    s = State([n], bits=8)
    root = torch.full((n,), 0.3, device="cuda")
    root[::256] = 1.0
    s.vs[0].fill_(1.0 / 448)
    s.v[0].copy_((root * 448).to(E4M3))
    s.ms[0].zero_()
    s.m[0].zero_()
    s.g[0].zero_()
    s.g[0][::256] = 1.0
    start = float(s.v[0].float()[1] * s.vs[0][0])
    for step in range(1, 41):
        s.call(step, beta2=0.999, lr=0.0)
    want = start * 0.999 ** 20
    got = (s.v[0].double() * spread(s.vs[0], n).double()).reshape(-1, 256)[:, 1:]
    # each of the 102000 values took 40 roundings between codes at most 16 / 448 apart, with a standard deviation of at
    # most half of that each: their mean's is under sqrt(40) x 8 / 448 / sqrt(102000) = 3.6e-4, six of which are allowed
    assert abs(float(got.mean()) - want) < 6 * 3.6e-4
    assert start - want > 5e-3


def test_special_values():
    """NaN and infinities stay in their element (32 bits) or block (8 bits)."""
    for bits in (32, 8):
        s = State([2048], bits=bits)
        s.g[0][300] = math.nan
        s.g[0][1000] = math.inf
        s.call()
        bad = torch.zeros(2048, dtype=torch.bool, device="cuda")
        bad[300] = bad[1000] = True
        assert torch.equal(~s.p[0].isfinite(), bad)
        if bits == 8:
            codes = s.m[0].float().isnan().reshape(8, 256)
            assert torch.equal(codes.all(dim=1), torch.tensor([False, True] + 6 * [False], device="cuda"))
            assert not bool(s.m[0].float().reshape(8, 256)[[0, 2, 4, 5, 6, 7]].isnan().any())
            assert torch.equal(s.vs[0].isnan(), torch.tensor([False, True] + 6 * [False], device="cuda"))
            assert bool(s.vs[0][3].isinf())
        else:
            assert torch.equal(~s.m[0].isfinite(), bad) and torch.equal(~s.v[0].isfinite(), bad)


def test_device_step_and_lr_in_a_graph():
    """A captured step reads lr and the step when it is replayed."""
    for bits in (32, 8):
        s = State([5000, 300], BF16, BF16, bits, True)
        eager = s.copy()
        step, lr = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(1, device="cuda")
        keep = s.copy()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step.fill_(1)
            s.call(step, lr=lr)
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(s.lists(), keep.lists()):
            for x, y in zip(a, b):
                x.copy_(y)
        step.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step += 1
            s.call(step, lr=lr)
        for i, rate in enumerate((0.0078125, 0.001953125, 0.5)):     # (fp32 values, so that the host's are the same)
            lr.fill_(rate)
            graph.replay()
            eager.call(i + 1, lr=rate)
            torch.cuda.synchronize()
            # pow in double on either side: an ulp of double, which may turn an fp32 factor's rounding
            for a, b in zip(s.lists(), eager.lists()):
                for x, y in zip(a, b):
                    assert float((x.double() - y.double()).norm()) <= 1e-6 * float(y.double().norm()) + 1e-30


def test_streams_do_not_meet():
    states = [State([40000 + i, 77], bits=8, seed=i) for i in range(3)]
    want = [s.copy() for s in states]
    for w in want:
        for step in range(1, 6):
            w.call(step)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    for step in range(1, 6):
        for s, st in zip(states, streams):
            s.call(step, stream=st)
    torch.cuda.synchronize()
    assert all(s.same(w) for s, w in zip(states, want))


def test_what_is_behind_a_tensor_stays():
    for bits in (32, 8):
        s = State([1000], bits=bits)
        around = [torch.full((1100,), 7.0, device="cuda").to(x[0].dtype) for x in (s.p, s.m, s.v)]
        inner = [a[50:1050] for a in around]
        for t, x in zip(inner, (s.p, s.m, s.v)):
            t.copy_(x[0])
        fm.fp8_adamw([inner[0]], s.g, [inner[1]], [inner[2]], 3, exp_avg_scales=s.ms or None, exp_avg_sq_scales=s.vs or None)
        for a in around:
            assert bool((a.float()[:50] == 7).all()) and bool((a.float()[1050:] == 7).all())


def test_autograd_sees_the_update():
    """A graph that saved a parameter refuses to go back through its updated values."""
    s = State([256])
    w = s.p[0].requires_grad_()
    y = (w * w).sum()
    s.call()
    with pytest.raises(RuntimeError, match="modified"):
        y.backward()


def test_empty():
    fm.fp8_adamw([], [], [], [], 1)
    e = torch.empty(0, device="cuda")
    fm.fp8_adamw([e], [e.clone()], [e.clone()], [e.clone()], 1)
    s = State([300])
    t = s.copy()
    t.call(3)
    fm.fp8_adamw([s.p[0], e], [s.g[0], e], [s.m[0], e], [s.v[0], e], 3, **HYPER)
    assert s.same(t)


def test_refusals():
    s, e = State([300, 20]), State([300, 20], bits=8)
    before, before8 = s.copy(), e.copy()
    good = dict(params=s.p, grads=s.g, exp_avgs=s.m, exp_avg_sqs=s.v, step=1)
    for kw in (dict(grads=s.g[:1]), dict(grads=None), dict(exp_avgs=[s.m[0], s.m[1][:-1]]), dict(exp_avg_sqs=s.v[::-1]),
               dict(params=[s.p[0], s.p[1].half()]), dict(grads=[s.g[0].cpu(), s.g[1]]), dict(masters=s.p[:1]),
               dict(masters=[s.p[0].half(), s.p[1].half()]), dict(exp_avg_scales=e.ms), dict(exp_avgs=e.m, exp_avg_sqs=e.v),
               dict(exp_avgs=[x.half() for x in s.m]), dict(exp_avgs=e.m, exp_avg_scales=e.ms, exp_avg_sq_scales=e.vs),
               dict(params=[s.p[0], torch.zeros(40, device="cuda")[::2]]),
               dict(grad_scale=torch.ones(2, device="cuda")), dict(grad_scale=torch.ones(1)),
               dict(step=torch.ones(1, device="cuda")), dict(step=torch.ones(1, dtype=torch.int64)),
               dict(lr=torch.ones(1, device="cuda", dtype=torch.float64)),
               dict(exp_avgs=e.m, exp_avg_sqs=e.v, exp_avg_scales=[e.ms[0][:-1], e.ms[1]], exp_avg_sq_scales=e.vs),
               dict(params=[s.p[0].double(), s.p[1].double()])):
        with pytest.raises(ValueError):
            fm.fp8_adamw(**{**good, **kw})
    for kw in (dict(step=0), dict(step=-3), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1e-8), dict(lr=math.nan),
               dict(weight_decay=math.inf)):
        with pytest.raises(fm.Fp8mmError, match="SHAPE"):
            fm.fp8_adamw(**{**good, **kw})
    # memory that is written twice, or read as a gradient
    for kw in (dict(params=[s.p[0], s.p[0][:20]]), dict(grads=[s.p[0], s.g[1]]), dict(exp_avg_sqs=s.m),
               dict(exp_avgs=[s.m[0], s.m[0][280:]])):
        with pytest.raises(fm.Fp8mmError, match="MODE"):
            fm.fp8_adamw(**{**good, **kw})
    with pytest.raises(TypeError):
        fm.fp8_adamw(**{**good, "params": [1.0, 2.0]})
    with pytest.raises(TypeError):
        fm.fp8_adamw(**{**good, "params": 3})
    torch.cuda.synchronize()
    assert s.same(before) and e.same(before8)
    # one gradient for two parameters is read only
    shared = State([300, 300])
    shared.g[1] = shared.g[0]
    check(shared)


def test_inference_tensors():
    """They are refused before anything is written, and updated inside InferenceMode."""
    with torch.inference_mode():
        s = State([300])
    old = s.copy()
    with pytest.raises(ValueError, match="inference"):
        s.call()
    assert s.same(old)
    with torch.inference_mode():
        s.call()
    old.call()
    assert s.same(old)


def test_tensors_in_any_sequence():
    a, b = State([300, 5]), State([300, 5])
    a.call()
    fm.fp8_adamw(tuple(b.p), (g for g in b.g), tuple(b.m), iter(b.v), 7, **HYPER)
    assert a.same(b)
