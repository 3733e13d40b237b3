"""A training step's end as it is used: layer norm with codes, the product with the
vocabulary and its loss, the gradients back through both, and the update of the
weights; against 64 bits, and captured in a graph."""
from __future__ import annotations

import pytest
import torch

import fp8_scaled_gemm_gb300 as fm
from tests._loss64 import IGNORE, Problem, assert_close, grad64, loss64

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
ROW = fm.SCALE_ROWWISE
HYPER = dict(beta1=0.9, beta2=0.99, eps=1e-3, weight_decay=0.1)


class Head:
    """A norm and a vocabulary's weights, trained: bf16 weights beside fp32 originals, 8-bit states for them, fp32 ones
    for the norm's parameters."""

    def __init__(self, tokens, width, vocabulary, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def randn(*shape, scale=1.0):
            return torch.randn(*shape, generator=g, device="cuda") * scale
        self.x = randn(tokens, width).to(BF16)
        self.target = torch.randint(0, vocabulary, (tokens,), generator=g, device="cuda")
        self.target[::7] = IGNORE
        self.dloss = (1.0 / (self.target != IGNORE).sum()).reshape(1)
        self.master = randn(vocabulary, width, scale=2.0 / width ** 0.5)
        self.w = self.master.to(BF16)
        self.norm = [1.0 + randn(width, scale=0.1), randn(width, scale=0.1)]
        blocks = -(-vocabulary * width // 256)
        self.w_states = [torch.zeros(vocabulary, width, device="cuda").to(E4M3) for _ in range(2)]
        self.w_scales = [torch.zeros(blocks, device="cuda") for _ in range(2)]
        self.norm_states = [[torch.zeros(width, device="cuda") for _ in range(2)] for _ in range(2)]
        self.step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def train(self, lr=0.01):
        """One step; what it computed."""
        _, mean, rstd, q, qs = fm.fp8_layer_norm(self.x, *self.norm, q_dtype=E4M3, return_y=False)
        wq, ws = fm.fp8_quantize(self.w, ROW)
        product = (q, wq.t(), qs, ws, ROW)
        loss, lse = fm.fp8_cross_entropy(*product, self.target)
        dy, dw, _ = fm.fp8_cross_entropy_grad(*product, self.target, lse, self.dloss)
        dx, dgamma, dbeta = fm.fp8_layer_norm_grad(dy, self.x, self.norm[0], mean, rstd)
        self.step += 1
        fm.fp8_adamw([self.w], [dw], self.w_states[:1], self.w_states[1:], self.step, lr=lr, masters=[self.master],
                     exp_avg_scales=self.w_scales[:1], exp_avg_sq_scales=self.w_scales[1:], **HYPER)
        fm.fp8_adamw(self.norm, [dgamma, dbeta], *self.norm_states, self.step, lr=lr, **HYPER)
        return dict(q=q, qs=qs, wq=wq, ws=ws, loss=loss, lse=lse, dy=dy, dw=dw, dx=dx, dgamma=dgamma, dbeta=dbeta, mean=mean,
                    rstd=rstd)

    def state(self):
        return [self.master, self.w, *self.norm, *self.w_states, *self.w_scales, *self.norm_states[0], *self.norm_states[1]]


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("tokens,width,vocabulary", [(40, 64, 300), (200, 144, 1000), (300, 512, 5003)])
def test_a_step_against_64_bits(tokens, width, vocabulary):
    h = Head(tokens, width, vocabulary)
    master, gamma = h.master.double(), h.norm[0].clone()
    r = h.train()
    # loss and gradients for the codes that the norm and the quantisation gave
    p = Problem(1, 1, 16)
    p.M, p.N, p.K, p.mode, p.bias = tokens, vocabulary, width, 1, None
    p.A, p.Bt, p.B, p.sa, p.sb, p.target, p.dloss = r["q"], r["wq"], r["wq"].t(), r["qs"], r["ws"], h.target, h.dloss
    want = loss64(p)
    assert_close(r["lse"], want[1], want[3], "lse")
    assert_close(r["loss"], want[0], want[2], "loss")
    grads, tol = grad64(p, r["lse"])
    assert_close(r["dy"], grads[0], tol[0], "dy")
    assert_close(r["dw"], grads[1], tol[1], "dw")
    # the norm's gradient, of the bf16 dy: fp32 sums of at most 600 terms in chains of at most 128
    x, dy = h.x.double(), r["dy"].double()
    xhat = (x - r["mean"].double()[:, None]) * r["rstd"].double()[:, None]
    wd = dy * gamma.double()
    dx = r["rstd"].double()[:, None] * (wd - wd.mean(dim=1, keepdim=True) - xhat * (wd * xhat).mean(dim=1, keepdim=True))
    size = r["rstd"].double()[:, None] * (wd.abs() + wd.abs().mean(dim=1, keepdim=True) +
                                          xhat.abs() * (wd * xhat).abs().mean(dim=1, keepdim=True))
    assert_close(r["dx"], dx, 2.0 ** -16 * size, "dx")
    assert_close(r["dgamma"], (dy * xhat).sum(dim=0), 2.0 ** -16 * (dy * xhat).abs().sum(dim=0), "dgamma")
    # from states of zeros, t = 1, the update is lr g / (|g| + eps); 12 roundings, of the terms' sizes
    g = r["dw"].double()
    new = master * (1 - 0.01 * 0.1) - 0.01 * g / (g.abs() + 1e-3)
    assert_close(h.master, new, 12 * 2.0 ** -24 * (master.abs() + 0.01), "master")
    assert torch.equal(h.w, h.master.to(BF16))


def test_a_captured_step_replayed():
    """A graph of the step gives the bits of the steps one after the other."""
    h, eager = Head(200, 144, 1000), Head(200, 144, 1000)
    first = [t.clone() for t in h.state()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        h.train()
    torch.cuda.current_stream().wait_stream(side)
    for t, old in zip(h.state(), first):
        t.copy_(old)
    h.step.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = h.train()
    for _ in range(4):
        graph.replay()
        r = eager.train()
        torch.cuda.synchronize()
        for k in kept:
            assert torch.equal(kept[k].view(torch.uint8), r[k].view(torch.uint8)), k
    for a, b in zip(h.state(), eager.state()):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert int(h.step) == 4 and fm.fp8mm_device_status() == 0
