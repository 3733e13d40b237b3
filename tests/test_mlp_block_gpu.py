"""The MLP block example on the GPU: its values and gradients against fp32
autograd of the same block, and a short training run.

Tolerance: with one scale per row, e4m3 codes (unit roundoff 2^-4) carry an
rms error of at most 2^-4 / sqrt(3) = 3.6 % of a value, e5m2 codes 7.2 %. A
product's result is a sum of many terms whose errors are independent, so its
relative error in the 2-norm is that of one term: at most sqrt(2) x 3.6 % for
two e4m3 operands, sqrt(3.6^2 + 7.2^2) = 8.1 % with an e5m2 one. Two products
follow each other in y - x (7.3 %), three quantised factors are behind the
deepest gradient (dx: 8.1 % twice and the activations' 5.1 %, together 12.5 %).
"""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load_example():
    spec = importlib.util.spec_from_file_location("mlp_block", os.path.join(ROOT, "examples", "mlp_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


@pytest.mark.parametrize("tokens,width,hidden", [(64, 64, 256), (272, 144, 400), (512, 512, 2048)])
def test_values_and_gradients_match_autograd(tokens, width, hidden):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m = load_example()
    block = m.MlpBlock(width, hidden)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(tokens, width, generator=g, device="cuda").bfloat16()
    dy = (torch.randn(tokens, width, generator=g, device="cuda") * 0.1).bfloat16()
    block.params["b1"] += 0.1 * torch.randn(hidden, generator=g, device="cuda")
    block.params["gamma"] += 0.1 * torch.randn(width, generator=g, device="cuda")

    p = {k: v.clone().requires_grad_() for k, v in block.params.items()}
    xr = x.float().requires_grad_()
    mean = xr.mean(dim=1, keepdim=True)
    n = (xr - mean) * torch.rsqrt((xr - mean).square().mean(dim=1, keepdim=True) + 1e-5) * p["gamma"] + p["beta"]
    z = n @ p["w1"].t() + p["b1"]
    want = xr + (0.5 * z * (1.0 + torch.erf(z * 0.5 ** 0.5))) @ p["w2"].t() + p["b2"]
    want.backward(dy.float())

    y = block.forward(x)
    dx = block.backward(dy)
    assert rel(y.float() - x.float(), (want - xr).detach()) < 0.08
    assert rel(dx.float() - dy.float(), xr.grad - dy.float()) < 0.14
    for k, tol in (("b2", 0.01), ("w2", 0.10), ("b1", 0.10), ("w1", 0.14), ("gamma", 0.14), ("beta", 0.14)):
        assert block.grads[k].shape == p[k].shape
        assert rel(block.grads[k], p[k].grad) < tol, k


def test_a_short_training_run_lowers_the_loss():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    losses = load_example().train(tokens=512, width=128, hidden=512, steps=40, log=lambda s: None)
    assert losses[-1] < 0.6 * losses[0]
