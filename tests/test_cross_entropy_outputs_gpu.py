"""Gradients of the cross entropy written into tensors that are given."""
from __future__ import annotations

import pytest
import torch

import fp8_scaled_gemm_gb300 as fm
from tests._loss64 import Problem

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def test_given_gradients_are_seen_by_autograd():
    """A graph that saved a tensor refuses to go back once a gradient was written into it."""
    p = Problem(20, 40, 64)
    lse = fm.fp8_cross_entropy(*p.operands, p.target)[1]
    for name, shape in (("da", (20, 64)), ("db", (40, 64))):
        x = torch.ones(shape, dtype=BF16, device="cuda")
        w = torch.ones(shape, dtype=BF16, device="cuda", requires_grad=True)
        y = (w * x).sum()
        fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, p.dloss, **{name: x})
        with pytest.raises(RuntimeError, match="modified"):
            y.backward()
    with torch.inference_mode():
        x = torch.ones(20, 64, dtype=BF16, device="cuda")
    fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, p.dloss, da=x)
