"""fp8_adamw refuses a gradient, moment or original whose shape is not its
parameter's, also where it has as many values."""
from __future__ import annotations

import pytest
import torch

import fp8_scaled_gemm_gb300 as fm

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("which", ["grads", "exp_avgs", "exp_avg_sqs", "masters"])
@pytest.mark.parametrize("shape", [(40, 24), (960,), (24, 40, 1), (1, 24, 40), (12, 80)])
def test_another_shape_is_refused(eight, which, shape):
    def zeros(dtype=torch.float32, shape=(24, 40)):
        return torch.zeros(shape, device="cuda").to(dtype)
    state = E4M3 if eight else torch.float32
    kw = dict(params=[zeros()], grads=[zeros() + 1.0], exp_avgs=[zeros(state)], exp_avg_sqs=[zeros(state)], masters=[zeros()], step=1)
    if eight:
        kw.update(exp_avg_scales=[zeros(shape=4)], exp_avg_sq_scales=[zeros(shape=(2, 2))])
    old = kw[which][0]
    kw[which] = [old.float().reshape(-1)[:960].reshape(shape).to(old.dtype)]
    with pytest.raises(ValueError, match="shape"):
        fm.fp8_adamw(**kw)
    torch.cuda.synchronize()
    assert not bool(kw["params"][0].any())
    kw[which] = [old]
    fm.fp8_adamw(**kw)
    assert bool((kw["params"][0] != 0).all())


def test_the_gradient_of_the_product_as_the_weights_lie():
    """The gradient of B's columns is [N, K]: the weights are updated as [N, K], their [K, N] view is refused (not contiguous)
    and so is a [K, N] copy."""
    w = torch.zeros(24, 40, device="cuda")
    g, m, v = (torch.ones(24, 40, device="cuda") for _ in range(3))
    fm.fp8_adamw([w], [g], [m], [v], 1)
    for p in (w.t(), w.t().contiguous()):
        with pytest.raises(ValueError):
            fm.fp8_adamw([p], [g], [m], [v], 1)


def test_numbers_and_empty_tensors():
    x = [torch.zeros((), device="cuda") for _ in range(4)]
    fm.fp8_adamw(x[:1], x[1:2], x[2:3], x[3:], 1)
    x = [torch.zeros(0, 5, device="cuda") for _ in range(4)]
    fm.fp8_adamw(x[:1], x[1:2], x[2:3], x[3:], 1)
    with pytest.raises(ValueError, match="shape"):
        fm.fp8_adamw(x[:1], [torch.zeros(5, 0, device="cuda")], x[2:3], x[3:], 1)
