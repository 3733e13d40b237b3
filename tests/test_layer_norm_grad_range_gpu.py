"""Layer norm's gradient where mean * rstd leaves the range of fp32: the
columns that a thread holds beyond the end of a row add nothing to its sums."""
from __future__ import annotations

import pytest
import torch

from tests import _reference64 as r64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("C", [5, 40, 41, 100, 129, 258, 264, 1000, 1001, 4100, 9000, 9001, 16392, 20002, 33001])
@pytest.mark.parametrize("x_dtype,dy_dtype", [(BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("gamma", [True, False])
def test_gradient_of_equal_elements_of_large_size(C, x_dtype, dy_dtype, gamma):
    """Rows of one value 2^120 (mean 2^120, rstd 316): xhat is 0 in every column
    of the row, so dx = rstd (w - mean w), finite."""
    import fp8_scaled_gemm_gb300 as fm
    R = 6
    g = torch.Generator().manual_seed(C)
    x = torch.full((R, C), 2.0 ** 120).to(x_dtype)
    dy = torch.randn((R, C), generator=g).to(dy_dtype)
    ga = torch.randn(C, generator=g) if gamma else None
    mean, rstd = torch.full((R,), 2.0 ** 120), torch.full((R,), 1e-5).rsqrt()
    args = (r64.f64(dy), r64.f64(x), r64.f64(ga) if gamma else 1.0, r64.f64(mean), r64.f64(rstd))
    want, tol = r64.layer_norm_grad(*args), r64.layer_norm_grad_tol(*args)
    got = fm.fp8_layer_norm_grad(dy.cuda(), x.cuda(), ga.cuda() if gamma else None, mean.cuda(), rstd.cuda())
    for name, a, b, c in zip(("dx", "dgamma", "dbeta"), got, want, tol):
        r64.assert_close(a, b, c, name)
