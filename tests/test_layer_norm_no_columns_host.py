"""Rows of no columns have no mean: layer norm refuses them instead of returning
statistics and scales that nothing has written (fake tensors: no GPU)."""
from __future__ import annotations

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import fp8_scaled_gemm_gb300 as fm
from fp8_scaled_gemm_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("q_dtype", [None, torch.float8_e4m3fn])
def test_rows_of_no_columns_are_refused(dtype, q_dtype):
    with FakeTensorMode():
        x = torch.empty((5, 0), dtype=dtype, device="cuda:0")
        y = torch.empty((5, 0), dtype=dtype, device="cuda:0")
    for kw in (dict(), dict(y=y), dict(return_y=False)):
        with pytest.raises(ValueError, match="at least one column"):
            fm.fp8_layer_norm(x, q_dtype=q_dtype, **kw)
