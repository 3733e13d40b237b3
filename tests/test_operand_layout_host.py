"""Operands of one row or one column: the kernels read K contiguous bytes of
each, so an inner stride other than 1 is refused there too (no GPU)."""
from __future__ import annotations

import pytest
import torch

import fp8_scaled_gemm_gb300 as fm

E4M3 = torch.float8_e4m3fn
K, N = 32, 8


def codes(*shape):
    return torch.zeros(shape).to(E4M3)


ONE = torch.ones(1)
OUT = torch.zeros((1, N), dtype=torch.bfloat16)
A, B = codes(1, K), codes(N, K).t()


def calls(a, b):
    """Each entry that takes the operands as they are."""
    m, n = a.shape[0], b.shape[1]
    out = torch.zeros((m, n), dtype=torch.bfloat16)
    args = (a, b, ONE, ONE, fm.SCALE_TENSOR)
    return {
        "mm": lambda: fm.fp8_scaled_mm(*args, out=out),
        "config": lambda: fm.fp8_scaled_mm_config(*args, out=out),
        "ex": lambda: fm.fp8_scaled_mm_ex(*args, out=out),
        "noalloc": lambda: fm.fp8_scaled_mm_noalloc(*args, out=out),
        "host": lambda: fm.fp8_scaled_mm_host(*args, out=out),
        "epilogue": lambda: fm.fp8_scaled_mm_epilogue(*args, out=out),
        "act_grad": lambda: fm.fp8_scaled_mm_act_grad(*args, out, fm.ACT_GELU),
    }


ENTRIES = sorted(calls(A, B))


@pytest.mark.parametrize("entry", ENTRIES)
def test_one_row_with_an_inner_stride_is_refused(entry):
    for a in (codes(2, 2 * K)[:1, ::2], codes(1, 2 * K)[:, ::2], codes(K, 3).t()[:1]):
        assert a.shape == (1, K) and a.stride(1) != 1
        with pytest.raises(ValueError, match="A must be row-major"):
            calls(a, B)[entry]()


@pytest.mark.parametrize("entry", ENTRIES)
def test_one_column_with_an_inner_stride_is_refused(entry):
    for b in (codes(K, 5)[:, :1], codes(N, 2 * K).t()[::2, :1]):
        assert b.shape == (K, 1) and b.stride(0) != 1
        with pytest.raises(ValueError, match="B must be column-major"):
            calls(A, b)[entry]()


@pytest.mark.parametrize("entry", [e for e in ENTRIES if e != "host"])
def test_one_row_and_one_column_of_contiguous_bytes_pass_the_layout_check(entry):
    """Whatever the outer stride: the next check (host tensors) refuses them."""
    for a, b in ((codes(3, 2 * K)[:1, :K], codes(1, K).t()), (codes(1, K), codes(4, 3 * K)[:, :K].t()[:, :1]),
                 (codes(1, K).as_strided((1, K), (1, 1)), codes(K, 1))):
        with pytest.raises(ValueError, match="CUDA tensors"):
            calls(a, b)[entry]()
