"""Refusals of the product's extended epilogue, before any CUDA call: status
codes of the C entries and the binding's own checks (no GPU)."""
from __future__ import annotations

import ctypes

import pytest
import torch

import fp8_scaled_gemm_gb300 as fm
from fp8_scaled_gemm_gb300 import _build

P = ctypes.c_void_p
AT = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fm.load()


def epilogue(lib, act=1, res=AT + 4096, ldr=0, pre=AT + 8192, ldp=0, out=AT + 64, M=64, N=64, K=64, out_type=0, ldo=0,
             a_type=0, variant=0, give=True):
    e = fm.Epilogue(act, res, ldr, pre, ldp)
    o = fm.Options(a_type, 0, out_type, variant, 0, 0, ldo)
    return lib.fp8_scaled_mm_epilogue(P(AT), P(AT), P(AT), P(AT), 1, None, P(out), M, N, K, None, ctypes.byref(o),
                                      ctypes.byref(e) if give else None)


@pytest.mark.parametrize("kw,code", [
    (dict(give=False), -1), (dict(act=-1), -4), (dict(act=5), -4), (dict(out_type=4), -4), (dict(out_type=-1), -4),
    (dict(ldr=63), -2), (dict(ldr=-1), -2), (dict(ldp=1), -2), (dict(ldp=1 << 36), -2),
    (dict(res=AT + 1), -3), (dict(pre=AT + 3), -3), (dict(res=AT + 2, out_type=2), -3), (dict(pre=AT + 6, out_type=2), -3),
    (dict(pre=AT + 64), -4),                               # z onto the output
    (dict(pre=AT + 4096), -4),                             # z onto the residual
    (dict(res=AT + 64, ldr=72), -4),                       # in place with another leading dimension
    (dict(res=AT + 64, out_type=3), -4),                   # in place over fp8 codes
    (dict(K=24), -2), (dict(M=-1), -2), (dict(a_type=2), -4), (dict(variant=9), -4),
])
def test_epilogue_refusals(lib, kw, code):
    assert epilogue(lib, **kw) == code


def test_epilogue_empty_problem_is_a_noop(lib):
    assert epilogue(lib, M=0) == 0
    assert epilogue(lib, N=0) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(act=0), -4), (dict(act=5), -4), (dict(z=None), -1), (dict(z=AT + 1), -3), (dict(ldz=32), -2),
    (dict(z=AT + 64, ldz=80), -4), (dict(out_type=7), -4), (dict(K=8), -2),
])
def test_act_grad_product_refusals(lib, kw, code):
    a = dict(act=2, z=AT + 4096, ldz=0, out_type=0, K=64) | kw
    o = fm.Options(0, 0, a["out_type"], 0, 0, 0, 0)
    assert lib.fp8_scaled_mm_act_grad(P(AT), P(AT), P(AT), P(AT), 1, a["act"], P(a["z"]) if a["z"] else None, a["ldz"],
                                      P(AT + 64), 64, 64, a["K"], None, ctypes.byref(o)) == code


def test_binding_refuses_wrong_operands():
    A = torch.zeros((4, 16)).to(torch.float8_e4m3fn)
    B = torch.zeros((8, 16)).to(torch.float8_e4m3fn).t()
    one, z = torch.ones(1), torch.zeros((4, 8), dtype=torch.bfloat16)
    for a, b, sa, sb, mode in ((A, B, one, one, 0),                        # host tensors
                               (A[0], B, one, one, 0), (A, B[:8], one, one, 0), (A.float(), B, one, one, 0),
                               (A.t().contiguous().t(), B, one, one, 0), (A, B.contiguous(), one, one, 0),
                               (A, B, one, one, 2), (A, B, one, one, 1), (A, B, one.double(), one, 0),
                               (A, B, one, torch.ones(2), 0)):
        with pytest.raises(ValueError):
            fm.fp8_scaled_mm_epilogue(a, b, sa, sb, mode)
        with pytest.raises(ValueError):
            fm.fp8_scaled_mm_act_grad(a, b, sa, sb, mode, z, 2)
    for call in (lambda: fm.fp8_scaled_mm_epilogue(None, B, one, one, 0),
                 lambda: fm.fp8_scaled_mm_epilogue(A, B, one, one, "row"),
                 lambda: fm.fp8_scaled_mm_act_grad(A, B, one, 1.0, 0, z, 2),
                 lambda: fm.fp8_layer_norm(3), lambda: fm.fp8_act_grad(z, "z", 1)):
        with pytest.raises(TypeError):
            call()
