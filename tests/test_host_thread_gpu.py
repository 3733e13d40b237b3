"""Calls from a host thread that has made no CUDA call before."""
from __future__ import annotations

import threading

import pytest
import torch

import fp8_scaled_gemm_gb300 as fm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(5, 128, 256), (300, 512, 512)])
@pytest.mark.parametrize("call", ["mm", "noalloc", "epilogue", "act_grad", "bmm"])
def test_first_call_of_a_thread(M, N, K, call):
    g = torch.Generator(device="cuda").manual_seed(0)
    A = torch.randn((M, K), generator=g, device="cuda").to(torch.float8_e4m3fn)
    B = torch.randn((N, K), generator=g, device="cuda").to(torch.float8_e4m3fn).t()
    args = (A, B, torch.rand(M, device="cuda"), torch.rand(N, device="cuda"), 1)
    z = torch.randn((M, N), generator=g, device="cuda").bfloat16()
    want, out = torch.empty_like(z), torch.full_like(z, 7.0)
    f = {"mm": lambda o: fm.fp8_scaled_mm(*args, out=o), "noalloc": lambda o: fm.fp8_scaled_mm_noalloc(*args, out=o),
         "epilogue": lambda o: fm.fp8_scaled_mm_epilogue(*args, activation=fm.ACT_GELU, residual=z, out=o),
         "act_grad": lambda o: fm.fp8_scaled_mm_act_grad(*args, z, fm.ACT_GELU, out=o),
         "bmm": lambda o: fm.fp8_scaled_bmm(A[None], B[None], args[2], args[3], 1, out=o[None])}[call]
    f(want)
    torch.cuda.synchronize()
    errors = []

    def work():
        try:
            f(out)
        except Exception as e:      # reported by the main thread
            errors.append(e)
    t = threading.Thread(target=work)
    t.start()
    t.join(timeout=60)
    assert not t.is_alive() and errors == []
    torch.cuda.synchronize()
    assert torch.equal(out, want)
