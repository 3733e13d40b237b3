"""Layer norm's fp8 codes are fp8_quantize's of the same rows, bit for bit:
scale = RN(max |y| / qmax) and code = fp8(RN(y / scale)), for every kernel.

With gamma = 0 the rows are beta's values exactly, so that the inputs can be
put on the ties between two codes, where a quotient that is one unit off takes
the other one.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_scaled_gemm_gb300 as fm

pytestmark = pytest.mark.gpu

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
QMAX = {E4M3: 448.0, E5M2: 57344.0}
MANTISSA = {E4M3: 3, E5M2: 2}

# lanes of a warp, a warp, CTAs, clusters of 2 and 8, the long kernel; groups of 8, pairs and single elements
WIDTHS = [24, 100, 512, 1002, 1003, 4096, 9000, 16384, 20002, 20001, 40000, 70001, 131080]


def codes_of(y, q_dtype):
    """(codes, scales) of fp32 rows y by correctly rounded divisions (numpy's)."""
    y = y.cpu()
    scale = np.abs(y.numpy()).max(axis=1) / np.float32(QMAX[q_dtype])
    assert scale.dtype == np.float32
    q = torch.from_numpy(y.numpy() / scale[:, None]).clamp(-QMAX[q_dtype], QMAX[q_dtype]).to(q_dtype)
    return q, torch.from_numpy(scale)


def assert_codes(got_q, got_scale, y, q_dtype):
    q, scale = codes_of(y, q_dtype)
    bad = got_scale.cpu().view(torch.int32) != scale.view(torch.int32)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} scales differ"
    bad = got_q.cpu().view(torch.uint8) != q.view(torch.uint8)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} codes differ"


def on_ties(C, q_dtype, seed, step=0):
    """Values whose quotients by their row's scale lie on the ties between two
    codes, or `step` fp32 units beside them."""
    g = torch.Generator().manual_seed(seed)
    amax = np.float32(1.0 + torch.rand(1, generator=g).item())
    scale = amax / np.float32(QMAX[q_dtype])
    m = MANTISSA[q_dtype]
    k = torch.randint(0, 1 << m, (C,), generator=g).double()
    e = torch.randint(-6, 8, (C,), generator=g).double()
    tie = (1.0 + (k + 0.5) / (1 << m)) * torch.exp2(e)                # between neighbouring codes
    v = (tie * float(scale)).float() * torch.where(torch.rand(C, generator=g) < 0.5, -1.0, 1.0)
    v = (v.view(torch.int32) + step).view(torch.float32)
    v[0] = float(amax)
    return v


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("q_dtype", [E4M3, E5M2])
def test_codes_on_ties(C, q_dtype):
    zero = torch.zeros(C, device="cuda")
    for seed in range(8):
        for step in (-1, 0, 1):
            beta = on_ties(C, q_dtype, 100 * C + seed, step).cuda()
            x = torch.randn((2, C), device="cuda")
            y, _, _, q, scale = fm.fp8_layer_norm(x, zero, beta, y_dtype=torch.float32, q_dtype=q_dtype)
            assert torch.equal(y, beta.expand(2, C))
            assert_codes(q, scale, y, q_dtype)


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_codes_of_normalised_rows(C, dtype):
    """The codes of the fp32 rows that the same call returns."""
    g = torch.Generator(device="cuda").manual_seed(C)
    x = torch.randn((max(3, (1 << 20) // C), C), generator=g, device="cuda").to(dtype)
    gamma, beta = (torch.randn(C, generator=g, device="cuda") for _ in range(2))
    y, _, _, q, scale = fm.fp8_layer_norm(x, gamma, beta, y_dtype=torch.float32, q_dtype=E4M3)
    assert_codes(q, scale, y, E4M3)


@pytest.mark.parametrize("C", [512, 4096, 20000, 131080])
@pytest.mark.parametrize("q_dtype", [E4M3, E5M2])
def test_codes_are_those_of_fp8_quantize(C, q_dtype):
    """Rows of bf16 values through both entries."""
    g = torch.Generator(device="cuda").manual_seed(C)
    for size in (1.0, 2.0 ** -110, 2.0 ** 110):       # scales in and out of the reciprocal's range
        beta = (torch.randn(C, generator=g, device="cuda") * size).bfloat16()
        want_q, want_scale = fm.fp8_quantize(beta[None], fm.SCALE_ROWWISE, dtype=q_dtype)
        got = fm.fp8_layer_norm(torch.randn((1, C), device="cuda"), torch.zeros_like(beta), beta, q_dtype=q_dtype)
        assert torch.equal(got[4].view(torch.int32), want_scale.view(torch.int32))
        assert torch.equal(got[3].view(torch.uint8), want_q.view(torch.uint8))
