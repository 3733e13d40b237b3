"""fp8_act_grad on the GPU against 64-bit formulas: dz within its type's
rounding and the fp32 slope's error; dbias within the error of fp32 sums in
chains of at most 128 additions (tests/_reference64.py)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import _reference64 as r64

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def on_gpu(t, ld=None, shift=0):
    M, N = t.shape
    ld = ld or N
    buf = torch.full((shift + M * ld + 8,), 7.0, dtype=t.dtype, device="cuda")
    v = buf[shift:shift + M * ld].view(M, ld)[:, :N]
    v.copy_(t)
    return v


def run(M, N, *, act="gelu", dtype=BF16, ld=(None, None, None), shift=0, dz=True, dbias=True, in_place=None, seed=3):
    import fp8_scaled_gemm_gb300 as fm
    dy, z = randn((M, N), dtype, seed, 0.5), randn((M, N), dtype, seed + 1, 2.0)
    want = r64.f64(dy) * r64.slope(r64.f64(z), act)
    gy, gz = on_gpu(dy, ld[0], shift), on_gpu(z, ld[1], shift)
    out = {"dy": gy, "z": gz}.get(in_place)
    if out is None and ld[2]:
        out = on_gpu(torch.zeros((M, N), dtype=dtype), ld[2], shift)
    got = fm.fp8_act_grad(gy, None if act == "none" else gz, r64.ACTS[act], dz=out, return_dz=dz, return_dbias=dbias)
    if dz:
        r64.assert_close(got[0], want, r64.ACT_ERR * np.abs(r64.f64(dy)), "dz")
    else:
        assert got[0] is None
    if dbias:
        tol = r64.SUM_ERR * np.abs(want).sum(axis=0) + r64.ACT_ERR * np.abs(r64.f64(dy)).sum(axis=0)
        r64.assert_close(got[1], want.sum(axis=0), tol, "dbias")
    else:
        assert got[1] is None


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("N", [264, 265])
def test_activations_and_types(act, dtype, N):
    _need_gpu()
    run(70, N, act=act, dtype=dtype)


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 130, 2100])
@pytest.mark.parametrize("N", [1, 3, 8, 255, 256, 257, 512, 1000, 5003])
def test_sizes(M, N):
    _need_gpu()
    run(M, N, act="silu")


@pytest.mark.parametrize("M,N", [(20000, 24), (20001, 33), (3, 70000), (2, 70001)])
def test_long_and_wide(M, N):
    _need_gpu()
    run(M, N, act="gelu_tanh")


@pytest.mark.parametrize("dz,dbias", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("N", [200, 201])
def test_parts(dz, dbias, act, N):
    _need_gpu()
    run(50, N, act=act, dz=dz, dbias=dbias)


@pytest.mark.parametrize("N,ld,shift", [(264, (272, 280, 288), 0), (264, (265, 270, 271), 0), (264, (264, 264, 264), 1),
                                        (263, (263, 300, 302), 3), (264, (265, 267, 269), 0),
                                        (264, (265, 267, 269), 1), (100, (101, 101, 103), 0)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides_and_alignment(N, ld, shift, dtype):
    _need_gpu()
    run(60, N, ld=ld, shift=shift, dtype=dtype)


@pytest.mark.parametrize("where", ["dy", "z"])
@pytest.mark.parametrize("N", [264, 265])
def test_in_place(where, N):
    _need_gpu()
    run(60, N, in_place=where)


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_non_finite_z(act):
    """Limits of the slope at infinities, NaN at NaN; relu blocks an infinite
    gradient where its slope is 0."""
    _need_gpu()
    import fp8_scaled_gemm_gb300 as fm
    z = torch.tensor([[float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1e30, -1e30, 60.0, -60.0]]).repeat(9, 1)
    dy = torch.ones_like(z) * 0.5
    got = fm.fp8_act_grad(dy.cuda(), z.cuda(), r64.ACTS[act])
    want = 0.5 * r64.slope(r64.f64(z), act)
    r64.assert_close(got[0], want, 4e-6, "dz")
    r64.assert_close(got[1], want.sum(axis=0), 4e-5, "dbias")
    if act == "relu":
        inf = torch.full((1, 3), float("inf"), device="cuda")
        z3 = torch.tensor([[-1.0, 0.0, 2.0]], device="cuda")
        assert fm.fp8_act_grad(inf, z3, 1)[0].tolist() == [[0.0, 0.0, float("inf")]]


def test_no_rows_repeatability_and_streams():
    _need_gpu()
    import fp8_scaled_gemm_gb300 as fm
    dz, db = fm.fp8_act_grad(torch.empty((0, 9), device="cuda"), torch.empty((0, 9), device="cuda"), 2)
    assert dz.shape == (0, 9) and not db.any() and db.numel() == 9
    dy, z = randn((3000, 1000), BF16, 1).cuda(), randn((3000, 1000), BF16, 2).cuda()
    first = fm.fp8_act_grad(dy, z, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = fm.fp8_act_grad(dy, z, 2, stream=s)
    s.synchronize()
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_stray_writes():
    _need_gpu()
    import fp8_scaled_gemm_gb300 as fm
    for N in (40, 41, 520):
        M = 21
        dy, z = randn((M, N), BF16, 1).cuda(), randn((M, N), BF16, 2).cuda()
        buf = torch.full((M + 2, N + 24), 9.0, dtype=BF16, device="cuda")
        keep = torch.ones_like(buf, dtype=torch.bool)
        keep[1:1 + M, 8:8 + N] = False
        sums = torch.full((N + 8,), 9.0, device="cuda")
        fm.fp8_act_grad(dy, z, 2, dz=buf[1:1 + M, 8:8 + N], dbias=sums[4:4 + N])
        assert bool((buf[keep] == 9.0).all())
        assert bool((sums[:4] == 9.0).all()) and bool((sums[4 + N:] == 9.0).all())


@pytest.mark.parametrize("N,ld,shift", [(2, None, 0), (62, None, 0), (90, None, 0), (130, None, 0), (1002, None, 0),
                                        (1002, (1004, 1006, 1010), 0), (1002, (1004, 1006, 1010), 2),
                                        (1002, (1002, 1002, 1002), 1), (1002, (1003, 1004, 1002), 0)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_even_widths(N, ld, shift, dtype):
    """Pairs of 16-bit elements where rows start on 4 bytes."""
    _need_gpu()
    kw = {} if ld is None else dict(ld=ld, shift=shift)
    for M in (1, 37, 700):
        run(M, N, dtype=dtype, **kw)

