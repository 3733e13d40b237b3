"""Layer norm forward and backward on the GPU against 64-bit formulas.

Bounds: tests/_reference64.py derives them from the lengths of the kernels'
fp32 summation chains; each output type adds its own rounding.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import _reference64 as r64

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
FP8 = {torch.float8_e4m3fn: (448.0, 2.0 ** -4, 2.0 ** -10), torch.float8_e5m2: (57344.0, 2.0 ** -3, 2.0 ** -17)}


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def rows(R, C, dtype, seed, offset=0.1, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((R, C), generator=g) * torch.exp(0.3 * torch.randn((R, 1), generator=g)) * scale + offset
    return x.to(dtype)


def vec(C, dtype, seed, centre):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(C, generator=g) * 0.2 + centre).to(dtype)


def on_gpu(t, ld=None, shift=0):
    """t [R, C] on the GPU with row stride ld, `shift` elements into its buffer."""
    if t is None or (ld is None and not shift):
        return None if t is None else t.cuda()
    R, C = t.shape
    ld = ld or C
    buf = torch.full((shift + R * ld + 8,), 7.0, dtype=t.dtype, device="cuda")
    v = buf[shift:shift + R * ld].view(R, ld)[:, :C]
    v.copy_(t)
    return v


def forward(R, C, *, x_dtype=BF16, y_dtype=None, p_dtype=F32, q_dtype=torch.float8_e4m3fn, gamma=True, beta=True,
            eps=1e-5, offset=0.1, scale=1.0, ldx=None, shift=0, return_y=True, seed=1):
    import fp8_scaled_gemm_gb300 as fm
    x = rows(R, C, x_dtype, seed, offset, scale)
    ga = vec(C, p_dtype, seed + 1, 1.0) if gamma else None
    be = vec(C, p_dtype, seed + 2, 0.0) if beta else None
    g64, b64 = (r64.f64(ga) if gamma else np.ones(C)), (r64.f64(be) if beta else np.zeros(C))
    d = lambda t: None if t is None else t.cuda()
    got = fm.fp8_layer_norm(on_gpu(x, ldx, shift), d(ga), d(be), eps, y_dtype=y_dtype, q_dtype=q_dtype,
                            return_y=return_y)
    want = r64.layer_norm(r64.f64(x), g64, b64, eps)
    tol = r64.layer_norm_tol(r64.f64(x), g64, b64, eps)
    if return_y:
        assert got[0].dtype == (y_dtype or x_dtype)
        r64.assert_close(got[0], want[0], tol[0], "y")
    else:
        assert got[0] is None
    r64.assert_close(got[1], want[1], tol[1], "mean")
    r64.assert_close(got[2], want[2], tol[2], "rstd")
    if q_dtype is not None:
        qmax, u, half = FP8[q_dtype]
        amax = np.abs(want[0]).max(axis=1)
        r64.assert_close(got[4], amax / qmax, (tol[0].max(axis=1) + 2.0 ** -22 * amax) / qmax, "q_scale")
        s = r64.f64(got[4])[:, None]
        back = r64.f64(got[3]) * s
        lim = u * np.abs(want[0]) * 1.001 + half * s + tol[0] * 1.1
        assert np.all(np.abs(back - want[0]) <= lim)
        # the largest value of each row takes the largest code
        assert np.all(np.abs(r64.f64(got[3])).max(axis=1)[amax > 0] == qmax)


WIDTHS = [1, 2, 7, 8, 24, 33, 64, 120, 255, 256, 264, 512, 520, 1000, 1024, 1032, 2048, 2056, 4095, 4096, 4104, 8192,
          8200, 8193, 16384, 16385, 16392, 20001, 32768, 32776, 33001, 40000, 65544, 70001]


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("x_dtype,y_dtype", [(BF16, BF16), (F32, BF16), (F32, F32), (F16, F16)])
def test_forward_widths(C, x_dtype, y_dtype):
    _need_gpu()
    forward(5, C, x_dtype=x_dtype, y_dtype=y_dtype)


@pytest.mark.parametrize("R", [1, 2, 3, 63, 64, 65, 1000])
@pytest.mark.parametrize("C", [16, 200, 201, 1024, 5000])
def test_forward_row_counts(R, C):
    _need_gpu()
    forward(R, C)


def test_forward_many_rows():
    _need_gpu()
    forward(40000, 24, q_dtype=torch.float8_e5m2)
    forward(20000, 33)
    forward(2001, 1001)
    forward(1500, 4999)


@pytest.mark.parametrize("p_dtype", [BF16, F16, F32])
@pytest.mark.parametrize("gamma,beta", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("C", [264, 265])
def test_forward_parameters(p_dtype, gamma, beta, C):
    _need_gpu()
    forward(9, C, p_dtype=p_dtype, gamma=gamma, beta=beta)


@pytest.mark.parametrize("q_dtype", [None, torch.float8_e4m3fn, torch.float8_e5m2])
@pytest.mark.parametrize("return_y", [True, False])
@pytest.mark.parametrize("C", [264, 265, 33000])
def test_forward_parts(q_dtype, return_y, C):
    _need_gpu()
    forward(6, C, q_dtype=q_dtype, return_y=return_y)


@pytest.mark.parametrize("C,ldx,shift", [(264, 272, 0), (264, 265, 0), (264, 264, 1), (263, 300, 3), (40000, 40008, 0)])
@pytest.mark.parametrize("x_dtype", [BF16, F32])
def test_forward_strides_and_alignment(C, ldx, shift, x_dtype):
    _need_gpu()
    forward(6, C, x_dtype=x_dtype, ldx=ldx, shift=shift)


@pytest.mark.parametrize("C", [64, 65, 1024, 8192, 40000])
def test_forward_large_offset(C):
    """A row offset 1000 times its spread: the variance is summed from centred values."""
    _need_gpu()
    forward(4, C, x_dtype=F32, offset=1000.0, eps=1e-6)


@pytest.mark.parametrize("C", [8, 9, 520, 8192, 40000])
def test_forward_constant_rows(C):
    """Equal elements: variance 0, y is beta, up to the fp32 mean's rounding."""
    _need_gpu()
    import fp8_scaled_gemm_gb300 as fm
    x = torch.full((3, C), 0.5, device="cuda")
    y, mean, rstd, q, s = fm.fp8_layer_norm(x, eps=1.0, q_dtype=torch.float8_e4m3fn)
    assert torch.equal(mean, torch.full((3,), 0.5, device="cuda"))
    assert torch.equal(rstd, torch.ones(3, device="cuda"))
    assert not y.any() and not q.view(torch.uint8).bitwise_and(0x7F).any() and not s.any()
    be = torch.linspace(-1, 1, C, device="cuda")
    y = fm.fp8_layer_norm(x, beta=be, eps=0.25)[0]
    assert torch.equal(y, be.expand(3, C))


@pytest.mark.parametrize("C", [8, 9, 520, 8192, 40000])
def test_forward_non_finite_rows_stay_alone(C):
    _need_gpu()
    import fp8_scaled_gemm_gb300 as fm
    x = rows(7, C, F32, 3)
    clean = [t.clone() for t in fm.fp8_layer_norm(x.cuda(), q_dtype=torch.float8_e4m3fn)]
    x[1, C // 2], x[3, 0], x[5, C - 1] = float("nan"), float("inf"), -float("inf")
    y, mean, rstd, q, s = fm.fp8_layer_norm(x.cuda(), q_dtype=torch.float8_e4m3fn)
    for r in (1, 3, 5):
        assert y[r].isnan().all() and rstd[r].isnan() and s[r].isnan()
        assert (q[r].view(torch.uint8) == 0x7F).all()
    for r in (0, 2, 4, 6):
        for a, b in zip(clean, (y, mean, rstd, q, s)):
            assert torch.equal(a[r:r + 1].view(torch.uint8), b[r:r + 1].view(torch.uint8))


def backward(R, C, *, x_dtype=BF16, dy_dtype=None, p_dtype=F32, gamma=True, residual=True, offset=0.1, ld=(None,) * 4,
             shift=0, in_place=False, params=True, seed=5):
    import fp8_scaled_gemm_gb300 as fm
    dy_dtype = dy_dtype or x_dtype
    x = rows(R, C, x_dtype, seed, offset)
    dy = rows(R, C, dy_dtype, seed + 1, 0.02, 0.5)
    res = rows(R, C, x_dtype, seed + 2, 0.0) if residual else None
    ga = vec(C, p_dtype, seed + 3, 1.0) if gamma else None
    g64 = r64.f64(ga) if gamma else np.ones(C)
    _, mean, rstd = r64.layer_norm(r64.f64(x), 1.0, 0.0, 1e-5)
    mean, rstd = torch.from_numpy(mean).float(), torch.from_numpy(rstd).float()
    rg = on_gpu(res, ld[2], shift)
    dx = rg if in_place else (None if ld[3] is None else on_gpu(torch.zeros((R, C), dtype=x_dtype), ld[3], shift))
    got = fm.fp8_layer_norm_grad(on_gpu(dy, ld[0], shift), on_gpu(x, ld[1], shift), None if ga is None else ga.cuda(),
                                 mean.cuda(), rstd.cuda(), residual_grad=rg, dx=dx, return_params=params)
    a = (r64.f64(dy), r64.f64(x), g64, r64.f64(mean), r64.f64(rstd))
    want, tol = list(r64.layer_norm_grad(*a)), list(r64.layer_norm_grad_tol(*a))
    if residual:
        want[0] = want[0] + r64.f64(res)
        tol[0] = tol[0] + 2.0 ** -23 * np.abs(want[0])
    r64.assert_close(got[0], want[0], tol[0], "dx")
    if params:
        r64.assert_close(got[1], want[1], tol[1], "dgamma")
        r64.assert_close(got[2], want[2], tol[2], "dbeta")
    else:
        assert got[1] is None and got[2] is None


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("x_dtype,dy_dtype", [(BF16, BF16), (F32, BF16), (F32, F32), (F16, F32)])
def test_backward_widths(C, x_dtype, dy_dtype):
    _need_gpu()
    backward(5, C, x_dtype=x_dtype, dy_dtype=dy_dtype)


@pytest.mark.parametrize("R", [1, 2, 3, 63, 64, 65, 1000])
@pytest.mark.parametrize("C", [16, 200, 201, 1024, 5000])
def test_backward_row_counts(R, C):
    _need_gpu()
    backward(R, C)


@pytest.mark.parametrize("C", [16392, 20000, 20001, 32768, 33000])
@pytest.mark.parametrize("x_dtype", [BF16, F32])
def test_wide_rows_many_turns(C, x_dtype):
    """Clusters that take several rows each, with and without codes."""
    _need_gpu()
    import fp8_scaled_gemm_gb300 as fm
    forward(500, C, x_dtype=x_dtype)
    forward(500, C, x_dtype=x_dtype, q_dtype=None)
    backward(500, C, x_dtype=x_dtype)
    backward(500, C // 2, x_dtype=x_dtype)
    assert fm.fp8mm_device_status() == 0


@pytest.mark.parametrize("R", [1, 2, 4, 5])
@pytest.mark.parametrize("C", [24, 255, 4096, 4097, 16384, 40000, 40001])
def test_backward_few_rows(R, C):
    _need_gpu()
    backward(R, C)
    backward(R, C, x_dtype=F32)


def test_backward_many_rows():
    _need_gpu()
    backward(40000, 24)
    backward(20000, 33)
    backward(3000, 520, x_dtype=F32)
    backward(700, 16392)
    backward(700, 16391)
    backward(301, 8195)
    backward(2001, 255)
    backward(2000, 1001)


@pytest.mark.parametrize("C", [264, 265, 40000])
@pytest.mark.parametrize("gamma,residual,params", [(1, 1, 0), (1, 0, 1), (0, 1, 1), (0, 0, 0)])
@pytest.mark.parametrize("p_dtype", [BF16, F32])
def test_backward_parts(C, gamma, residual, params, p_dtype):
    _need_gpu()
    backward(6, C, gamma=bool(gamma), residual=bool(residual), params=bool(params), p_dtype=p_dtype)


@pytest.mark.parametrize("C,ld,shift", [(264, (272, 280, 288, 296), 0), (264, (265, 264, 270, 271), 0),
                                        (264, (265, 265, 267, 269), 0), (264, (265, 265, 267, 269), 1),
                                        (1264, (1265, 1265, 1267, 1269), 0),
                                        (264, (264, 264, 264, 264), 1), (263, (263, 300, 301, 302), 3),
                                        (40000, (40008, 40000, 40016, 40000), 0)])
@pytest.mark.parametrize("x_dtype", [BF16, F32])
def test_backward_strides_and_alignment(C, ld, shift, x_dtype):
    _need_gpu()
    backward(6, C, x_dtype=x_dtype, ld=ld, shift=shift)


@pytest.mark.parametrize("C", [264, 265, 8192, 40000])
def test_backward_in_place_over_the_residual_gradient(C):
    _need_gpu()
    backward(9, C, in_place=True)


def test_backward_of_no_rows_and_repeatability():
    _need_gpu()
    import fp8_scaled_gemm_gb300 as fm
    e = torch.empty((0, 40), device="cuda")
    dx, dg, db = fm.fp8_layer_norm_grad(e, e, None, torch.empty(0, device="cuda"), torch.empty(0, device="cuda"))
    assert dx.shape == (0, 40) and not dg.any() and not db.any()
    y, mean, rstd = fm.fp8_layer_norm(e)
    assert y.shape == (0, 40) and mean.numel() == 0
    for C in (1000, 1001, 5001, 40000):
        x, dy = rows(700, C, BF16, 1).cuda(), rows(700, C, BF16, 2).cuda()
        y, mean, rstd = fm.fp8_layer_norm(x)
        first = fm.fp8_layer_norm_grad(dy, x, None, mean, rstd)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        again = fm.fp8_layer_norm_grad(dy, x, None, mean, rstd, stream=s)
        s.synchronize()
        for a, b in zip(first, again):
            assert torch.equal(a, b)


def test_backward_against_differences_of_the_forward_pass():
    """A directional difference of sum(y dy) through the fp32 forward kernel."""
    _need_gpu()
    import fp8_scaled_gemm_gb300 as fm
    R, C, h = 4, 256, 2.0 ** -5
    x, dy, v = (rows(R, C, F32, s, 0.0).cuda() for s in (1, 2, 3))
    ga, be = vec(C, F32, 4, 1.0).cuda(), vec(C, F32, 5, 0.0).cuda()
    _, mean, rstd = fm.fp8_layer_norm(x, ga, be)
    dx, dg, db = fm.fp8_layer_norm_grad(dy, x, ga, mean, rstd)

    def f(x_, ga_, be_):
        return (fm.fp8_layer_norm(x_, ga_, be_)[0].double() * dy.double()).sum(dim=1)
    # y moves by at most 2^-17 of its values (the forward bound), each row
    # sums C of them: the difference's noise is that over h; the third
    # derivative along v, |v / std| about 1, adds h^2 of the same size
    noise = (dy.abs().double().sum(dim=1) * 4 * 2.0 ** -17 / h).cpu()
    curve = (dy.abs().double() * v.abs().double()).sum(dim=1).cpu() * 4 * h * h
    d = ((f(x + h * v, ga, be) - f(x - h * v, ga, be)) / (2 * h)).cpu()
    assert ((d - (dx.double() * v.double()).sum(dim=1).cpu()).abs() < noise + curve).all()
    w = v[0]
    d = float(((f(x, ga + h * w, be) - f(x, ga - h * w, be)) / (2 * h)).sum())
    assert abs(d - float((dg.double() * w.double()).sum())) < float(noise.sum())
    d = float(((f(x, ga, be + h * w) - f(x, ga, be - h * w)) / (2 * h)).sum())
    assert abs(d - float((db.double() * w.double()).sum())) < float(noise.sum())


def test_stray_writes():
    """Bytes between rows and around every output stay."""
    _need_gpu()
    import fp8_scaled_gemm_gb300 as fm
    for C in (40, 41, 1024, 5001, 33000):
        R = 7
        x, dy = rows(R, C, BF16, 1).cuda(), rows(R, C, BF16, 2).cuda()
        buf = torch.full((R + 2, C + 24), 9.0, dtype=BF16, device="cuda")
        inner = buf[1:1 + R, 8:8 + C]
        keep = torch.ones_like(buf, dtype=torch.bool)
        keep[1:1 + R, 8:8 + C] = False
        _, mean, rstd = fm.fp8_layer_norm(x, y=inner)
        assert bool((buf[keep] == 9.0).all())
        buf.fill_(9.0)
        fm.fp8_layer_norm_grad(dy, x, None, mean, rstd, dx=inner)
        assert bool((buf[keep] == 9.0).all())


# Even widths that are not multiples of 8: pairs of 16-bit elements where rows
# start on 4 bytes, single elements where they do not.
EVEN = [2, 6, 90, 202, 258, 514, 1002, 1026, 4094, 4998, 8190, 8194, 9132, 16386, 20002]


@pytest.mark.parametrize("C", EVEN)
@pytest.mark.parametrize("x_dtype,y_dtype", [(BF16, None), (F16, F32), (F32, BF16)])
def test_forward_even_widths(C, x_dtype, y_dtype):
    _need_gpu()
    forward(300, C, x_dtype=x_dtype, y_dtype=y_dtype, p_dtype=F32 if y_dtype else BF16)
    forward(9, C, x_dtype=x_dtype, y_dtype=y_dtype, q_dtype=None, gamma=False)


@pytest.mark.parametrize("C", EVEN)
@pytest.mark.parametrize("x_dtype,dy_dtype", [(BF16, BF16), (F16, BF16), (BF16, F32)])
def test_backward_even_widths(C, x_dtype, dy_dtype):
    _need_gpu()
    backward(300, C, x_dtype=x_dtype, dy_dtype=dy_dtype)
    backward(9, C, x_dtype=x_dtype, dy_dtype=dy_dtype, p_dtype=BF16, residual=False)


@pytest.mark.parametrize("C,ld,shift", [(1002, (1002, 1004, 1006, 1008), 2), (1002, (1002, 1004, 1005, 1008), 0),
                                        (1002, (1002, 1002, 1002, 1002), 1), (1002, (1003, 1003, 1003, 1003), 0),
                                        (4998, (4998, 5000, 5002, 4998), 0), (9132, (9132, 9134, 9136, 9138), 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_even_widths_strides_and_alignment(C, ld, shift, in_place):
    _need_gpu()
    forward(60, C, ldx=ld[1], shift=shift)
    backward(60, C, ld=ld, shift=shift, in_place=in_place)

