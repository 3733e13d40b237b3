"""Layer norm and activation gradient without a GPU: refusals of the C
entries before any CUDA call, the binding's checks, and the reference
formulas' gradients against differences of their forward values."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import fp8_scaled_gemm_gb300 as fm
from fp8_scaled_gemm_gb300 import _build
from tests import _reference64 as r64

P = ctypes.c_void_p
AT = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fm.load()


def norm(lib, **kw):
    a = dict(x=AT, xt=0, ldx=0, ga=AT + 16, be=AT + 32, pt=2, eps=1e-5, y=AT + 64, yt=0, ldy=0, mean=AT + 128,
             rstd=AT + 256, q=AT + 512, qt=0, qs=AT + 1024, R=4, C=64) | kw
    p = {k: (P(v) if v else None) for k, v in a.items() if k in ("x", "ga", "be", "y", "mean", "rstd", "q", "qs")}
    return lib.fp8_layer_norm(p["x"], a["xt"], a["ldx"], p["ga"], p["be"], a["pt"], a["eps"], p["y"], a["yt"], a["ldy"],
                              p["mean"], p["rstd"], p["q"], a["qt"], p["qs"], a["R"], a["C"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(xt=3), -4), (dict(yt=-1), -4), (dict(pt=4), -4), (dict(qt=2), -4), (dict(R=-1), -2), (dict(C=-1), -2),
    (dict(eps=-1e-5), -2), (dict(eps=float("nan")), -2), (dict(eps=float("inf")), -2),
    (dict(R=1 << 30, C=1 << 30), -2), (dict(ldx=63), -2), (dict(ldx=-5), -2), (dict(ldy=1), -2), (dict(ldy=1 << 36), -2),
    (dict(x=AT + 1), -3), (dict(xt=2, x=AT + 2), -3), (dict(y=AT + 65), -3), (dict(ga=AT + 2), -3), (dict(be=AT + 1), -3),
    (dict(mean=AT + 2), -3), (dict(rstd=AT + 1), -3), (dict(qs=AT + 2), -3),
    (dict(x=None), -1), (dict(qs=None), -1), (dict(y=AT), -4), (dict(q=AT), -4), (dict(q=AT + 64), -4),
])
def test_layer_norm_refusals(lib, kw, code):
    assert norm(lib, **kw) == code


def test_empty_rows_are_a_noop(lib):
    assert norm(lib, R=0, x=None) == 0
    assert norm(lib, C=0) == 0


def norm_grad(lib, **kw):
    a = dict(dy=AT, dt=0, lddy=0, x=AT + 64, xt=0, ldx=0, ga=AT + 16, pt=2, mean=AT + 128, rstd=AT + 256, res=AT + 512,
             ldr=0, dx=AT + 768, ldd=0, dg=AT + 1024, db=AT + 2048, R=4, C=64, ws=AT + 4096, wb=1 << 40) | kw
    p = {k: (P(v) if v else None) for k, v in a.items()
         if k in ("dy", "x", "ga", "mean", "rstd", "res", "dx", "dg", "db", "ws")}
    return lib.fp8_layer_norm_grad(p["dy"], a["dt"], a["lddy"], p["x"], a["xt"], a["ldx"], p["ga"], a["pt"], p["mean"],
                                   p["rstd"], p["res"], a["ldr"], p["dx"], a["ldd"], p["dg"], p["db"], a["R"], a["C"],
                                   p["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=3), -4), (dict(xt=9), -4), (dict(pt=-1), -4), (dict(R=-1), -2), (dict(C=-2), -2), (dict(lddy=3), -2),
    (dict(ldx=63), -2), (dict(ldr=63), -2), (dict(ldd=-1), -2), (dict(dy=AT + 1), -3), (dict(x=AT + 65), -3),
    (dict(dg=AT + 1026), -3), (dict(mean=AT + 129), -3), (dict(ws=AT + 4097), -3), (dict(dg=None), -1), (dict(db=None), -1),
    (dict(dy=None), -1), (dict(x=None), -1), (dict(mean=None), -1), (dict(rstd=None), -1),
    (dict(dx=AT), -4), (dict(dx=AT + 64), -4), (dict(dx=AT + 512, ldd=72), -4),
])
def test_layer_norm_grad_refusals(lib, kw, code):
    assert norm_grad(lib, **kw) == code


@pytest.mark.parametrize("off", [4, 8, 12])
def test_layer_norm_grad_workspace_is_stored_to_in_16_bytes(lib, off):
    assert norm_grad(lib, ws=AT + 4096 + off) == -3


def test_empty_gradient_is_a_noop(lib):
    assert norm_grad(lib, C=0) == 0
    assert norm_grad(lib, R=0, dg=None, db=None) == 0
    assert lib.fp8_layer_norm_grad_workspace(-1, 4) == -2


def act_grad(lib, **kw):
    a = dict(dy=AT, ldy=0, z=AT + 64, ldz=0, t=0, act=2, dz=AT + 128, ldd=0, db=AT + 256, M=4, N=64, ws=AT + 512,
             wb=1 << 40) | kw
    p = {k: (P(v) if v else None) for k, v in a.items() if k in ("dy", "z", "dz", "db", "ws")}
    return lib.fp8_act_grad(p["dy"], a["ldy"], p["z"], a["ldz"], a["t"], a["act"], p["dz"], a["ldd"], p["db"], a["M"],
                            a["N"], p["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(t=3), -4), (dict(act=5), -4), (dict(act=-1), -4), (dict(M=-1), -2), (dict(N=-1), -2), (dict(N=1 << 31), -2),
    (dict(ldy=63), -2), (dict(ldz=1), -2), (dict(ldd=-1), -2), (dict(dy=AT + 1), -3), (dict(z=AT + 65), -3),
    (dict(dz=AT + 129), -3), (dict(db=AT + 258), -3), (dict(ws=AT + 513), -3), (dict(dy=None), -1), (dict(z=None), -1),
    (dict(dz=AT, ldd=72), -4), (dict(dz=AT + 64, ldd=72), -4),
])
def test_act_grad_refusals(lib, kw, code):
    assert act_grad(lib, **kw) == code


def test_act_grad_nothing_wanted_is_a_noop(lib):
    assert act_grad(lib, N=0) == 0
    assert act_grad(lib, dz=None, db=None) == 0
    assert act_grad(lib, M=0, db=None) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros((4, 8))
    for call in (lambda: fm.fp8_layer_norm(x), lambda: fm.fp8_act_grad(x, x, 1),
                 lambda: fm.fp8_layer_norm_grad(x, x, None, torch.zeros(4), torch.zeros(4))):
        with pytest.raises(ValueError):
            call()


def test_reference_slopes_against_differences():
    z = np.linspace(-8, 8, 4001) + 1e-3
    h = 1e-5
    for name in ("relu", "gelu", "gelu_tanh", "silu"):
        d = (r64.act(z + h, name) - r64.act(z - h, name)) / (2 * h)
        assert np.abs(d - r64.slope(z, name)).max() < 1e-9 / h * 1e-1, name


def test_reference_layer_norm_gradient_against_differences():
    rng = np.random.default_rng(0)
    x, dy, v = (rng.standard_normal((3, 40)) for _ in range(3))
    ga, be = 1 + 0.2 * rng.standard_normal(40), 0.1 * rng.standard_normal(40)
    h = 1e-6

    def loss(x_, ga_, be_):
        return (r64.layer_norm(x_, ga_, be_, 1e-5)[0] * dy).sum()
    _, mean, rstd = r64.layer_norm(x, ga, be, 1e-5)
    dx, dg, db = r64.layer_norm_grad(dy, x, ga, mean, rstd)
    w = v[0]
    for got, a, b in (((dx * v).sum(), (x + h * v, ga, be), (x - h * v, ga, be)),
                      ((dg * w).sum(), (x, ga + h * w, be), (x, ga - h * w, be)),
                      ((db * w).sum(), (x, ga, be + h * w), (x, ga, be - h * w))):
        assert abs((loss(*a) - loss(*b)) / (2 * h) - got) < 1e-6
