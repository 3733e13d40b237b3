"""Plain 64-bit formulas of the operators around the product, for the tests:
numpy only, on the CPU, nothing shared with the CUDA path."""
from __future__ import annotations

import math

import numpy as np
import torch

ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

# unit roundoff and half of the smallest step of each output type
ROUND = {torch.bfloat16: (2.0 ** -8, 2.0 ** -134), torch.float16: (2.0 ** -11, 2.0 ** -25),
         torch.float32: (2.0 ** -24, 2.0 ** -150), torch.float8_e4m3fn: (2.0 ** -4, 2.0 ** -10)}

# Error of the kernels' fp32 activations against the definition, relative to
# |z| (values) or to 1 (slopes). Value: |x| Phi(-|x|) carries at most 2e-6
# relative error near the origin (fit 1.3e-6, ex2 and rcp 2^-22 each) and
# less against |x| further out, where Phi(-|x|) < 1 falls; the logistic forms
# carry 2^-22 + 2^-23 and the roundings of the argument. Slope: the same
# errors times a factor of at most 2 (x s (1 - s) and x phi(x) are below 0.6).
ACT_ERR = 4e-6


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


_erf = np.vectorize(math.erf)
_erfc = np.vectorize(math.erfc)


def phi(x):
    return 0.5 * _erfc(-np.clip(x, -40, 40) / math.sqrt(2.0))


def logistic(x):
    x = np.clip(x, -700, 700)
    return 1.0 / (1.0 + np.exp(-x))


def act(z, name):
    """act(z) with its limits: inf -> inf, -inf -> 0, NaN -> NaN."""
    z = np.asarray(z, dtype=np.float64)
    x = np.clip(z, -1e30, 1e30)
    if name == "none":
        return z
    if name == "relu":
        y = np.where(x > 0, x, 0.0)
    elif name == "gelu":
        y = x * phi(x)
    elif name == "gelu_tanh":
        xc = np.clip(x, -50, 50)
        y = x * logistic(2 * math.sqrt(2 / math.pi) * (xc + 0.044715 * xc ** 3))
    else:
        y = x * logistic(x)
    y = np.where(z == np.inf, np.inf, np.where(z == -np.inf, 0.0, y))
    return np.where(np.isnan(z), np.nan, y)


def slope(z, name):
    z = np.asarray(z, dtype=np.float64)
    x = np.clip(z, -50, 50)
    if name == "none":
        return np.ones_like(z)
    if name == "relu":
        d = np.where(x > 0, 1.0, 0.0)
    elif name == "gelu":
        d = phi(x) + x * np.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    elif name == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        s = logistic(c * (x + 0.044715 * x ** 3))
        d = s + x * s * (1 - s) * c * (1 + 3 * 0.044715 * x ** 2)
    else:
        s = logistic(x)
        d = s * (1 + x * (1 - s))
    return np.where(np.isnan(z), np.nan, d)


def product(A, Bt, sa, sb, rowwise):
    """(acc * scales, sum of |a b| * scales) of codes A [M, K], Bt [N, K]."""
    a, b = f64(A), f64(Bt)
    s = (f64(sa)[:, None] * f64(sb)[None, :]) if rowwise else f64(sa)[0] * f64(sb)[0]
    return (a @ b.T) * s, (np.abs(a) @ np.abs(b).T) * s


def assert_close(got: torch.Tensor, want: np.ndarray, tol: np.ndarray, what=""):
    """|got - round(want)| within rounding of got's type plus tol; NaN and
    infinities in the same places."""
    u, tiny = ROUND[got.dtype]
    g = f64(got)
    assert g.shape == want.shape, (what, g.shape, want.shape)
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(g), np.isnan(want)), f"{what}: NaN in other places"
    inf = ~fin & ~np.isnan(want)
    assert np.array_equal(g[inf], want[inf]), f"{what}: infinities differ"
    tol = np.broadcast_to(np.asarray(tol, dtype=np.float64), want.shape)
    err = np.abs(g - want)[fin]
    lim = (u * (np.abs(want) + tol) + tol + tiny)[fin]
    bad = err > lim
    if bad.any():
        i = int(np.argmax(np.where(bad, err / np.maximum(lim, 1e-300), 0)))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off; worst {g[fin][i]} for {want[fin][i]} "
                             f"(error {err[i]:.3g}, allowed {lim[i]:.3g})")


# ------------------------------------------------------------ layer norm ---

def layer_norm(x, gamma, beta, eps):
    """(y, mean, rstd) of rows x in 64 bits."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(axis=1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(axis=1) + eps)
    return (x - mean[:, None]) * rstd[:, None] * gamma + beta, mean, rstd


def layer_norm_grad(dy, x, gamma, mean, rstd):
    """(dx, dgamma, dbeta) for given statistics."""
    h = (x - mean[:, None]) * rstd[:, None]
    w = dy * gamma
    dx = rstd[:, None] * (w - w.mean(axis=1, keepdims=True) - h * (w * h).mean(axis=1, keepdims=True))
    return dx, (dy * h).sum(axis=0), dy.sum(axis=0)


# A fp32 sum of n terms made of chains of at most 128 additions (per thread,
# then over lanes, warps and CTAs) is off by at most 128 x 2^-24 of the sum of
# the terms' magnitudes.
SUM_ERR = 2.0 ** -17


def layer_norm_tol(x, gamma, beta, eps):
    """Bounds of the fp32 kernels' error in (y, mean, rstd)."""
    y, mean, rstd = layer_norm(x, gamma, beta, eps)
    mean_tol = SUM_ERR * np.abs(x).mean(axis=1) + 2.0 ** -23 * np.abs(mean)
    h = (x - mean[:, None]) * rstd[:, None]
    # the variance: its own sum, the squared error of the mean (second order),
    # and 8 roundings; rstd takes half of its relative error
    rstd_rel = SUM_ERR + 2.0 ** -20 + (mean_tol * rstd) ** 2
    y_tol = np.abs(gamma) * (rstd[:, None] * mean_tol[:, None] + np.abs(h) * (rstd_rel[:, None] + 2.0 ** -21)) + \
        2.0 ** -22 * (np.abs(y) + np.abs(beta))
    return y_tol, mean_tol, rstd * rstd_rel


def layer_norm_grad_tol(dy, x, gamma, mean, rstd):
    """Bounds of the fp32 kernels' error in (dx, dgamma, dbeta)."""
    h = np.abs((x - mean[:, None]) * rstd[:, None])
    w = np.abs(dy * gamma)
    m1, m2 = w.mean(axis=1, keepdims=True), (w * h).mean(axis=1, keepdims=True)
    dx = rstd[:, None] * ((SUM_ERR + 2.0 ** -20) * (m1 + h * m2) + 2.0 ** -20 * w)
    return dx, (SUM_ERR + 2.0 ** -21) * (np.abs(dy) * h).sum(axis=0), SUM_ERR * np.abs(dy).sum(axis=0)
