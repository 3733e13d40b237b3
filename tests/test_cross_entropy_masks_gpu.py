"""Cross entropy where whole stretches of the vocabulary are ruled out by a finite
bias (a padded vocabulary, a range of special tokens), for any such value;
where rows are infinite up to the vocabulary's ragged end; and where ignored rows hold anything."""
from __future__ import annotations

import math

import pytest
import torch

import fp8_scaled_gemm_gb300 as fm
from tests._loss64 import E4M3, E5M2, IGNORE, Problem, assert_close, grad64, loss64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
VALUES = [-1e4, -1e6, -1e9, -1e10, -1e20, -1e30, -1e38, "lowest"]


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    assert fm.fp8mm_device_status() == 0, fm.fp8mm_last_error()


class Masked(Problem):
    """z far under its row's largest adds nothing to the row, whatever its error: exp(-200 + 100) is under 2^-144 of a term
    of 1, and the error of such a z, 2^-23 of it, is under half of its distance to the largest."""

    def logits(self):
        z, err = super().logits()
        return z, torch.where(z < z.amax(dim=1, keepdim=True) - 200.0, 0.0, err)


class Alike(Problem):
    """Every z is its bias: the product is under half a unit in the last place of it."""

    def logits(self):
        z = self.bias.double().expand(self.M, self.N)
        return z, torch.zeros_like(z)


def value(v, dtype):
    return torch.finfo(dtype).min if v == "lowest" else v


# the first columns of a unit, an epilogue warp's block, its whole share, a tile, the padded end; and all but a few
RANGES = [(0, 32), (0, 64), (32, 64), (64, 128), (0, 256), (256, 512), (839, 900), (1, 899)]


@pytest.mark.parametrize("v", VALUES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_masked_stretches(v, dtype):
    for at, to in RANGES:
        p = Masked(70, 900, 64, bias=dtype, ignored=0.1)
        p.bias[at:to] = value(v, dtype)
        inside = (p.target >= at) & (p.target < to)
        p.target = torch.where(inside, IGNORE, p.target)
        p.target[0] = 0 if at > 0 else 899
        loss, lse = fm.fp8_cross_entropy(*p.operands, p.target, bias=p.bias)
        want = loss64(p)
        assert_close(lse, want[1], want[3], f"lse, columns {at} to {to}")
        assert_close(loss, want[0], want[2], f"loss, columns {at} to {to}")
        got = fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, p.dloss, bias=p.bias, out_dtype=F32, return_dbias=True)
        want, tol = grad64(p, lse)
        for name, r, w, t in zip(("da", "db", "dbias"), got, want, tol):
            assert_close(r, w, t, f"{name}, columns {at} to {to}")
        assert not bool(got[2][at:to].any())


@pytest.mark.parametrize("v", VALUES)
@pytest.mark.parametrize("M,N,K", [(40, 300, 64), (300, 20000, 32)])
def test_every_column_at_one_finite_value(v, M, N, K):
    p = Alike(M, N, K, bias=F32)
    # (half of the lowest, so that the product does not leave the type's range)
    p.bias.fill_(value(v, F32) / (2 if v == "lowest" else 1))
    p.sa.mul_(2.0 ** -40)
    loss, lse = fm.fp8_cross_entropy(*p.operands, p.target, bias=p.bias)
    b = p.bias[:1].double().expand(M)
    # the sum's logarithm, and the rounding of its sum with the maximum
    assert_close(lse, b + math.log(N), 1e-5 + 2.0 ** -24 * b.abs(), "lse")
    want = torch.where(p.target == IGNORE, 0.0, math.log(N)).double()
    assert_close(loss, want, torch.full_like(want, 1e-5), "loss")
    got = fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, p.dloss, bias=p.bias, out_dtype=F32, return_dbias=True)
    want, tol = grad64(p, lse)
    for name, r, w, t in zip(("da", "db", "dbias"), got, want, tol):
        assert_close(r, w, t, name)


def test_large_logits_of_both_signs():
    """Rows whose largest z is far from zero, without a mask."""
    for shift in (1e5, -1e5, 3e6, 1e10, -1e10, 1e30):
        p = Alike(50, 700, 64, bias=F32)
        p.bias.fill_(shift)
        p.bias[::2] = shift * (1 - 2.0 ** -16)
        p.sa.mul_(2.0 ** -60)
        loss, lse = fm.fp8_cross_entropy(*p.operands, p.target, bias=p.bias)
        want = loss64(p)
        assert_close(lse, want[1], want[3], f"lse at {shift}")
        # (relative to the largest z: at 1e30 even 64 bits hold no logarithm beside it)
        z = p.logits()[0]
        top = z.amax(dim=1)
        zt = z.gather(1, p.target.clamp_min(0)[:, None])[:, 0]
        want = torch.where(p.target == IGNORE, 0.0, torch.logsumexp(z - top[:, None], dim=1) + (top - zt))
        # top - z is exact; a sum's relative error is that of loss64, 2.1e-5 at most
        assert_close(loss, want, 4e-5 + 2.0 ** -22 * want.abs(), f"loss at {shift}")


def test_an_ignored_rows_lse_does_not_change_others():
    p = Problem(64, 600, 64)
    p.target[5:9] = IGNORE
    p.target[9] = 3
    lse = fm.fp8_cross_entropy(*p.operands, p.target)[1]
    want = fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, p.dloss, return_dbias=True)
    for v in (-1e30, 1e10, math.inf, -math.inf, math.nan):
        lse[5:9] = v
        got = fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, p.dloss, return_dbias=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("N", [1, 31, 32, 33, 300, 320, 5000])
@pytest.mark.parametrize("how", ["code", "scale"])
def test_rows_of_minus_infinity_up_to_a_ragged_end(N, how):
    """Every z of a row is -inf: lse = -inf, whether the vocabulary ends inside a block of columns or not."""
    p = Problem(40, N, 64, a=E5M2, b=E4M3, ignored=0.0)
    # products of one sign
    p.A.view(torch.uint8).bitwise_and_(0x7F)
    p.A.view(torch.uint8)[p.A.view(torch.uint8) == 0] = 0x3C
    p.Bt.view(torch.uint8).bitwise_or_(0x80)
    p.Bt.view(torch.uint8)[p.Bt.view(torch.uint8) == 0x80] = 0xB8
    p.target[3] = IGNORE
    for row in (3, 7):
        if how == "code":
            p.A.view(torch.uint8)[row, 9] = 0x7C
        else:
            p.sa[row] = math.inf
    loss, lse = fm.fp8_cross_entropy(*p.operands, p.target)
    off = torch.zeros(40, dtype=torch.bool, device="cuda")
    off[3] = off[7] = True
    assert bool((lse[off] == -math.inf).all()) and bool(lse[~off].isfinite().all())
    assert float(loss[3]) == 0.0 and bool(loss[7].isnan()) and bool(loss[~off].isfinite().all())
