"""Gradients of the cross entropy where rows' dloss differ by many powers of two:
a row's gradient is as exact as the row by itself has it."""
from __future__ import annotations

import pytest
import torch

import fp8_scaled_gemm_gb300 as fm
from tests._loss64 import E4M3, E5M2, Problem, assert_close, grad64

pytestmark = pytest.mark.gpu

F32 = torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    assert fm.fp8mm_device_status() == 0, fm.fp8mm_last_error()


def only(p, rows):
    """The problem of some rows of p."""
    q = Problem(1, 1, 16)
    q.M, q.N, q.K, q.mode, q.bias = int(rows.sum()), p.N, p.K, p.mode, p.bias
    q.A, q.Bt, q.B, q.sb = p.A[rows], p.Bt, p.B, p.sb
    q.sa = p.sa[rows] if p.mode else p.sa
    q.target, q.dloss = p.target[rows], p.dloss[rows]
    return q


# norms found within the gradient's kernel and by one of their own; K slices of da; in every form of scales and codes
@pytest.mark.parametrize("M,N,K,rowwise,a", [(60, 3000, 64, True, E4M3), (60, 3000, 64, False, E5M2), (40, 20000, 80, True, E5M2),
                                             (40, 20000, 80, False, E4M3), (300, 9000, 272, True, E4M3)])
@pytest.mark.parametrize("ratio", [2.0 ** -10, 1e-5, 1e-7, 1e-12, 1e-25])
def test_rows_of_small_dloss(M, N, K, rowwise, a, ratio):
    p = Problem(M, N, K, rowwise=rowwise, a=a, bias=F32, spread=1.0)
    small = torch.arange(M, device="cuda") % 3 == 1
    p.dloss = torch.where(small, p.dloss * ratio, p.dloss)
    p.dloss[::2] *= -1.0
    lse = fm.fp8_cross_entropy(*p.operands, p.target, bias=p.bias)[1]
    da, db, dbias = fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, p.dloss, bias=p.bias, out_dtype=F32, return_dbias=True)
    want, tol = grad64(p, lse)
    assert_close(db, want[1], tol[1], "db")
    assert_close(dbias, want[2], tol[2], "dbias")
    for rows in (small, ~small):
        # the bounds of a call with these rows only
        want, tol = grad64(only(p, rows), lse[rows])
        assert_close(da[rows], want[0], tol[0], "da")
    # without the others' gradients the same
    alone = fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, p.dloss, bias=p.bias, out_dtype=F32, return_db=False)[0]
    want, tol = grad64(only(p, small), lse[small])
    assert_close(alone[small], want[0], tol[0], "da alone")


def test_a_row_does_not_see_the_others_dloss():
    """da of a row has the same bits whatever the other rows' dloss, where its sums are of the same slices."""
    p = Problem(60, 3000, 64, ignored=0.0)
    lse = fm.fp8_cross_entropy(*p.operands, p.target)[1]
    want = fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, p.dloss, out_dtype=F32)[0]
    for factor in (2.0 ** 30, 3.0, 1e-20, 0.0):
        d = p.dloss.clone()
        d[20:] *= factor
        got = fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, d, out_dtype=F32)[0]
        # (equal up to the rounding of the sums' last factor)
        assert_close(got[:20], want[:20].double(), 2.0 ** -23 * want[:20].abs().double())


def test_rows_whose_gradient_counts_for_little_in_db():
    """db keeps a row's share where it is all there is in its columns: codes of 256 are exact down to 2^-32 (e5m2: 2^-30) of
    the largest scale times dloss."""
    for a, least in ((E4M3, 2.0 ** -32), (E5M2, 2.0 ** -30)):
        p = Problem(2, 64, 64, a=a, ignored=0.0, bias=F32, rowwise=False)
        p.A.copy_((torch.ones(2, 64, device="cuda") * 256).to(a))
        p.bias.fill_(-float("inf"))
        # two columns for each row: the others' probability is zero
        p.Bt.copy_(torch.zeros(64, 64, device="cuda").to(p.Bt.dtype))
        p.bias[:4] = 0.0
        p.Bt[0:2, :32] = torch.tensor(28.0, device="cuda").to(p.Bt.dtype)
        p.Bt[2:4, 32:] = torch.tensor(28.0, device="cuda").to(p.Bt.dtype)
        p.A.view(torch.uint8)[0, 32:] = 0
        p.A.view(torch.uint8)[1, :32] = 0
        p.sb.fill_(1.0)
        p.sa.fill_(1.0)
        p.target = torch.tensor([0, 2], device="cuda")
        p.dloss = torch.tensor([1.0, least], device="cuda")
        lse = fm.fp8_cross_entropy(*p.operands, p.target, bias=p.bias)[1]
        db = fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, p.dloss, bias=p.bias, out_dtype=F32)[1]
        # dz = -+ 1/2 dloss (lse is rounded to 2^-24 of 229376 + log 2: exp of its error is within 1/64)
        want = -0.5 * least * 256.0
        assert bool(((db[2, 32:] / want - 1).abs() < 1 / 32).all()) and bool(((db[3, 32:] / want + 1).abs() < 1 / 32).all())


def test_ignored_rows_weights_stay_out():
    """dloss, codes and scales of rows to be ignored do not enter the norms, da, db or dbias."""
    for M, N in ((60, 3000), (60, 20000), (9000, 70)):
        p = Problem(M, N, 64, bias=F32)
        lse = fm.fp8_cross_entropy(*p.operands, p.target, bias=p.bias)[1]
        want = fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, p.dloss, bias=p.bias, return_dbias=True)
        off = p.target == -100
        for d, scale in ((float("nan"), 1.0), (float("inf"), float("nan")), (1e30, 1e30), (0.0, 0.0)):
            p.dloss[off], p.sa[off] = d, scale
            got = fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, p.dloss, bias=p.bias, return_dbias=True)
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_an_infinite_or_nan_row_makes_db_nan():
    for M, N in ((40, 300), (40, 9000)):
        p = Problem(M, N, 64, ignored=0.0)
        lse = fm.fp8_cross_entropy(*p.operands, p.target)[1]
        for d, scale in ((float("inf"), 1.0), (float("nan"), 1.0), (1.0, float("inf")), (1.0, float("nan")), (0.0, float("inf"))):
            dloss, sa = p.dloss.clone(), p.sa.clone()
            dloss[5], sa[5] = d, scale
            db = fm.fp8_cross_entropy_grad(p.A, p.B, sa, p.sb, p.mode, p.target, lse, dloss)[1]
            assert bool(db.isnan().all())
