"""fp8_cross_entropy and fp8_cross_entropy_grad on the GPU against 64-bit
formulas, within the bounds that tests/_loss64.py derives."""
from __future__ import annotations

import math

import pytest
import torch

import fp8_scaled_gemm_gb300 as fm
from tests._loss64 import E4M3, E5M2, IGNORE, Problem, assert_close, grad64, loss64

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    assert fm.fp8mm_device_status() == 0, fm.fp8mm_last_error()


def check_loss(p, **kw):
    loss, lse = fm.fp8_cross_entropy(*p.operands, p.target, bias=p.bias, **kw)
    assert loss.dtype == lse.dtype == F32
    want = loss64(p)
    assert_close(lse, want[1], want[3], "lse")
    assert_close(loss, want[0], want[2], "loss")
    return loss, lse


def check_grad(p, out_dtype=BF16, dloss=None, parts=(True, True, True), **kw):
    lse = fm.fp8_cross_entropy(*p.operands, p.target, bias=p.bias)[1]
    got = fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, p.dloss if dloss is None else dloss, bias=p.bias,
                                    out_dtype=out_dtype, return_da=parts[0], return_db=parts[1], return_dbias=parts[2], **kw)
    want, tol = grad64(p, lse, dloss)
    for name, wanted, r, w, t in zip(("da", "db", "dbias"), parts, got, want, tol):
        if wanted:
            assert r.dtype == (F32 if name == "dbias" else out_dtype)
            assert_close(r, w, t, name)
        else:
            assert r is None
    return got


@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 1000, 64), (3, 127, 16), (31, 128, 32), (33, 129, 48), (128, 256, 128),
                                   (129, 257, 144), (255, 511, 512), (256, 512, 256), (257, 513, 272), (700, 2000, 400),
                                   (40, 40000, 80), (300, 30000, 64), (1024, 1100, 64), (1025, 300, 64), (90, 10000, 2064)])
@pytest.mark.parametrize("rowwise", [False, True])
def test_loss_sizes(M, N, K, rowwise):
    check_loss(Problem(M, N, K, rowwise=rowwise))


@pytest.mark.parametrize("a", [E4M3, E5M2])
@pytest.mark.parametrize("b", [E4M3, E5M2])
@pytest.mark.parametrize("bias", [None, BF16, F16, F32])
def test_loss_types(a, b, bias):
    check_loss(Problem(150, 700, 96, a=a, b=b, bias=bias))


def test_loss_of_sharp_rows():
    """Logits far apart: one column takes nearly all, and targets nearly none."""
    check_loss(Problem(200, 3001, 64, spread=60.0))


@pytest.mark.parametrize("lowest", [-math.inf, torch.finfo(BF16).min])
def test_masked_columns(lowest):
    p = Problem(70, 900, 64, bias=BF16, ignored=0.1)
    p.bias[torch.randperm(900, generator=torch.Generator().manual_seed(1))[:500].cuda()] = lowest
    p.target = torch.where(p.bias[p.target.clamp_min(0)] < -1e30, IGNORE, p.target)
    check_loss(p)
    check_grad(p)


def test_all_columns_masked():
    p = Problem(40, 300, 64, bias=F32)
    p.bias.fill_(-math.inf)
    loss, lse = fm.fp8_cross_entropy(*p.operands, p.target, bias=p.bias)
    assert torch.equal(lse, torch.full_like(lse, -math.inf))
    assert torch.equal(loss.isnan(), p.target != IGNORE) and bool((loss[p.target == IGNORE] == 0).all())
    # with the lowest finite value instead, the columns are alike
    p.bias.fill_(torch.finfo(F32).min / 2)
    p.sa.fill_(2.0 ** -30)
    loss, lse = fm.fp8_cross_entropy(*p.operands, p.target, bias=p.bias)
    want = torch.where(p.target == IGNORE, 0.0, math.log(300.0))
    assert torch.equal(lse, p.bias[:1].expand(40))
    assert_close(loss, want.double().cuda(), torch.full((40,), 1e-5, dtype=torch.float64, device="cuda"), "loss")


def test_infinities_and_nan_in_logits():
    p = Problem(64, 600, 64, bias=F32, ignored=0.0)
    p.bias[7] = math.inf
    loss, lse = fm.fp8_cross_entropy(*p.operands, p.target, bias=p.bias)
    assert bool(lse.isnan().all()) and bool(loss.isnan().all())
    p.bias[7] = math.nan
    loss, lse = fm.fp8_cross_entropy(*p.operands, p.target, bias=p.bias)
    assert bool(lse.isnan().all()) and bool(loss.isnan().all())
    # in one row only
    p.bias[7] = 0.0
    p.sa[5] = math.nan
    loss, lse = fm.fp8_cross_entropy(*p.operands, p.target, bias=p.bias)
    assert torch.equal(lse.isnan(), torch.arange(64, device="cuda") == 5) and torch.equal(loss.isnan(), lse.isnan())


@pytest.mark.parametrize("ignore", [IGNORE, -1, 5])
def test_ignore_index(ignore):
    p = Problem(90, 400, 64, ignored=0.0)
    p.target[::3] = ignore
    p.target[3::9] = ignore
    loss, lse = fm.fp8_cross_entropy(*p.operands, p.target, ignore_index=ignore)
    want = loss64(p, ignore)
    assert_close(loss, want[0], want[2], "loss")
    got = fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, p.dloss, ignore_index=ignore, return_dbias=True)
    w, tol = grad64(p, lse, ignore=ignore)
    for r, x, t in zip(got, w, tol):
        assert_close(r, x, t)


def test_every_row_ignored():
    p = Problem(50, 300, 64, ignored=2.0)
    loss, lse = fm.fp8_cross_entropy(*p.operands, p.target)
    assert not bool(loss.any())
    lse[3], p.dloss[4], p.dloss[5] = math.nan, math.inf, math.nan
    # (the last one: of a mean over no rows)
    for dloss in (p.dloss, p.dloss[5:6], p.dloss[5].expand(50)):
        for r in fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, dloss, return_dbias=True):
            assert not bool(r.any())


def test_target_out_of_range():
    p = Problem(50, 300, 64, ignored=0.0)
    for bad in (300, -1, 1 << 40, -(1 << 40)):
        p.target[17] = bad
        loss, lse = fm.fp8_cross_entropy(*p.operands, p.target)
        assert torch.equal(loss.isnan(), torch.arange(50, device="cuda") == 17) and bool(lse.isfinite().all())
        da, db, _ = fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, p.dloss)
        assert torch.equal(da.isnan().all(dim=1), torch.arange(50, device="cuda") == 17)
        assert torch.equal(da.isnan().any(dim=1), torch.arange(50, device="cuda") == 17)
        assert bool(db.isnan().all())


@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 1000, 64), (2, 130, 16), (31, 128, 32), (65, 63, 48), (128, 256, 128),
                                   (129, 257, 144), (257, 513, 272), (700, 2000, 400), (2100, 100, 64), (40, 20000, 80),
                                   (10, 3000, 1040), (300, 10000, 64), (1024, 500, 64), (1100, 2000, 528), (20, 20000, 16),
                                   (5000, 300, 304)])
@pytest.mark.parametrize("rowwise", [False, True])
def test_grad_sizes(M, N, K, rowwise):
    check_grad(Problem(M, N, K, rowwise=rowwise))


@pytest.mark.parametrize("a", [E4M3, E5M2])
@pytest.mark.parametrize("b", [E4M3, E5M2])
@pytest.mark.parametrize("out", [BF16, F16, F32])
def test_grad_types(a, b, out):
    check_grad(Problem(150, 700, 96, a=a, b=b, bias=F16), out)


@pytest.mark.parametrize("parts", [(True, False, False), (False, True, False), (False, False, True), (False, True, True),
                                   (False, False, False)])
def test_grad_parts(parts):
    check_grad(Problem(150, 700, 96, bias=F32), parts=parts)


def test_grad_of_sharp_rows():
    check_grad(Problem(200, 3001, 64, spread=60.0), F32)


def test_one_dloss_for_all_rows():
    p = Problem(70, 300, 64)
    one = torch.full((1,), 1.0 / 70, device="cuda")
    x = check_grad(p, dloss=one)
    for same in (one[0].expand(70), one.expand(70).contiguous(), one[0]):
        y = fm.fp8_cross_entropy_grad(*p.operands, p.target, fm.fp8_cross_entropy(*p.operands, p.target)[1], same,
                                      return_dbias=True)
        assert all(torch.equal(a, b) for a, b in zip(x, y))


def test_dloss_of_very_different_rows():
    """Zero, tiny, negative and large factors in one call."""
    p = Problem(300, 500, 64, ignored=0.0)
    p.dloss = torch.randn(300, device="cuda") * torch.logspace(-12, 3, 300, device="cuda")
    p.dloss[::7] = 0.0
    check_grad(p, F32)
    p.dloss.zero_()
    for r in check_grad(p, F32):
        assert not bool(r.any())


def test_scales_of_very_different_rows():
    p = Problem(300, 500, 64, spread=0.5)
    p.sb *= torch.logspace(-6, 1, 500, device="cuda")
    p.sa *= torch.logspace(1, -6, 300, device="cuda")
    check_grad(p, F32)
    p.sb[::3] = 0.0
    p.sa[1] = 0.0
    check_loss(p)
    check_grad(p, F32)


def test_given_outputs_and_streams():
    p = Problem(150, 700, 96, bias=BF16)
    lse = fm.fp8_cross_entropy(*p.operands, p.target, bias=p.bias)[1]
    want = fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, p.dloss, bias=p.bias)
    da, db = torch.empty(150, 96, dtype=BF16, device="cuda"), torch.empty(700, 96, dtype=BF16, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, p.dloss, bias=p.bias, da=da, db=db, stream=s)
    loss2, lse2 = fm.fp8_cross_entropy(*p.operands, p.target, bias=p.bias, stream=s)
    s.synchronize()
    assert got[0] is da and got[1] is db and torch.equal(da, want[0]) and torch.equal(db, want[1])
    assert torch.equal(lse, lse2)


def test_calls_repeat_and_do_not_meet_on_streams():
    problems = [Problem(700, 3000, 272, seed=i) for i in range(3)]

    def both(p):
        loss, lse = fm.fp8_cross_entropy(*p.operands, p.target)
        return (loss, lse) + fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, p.dloss, return_dbias=True)
    want = [both(p) for p in problems]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in problems]
    got = [[] for _ in problems]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(both(problems[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for i in range(3) for r in got[i] for x, y in zip(r, want[i]))


def test_captured_and_replayed():
    """A graph reads what the operands hold when it is replayed."""
    p, other = Problem(300, 2000, 272, seed=1), Problem(300, 2000, 272, seed=2)

    def both(p):
        loss, lse = fm.fp8_cross_entropy(*p.operands, p.target)
        return (loss, lse) + fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, p.dloss, return_dbias=True)
    want = [[t.clone() for t in both(x)] for x in (p, other)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both(p)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(p)
    for w in (want[0], want[1], want[1]):
        if w is want[1]:
            for name in ("A", "Bt", "sa", "sb", "target", "dloss"):
                getattr(p, name).copy_(getattr(other, name))
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, w))


def test_pieces_of_the_vocabulary():
    """Rows long enough that the vocabulary goes in several pieces, the last a short one."""
    # a piece is 2^29 / M columns, rounded down to 256: 32512 and less here
    p = Problem(16500, 33000, 16, ignored=0.1)
    assert fm.load().fp8_cross_entropy_grad_workspace(16500, 33000, 16, 1, 1, 1) < 16500 * 33000 * 2
    lse = fm.fp8_cross_entropy(*p.operands, p.target)[1]
    da, db, dbias = fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, p.dloss, out_dtype=F32, return_dbias=True)
    # sampled rows of da, and columns of db with all rows
    rows = torch.cat([torch.arange(0, 16500, 331), torch.arange(16490, 16500)]).cuda()
    cols = torch.cat([torch.arange(0, 33000, 700), torch.arange(16380, 16400), torch.arange(32990, 33000)]).cuda()
    for r, c in ((rows, torch.arange(33000, device="cuda")), (torch.arange(16500, device="cuda"), cols)):
        part = Problem(len(r), len(c), 16)
        part.A, part.sa, part.dloss = p.A[r], p.sa[r], p.dloss[r]
        part.Bt, part.sb = p.Bt[c], p.sb[c]
        t = p.target[r]
        where = torch.full((33000,), -1, dtype=torch.int64, device="cuda")
        where[c] = torch.arange(len(c), device="cuda")
        on = t != IGNORE
        # a target outside the columns taken: none of them is it, but the row counts
        part.target = torch.where(on, where[t.clamp_min(0)], IGNORE)
        if len(c) < 33000:
            outside = on & (part.target < 0)
            part.Bt = torch.cat([part.Bt, part.Bt[:1]])
            part.sb = torch.cat([part.sb, torch.zeros(1, device="cuda")])
            part.N += 1
            part.target = torch.where(outside, part.N - 1, part.target)
        want, tol = grad64(part, lse[r])
        if len(c) == 33000:
            assert_close(da[r], want[0], tol[0], "da")
        else:
            n = len(c)
            assert_close(db[c], want[1][:n], tol[1][:n], "db")
            assert_close(dbias[c], want[2][:n], tol[2][:n], "dbias")


def test_gradients_match_differences():
    """da, db and dbias against central differences of the 64-bit loss along random directions."""
    p = Problem(60, 200, 64, bias=F32, rowwise=False, ignored=0.2)
    lse = fm.fp8_cross_entropy(*p.operands, p.target, bias=p.bias)[1]
    da, db, dbias = fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, p.dloss, bias=p.bias, out_dtype=F32,
                                              return_dbias=True)
    a, w, b = p.A.double() * p.sa.double(), p.Bt.double() * p.sb.double(), p.bias.double()
    on = p.target != IGNORE

    def total(a, w, b):
        z = a @ w.t() + b
        loss = torch.logsumexp(z, dim=1) - z.gather(1, p.target.clamp_min(0)[:, None])[:, 0]
        return float((torch.where(on, loss, 0.0) * p.dloss.double()).sum())
    g = torch.Generator(device="cuda").manual_seed(4)
    for x, grad in ((0, da), (1, db), (2, dbias)):
        args = [a, w, b]
        d = torch.randn(args[x].shape, generator=g, device="cuda", dtype=torch.float64) * args[x].std()
        h = 1e-4
        lo, hi = list(args), list(args)
        lo[x], hi[x] = args[x] - h * d, args[x] + h * d
        diff = (total(*hi) - total(*lo)) / (2 * h)
        # the difference is off by h^2 times a third derivative of order one per row; the gradients by 2^-11 of each term
        size = float((grad.double().abs() * d.abs()).sum())
        assert abs(diff - float((grad.double() * d).sum())) < 3 * 2.0 ** -11 * size + 1e-6


@pytest.mark.parametrize("M,N,K", [(1, 33, 16), (33, 129, 48), (300, 1000, 272), (40, 20000, 80), (5000, 100, 64)])
@pytest.mark.parametrize("out", [BF16, F32])
def test_what_lies_around_the_outputs_stays(M, N, K, out):
    p = Problem(M, N, K)
    lse = fm.fp8_cross_entropy(*p.operands, p.target)[1]
    around = [torch.full((n + 8, K), 7.0, dtype=out, device="cuda") for n in (M, N)]
    fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, p.dloss, out_dtype=out, da=around[0][4:4 + M], db=around[1][4:4 + N])
    want, tol = grad64(p, lse)
    for a, n, w, t in zip(around, (M, N), want, tol):
        assert bool((a[:4] == 7).all()) and bool((a[4 + n:] == 7).all())
        assert_close(a[4:4 + n], w, t)


def test_codes_that_are_nan_or_infinite():
    p = Problem(40, 300, 64, b=E5M2, ignored=0.0)
    p.target[3] = IGNORE
    for code in (0x7C, 0x7E):           # infinity, NaN
        Bt = p.Bt.clone()
        Bt.view(torch.uint8)[17, 5] = code
        mm = (p.A, Bt.t(), p.sa, p.sb, p.mode)
        z = (p.A.double() @ Bt.double().t())[:, 17]
        loss, lse = fm.fp8_cross_entropy(*mm, p.target)
        # a column at minus infinity is left out, one at plus infinity or NaN makes the row NaN
        assert torch.equal(lse.isnan(), z.isnan() | (z == math.inf))
        da, db, _ = fm.fp8_cross_entropy_grad(*mm, p.target, lse, p.dloss)
        assert bool(da[p.target != IGNORE][:, 5].isnan().all()) and bool(db.isnan().any())
    A = p.A.clone()
    A.view(torch.uint8)[7, 3] = 0x7F
    mm = (A, p.B, p.sa, p.sb, p.mode)
    loss, lse = fm.fp8_cross_entropy(*mm, p.target)
    assert torch.equal(loss.isnan(), torch.arange(40, device="cuda") == 7) and torch.equal(lse.isnan(), loss.isnan())
    da, db, _ = fm.fp8_cross_entropy_grad(*mm, p.target, lse, p.dloss)
    assert torch.equal(da.isnan().any(dim=1), torch.arange(40, device="cuda") == 7) and bool(db.isnan().all())


@pytest.mark.parametrize("M,N,K,a", [(90, 300, 64, E4M3), (300, 9000, 272, E5M2), (1, 40, 16, E4M3), (9000, 70, 48, E4M3)])
@pytest.mark.parametrize("rowwise", [False, True])
def test_ignored_rows_may_hold_anything(M, N, K, a, rowwise):
    """NaN codes, scales, lse and dloss in the rows behind a batch's last one and between others."""
    p = Problem(M, N, K, a=a, bias=F32, rowwise=rowwise)
    p.target[M - M // 3 - 1:] = IGNORE
    want = check_grad(p)
    off = p.target == IGNORE
    p.A.view(torch.uint8)[off] = 0x7F
    if rowwise:
        p.sa[off] = torch.where(torch.arange(M, device="cuda")[off] % 2 == 0, math.nan, math.inf)
    p.dloss[off] = math.nan
    loss, lse = fm.fp8_cross_entropy(*p.operands, p.target, bias=p.bias)
    assert not bool(loss[off].any()) and bool(lse[off].isnan().all())
    got = fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, p.dloss, bias=p.bias, return_db=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and not bool(got[0][off].any())


def test_a_workspace_in_an_input_is_refused():
    p = Problem(40, 300, 64, bias=F32)
    lse = fm.fp8_cross_entropy(*p.operands, p.target, bias=p.bias)[1]
    da, lib = torch.empty(40, 64, dtype=BF16, device="cuda"), fm.load()
    need = lib.fp8_cross_entropy_grad_workspace(40, 300, 64, 1, 0, 0)
    memory = torch.zeros(need + 4096, dtype=torch.uint8, device="cuda")
    for at in (0, need - 256):
        A = memory[at:at + 40 * 64].view(E4M3)
        rc = lib.fp8_cross_entropy_grad(A.data_ptr(), 0, p.Bt.data_ptr(), 0, p.sa.data_ptr(), p.sb.data_ptr(), p.mode,
                                        p.bias.data_ptr(), 2, p.target.data_ptr(), IGNORE, lse.data_ptr(), p.dloss.data_ptr(),
                                        40, da.data_ptr(), None, 0, None, 40, 300, 64, memory.data_ptr(), need, None)
        assert rc == -4


def test_infinite_and_nan_dloss_or_scales_show():
    p = Problem(40, 300, 64, ignored=0.0)
    lse = fm.fp8_cross_entropy(*p.operands, p.target)[1]
    for bad in (math.inf, math.nan):
        d = p.dloss.clone()
        d[3] = bad
        da, db, _ = fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, d)
        assert bool(da[3].isnan().all()) and bool(db.isnan().all())
        for which in (2, 3):
            mm = list(p.operands)
            mm[which] = mm[which].clone()
            mm[which][5] = bad
            da, db, _ = fm.fp8_cross_entropy_grad(*mm, p.target, lse, p.dloss)
            assert bool(da.isnan().any()) and bool(db.isnan().any())


def test_large_vocabulary_and_one_row():
    p = Problem(1, 1000003, 16, ignored=0.0)
    check_loss(p)
    check_grad(p)


def test_no_rows():
    p = Problem(0, 300, 64)
    loss, lse = fm.fp8_cross_entropy(*p.operands, p.target)
    assert loss.shape == lse.shape == (0,)
    da, db, dbias = fm.fp8_cross_entropy_grad(*p.operands, p.target, lse, p.dloss, return_dbias=True)
    assert da.shape == (0, 64) and not bool(db.any()) and not bool(dbias.any())


def test_refusals():
    p = Problem(20, 40, 64, bias=F32)
    ok = dict(target=p.target, bias=p.bias)
    for kw in (dict(target=p.target.int()), dict(target=p.target[:-1]), dict(target=p.target.cpu()), dict(bias=p.bias[:-1]),
               dict(bias=p.bias.double()), dict(bias=p.bias.cpu())):
        with pytest.raises(ValueError):
            fm.fp8_cross_entropy(*p.operands, **{**ok, **kw})
    with pytest.raises(TypeError):
        fm.fp8_cross_entropy(*p.operands, None)
    with pytest.raises(ValueError):
        fm.fp8_cross_entropy(p.A.float(), p.B, p.sa, p.sb, 1, p.target)
    with pytest.raises(fm.Fp8mmError):
        fm.fp8_cross_entropy(p.A, torch.empty(0, 64, device="cuda").to(E4M3).t(), p.sa, p.sb[:0], 1, p.target)
    loss, lse = fm.fp8_cross_entropy(*p.operands, **ok)
    ok = dict(target=p.target, lse=lse, dloss=p.dloss)
    for kw in (dict(lse=lse[:-1]), dict(lse=lse.double()), dict(dloss=p.dloss[:-1]), dict(dloss=p.dloss.half()),
               dict(dloss=p.dloss.cpu()), dict(out_dtype=E4M3), dict(da=torch.empty(20, 64, device="cuda")),
               dict(da=torch.empty(64, 20, dtype=BF16, device="cuda").t()), dict(db=torch.empty(40, 48, dtype=BF16, device="cuda"))):
        with pytest.raises(ValueError):
            fm.fp8_cross_entropy_grad(*p.operands, **{**ok, **kw})
    # outputs start on 16 bytes
    off = torch.empty(20 * 64 + 1, dtype=BF16, device="cuda")[1:].view(20, 64)
    with pytest.raises(fm.Fp8mmError, match="ALIGN"):
        fm.fp8_cross_entropy_grad(*p.operands, **ok, da=off)
