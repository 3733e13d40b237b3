"""The binding of the MLP block's operators: refusals of wrong tensors, given
outputs, errors of the C entries, and that nothing is kept."""
import gc
import sys

import pytest
import torch

import fp8_scaled_gemm_gb300 as fm

pytestmark = pytest.mark.gpu
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape, dtype=BF16):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)
    return dict(A=randn(20, 64, dtype=E4M3), B=randn(40, 64, dtype=E4M3).t(), sa=torch.rand(20, device="cuda"),
                sb=torch.rand(40, device="cuda"), x=randn(20, 40), dy=randn(20, 40), z=randn(20, 40),
                gamma=randn(40, dtype=F32), mean=randn(20, dtype=F32), rstd=torch.rand(20, device="cuda"))


def wrong(t):
    """Matrices that cannot stand in for t [M, N] bf16."""
    M, N = t.shape
    return [t[:, :-1], t[:-1], t.float(), t.cpu(), torch.zeros((N, M), dtype=t.dtype, device="cuda").t(),
            torch.zeros((M, 2 * N), dtype=t.dtype, device="cuda")[:, ::2], t[0], t[None]]


def test_products_refuse_wrong_matrices(ops):
    o = ops
    mm = (o["A"], o["B"], o["sa"], o["sb"], 1)
    for bad in wrong(o["z"]):
        for kw in (dict(residual=bad), dict(preact=bad)):
            with pytest.raises(ValueError):
                fm.fp8_scaled_mm_epilogue(*mm, **kw)
        with pytest.raises(ValueError):
            fm.fp8_scaled_mm_act_grad(*mm, bad, fm.ACT_GELU, out_dtype=BF16)
    for bad in wrong(o["z"]):
        if bad.dtype != F32:              # an fp32 output is a right one
            with pytest.raises(ValueError):
                fm.fp8_scaled_mm_epilogue(*mm, out=bad)
    for bias in (o["gamma"][:-1], o["gamma"], o["x"][:, 0], torch.zeros(40, dtype=BF16)):
        with pytest.raises(ValueError):
            fm.fp8_scaled_mm_epilogue(*mm, bias=bias)
    for dtype in (torch.float64, torch.int8, torch.float8_e5m2):
        with pytest.raises(ValueError):
            fm.fp8_scaled_mm_epilogue(*mm, out_dtype=dtype)
    with pytest.raises(TypeError):
        fm.fp8_scaled_mm_epilogue(*mm, out_dtype="bf16")


def test_row_operators_refuse_wrong_tensors(ops):
    o = ops
    x, dy, z, gamma, mean, rstd = (o[k] for k in ("x", "dy", "z", "gamma", "mean", "rstd"))
    for bad in wrong(x):
        with pytest.raises(ValueError):
            fm.fp8_act_grad(dy, bad, fm.ACT_SILU)
        with pytest.raises(ValueError):
            fm.fp8_act_grad(dy, z, fm.ACT_SILU, dz=bad)
        for kw in (dict(residual_grad=bad), dict(dx=bad)):
            with pytest.raises(ValueError):
                fm.fp8_layer_norm_grad(dy, x, gamma, mean, rstd, **kw)
        if bad.dtype != F32:
            with pytest.raises(ValueError):
                fm.fp8_layer_norm(x, gamma, y=bad)
            with pytest.raises(ValueError):
                fm.fp8_layer_norm_grad(bad, x, gamma, mean, rstd)
    for bad in (gamma[:-1], gamma.double(), gamma.cpu(), torch.zeros(80, device="cuda")[::2]):
        for call in (lambda: fm.fp8_layer_norm(x, bad), lambda: fm.fp8_layer_norm(x, None, bad),
                     lambda: fm.fp8_layer_norm_grad(dy, x, bad, mean, rstd),
                     lambda: fm.fp8_act_grad(dy, z, 1, dbias=bad)):
            with pytest.raises(ValueError):
                call()
    for bad in (mean[:-1], mean.bfloat16(), mean.cpu()):
        with pytest.raises(ValueError):
            fm.fp8_layer_norm_grad(dy, x, gamma, bad, rstd)
        with pytest.raises(ValueError):
            fm.fp8_layer_norm_grad(dy, x, gamma, mean, bad)
    for call in (lambda: fm.fp8_layer_norm(x, gamma, gamma.bfloat16()), lambda: fm.fp8_layer_norm(x, q_dtype=BF16),
                 lambda: fm.fp8_layer_norm(x, y_dtype=E4M3), lambda: fm.fp8_layer_norm(x, y=x.clone(), y_dtype=F32)):
        with pytest.raises(ValueError):
            call()


def test_errors_of_the_c_entries(ops):
    o = ops
    for call, status in ((lambda: fm.fp8_scaled_mm_epilogue(o["A"], o["B"], o["sa"], o["sb"], 1, activation=9), -4),
                         (lambda: fm.fp8_scaled_mm_act_grad(o["A"], o["B"], o["sa"], o["sb"], 1, o["z"], 0), -4),
                         (lambda: fm.fp8_act_grad(o["dy"], o["z"], 7), -4),
                         (lambda: fm.fp8_act_grad(o["dy"], None, fm.ACT_GELU), -1),
                         (lambda: fm.fp8_layer_norm(o["x"], eps=-1.0), -2),
                         (lambda: fm.fp8_layer_norm(o["x"], y=o["x"]), -4)):
        with pytest.raises(fm.Fp8mmError) as e:
            call()
        assert e.value.status == status


def test_given_outputs_come_back_and_nothing_is_kept(ops):
    o = ops
    mm = (o["A"], o["B"], o["sa"], o["sb"], 1)
    out, pre, dz, db, y, dx = (torch.empty_like(o["z"]), torch.empty_like(o["z"]), torch.empty_like(o["z"]),
                               torch.empty(40, device="cuda"), torch.empty_like(o["x"]), torch.empty_like(o["x"]))

    def calls():
        r = fm.fp8_scaled_mm_epilogue(*mm, out=out, preact=pre, activation=2, return_preact=True)
        assert r[0] is out and r[1] is pre
        assert fm.fp8_scaled_mm_epilogue(*mm, out=out, residual=o["z"]) is out
        assert fm.fp8_scaled_mm_act_grad(*mm, o["z"], 2, out=out) is out
        r = fm.fp8_act_grad(o["dy"], o["z"], 3, dz=dz, dbias=db)
        assert r[0] is dz and r[1] is db
        assert fm.fp8_act_grad(o["dy"], o["z"], 3, return_dz=False)[0] is None
        assert fm.fp8_layer_norm(o["x"], o["gamma"], y=y, q_dtype=E4M3)[0] is y
        assert fm.fp8_layer_norm(o["x"], return_y=False)[0] is None
        assert fm.fp8_layer_norm_grad(o["dy"], o["x"], None, o["mean"], o["rstd"], dx=dx, return_params=False)[0] is dx
        for bad in (lambda: fm.fp8_layer_norm(o["x"], y=o["x"][:1]), lambda: fm.fp8_act_grad(o["dy"], o["z"], 7)):
            with pytest.raises((ValueError, fm.Fp8mmError)):
                bad()
    calls()
    gc.collect()
    before = torch.cuda.memory_allocated(), [sys.getrefcount(t) for t in (out, pre, dz, db, y, dx, *o.values())]
    for _ in range(50):
        calls()
    gc.collect()
    assert before == (torch.cuda.memory_allocated(),
                      [sys.getrefcount(t) for t in (out, pre, dz, db, y, dx, *o.values())])


def test_new_outputs_on_the_callers_stream(ops):
    """Tensors made on a side stream are the allocator's for that stream, and
    the results are the current stream's."""
    o = ops
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    want = fm.fp8_scaled_mm_epilogue(o["A"], o["B"], o["sa"], o["sb"], 1, activation=2, residual=o["z"])
    norm = fm.fp8_layer_norm(o["x"], o["gamma"], q_dtype=E4M3)
    got = fm.fp8_scaled_mm_epilogue(o["A"], o["B"], o["sa"], o["sb"], 1, activation=2, residual=o["z"], stream=s)
    on = fm.fp8_layer_norm(o["x"], o["gamma"], q_dtype=E4M3, stream=s)
    with torch.cuda.stream(s):
        inside = fm.fp8_scaled_mm_epilogue(o["A"], o["B"], o["sa"], o["sb"], 1, activation=2, residual=o["z"])
    assert torch.cuda.current_stream() != s
    torch.cuda.synchronize()
    assert torch.equal(want, got) and torch.equal(want, inside)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(norm, on))


def test_threads_with_streams_of_their_own(ops):
    """Calls of several threads at once give the results of one."""
    import threading
    o = ops

    def once():
        r = [fm.fp8_scaled_mm_epilogue(o["A"], o["B"], o["sa"], o["sb"], 1, activation=2, residual=o["z"])]
        r += fm.fp8_act_grad(o["dy"], o["z"], fm.ACT_SILU)
        r += fm.fp8_layer_norm(o["x"], o["gamma"])
        r += fm.fp8_layer_norm_grad(o["dy"], o["x"], o["gamma"], o["mean"], o["rstd"])
        return r
    want = once()
    torch.cuda.synchronize()
    bad = []

    def work():
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(60):
                    got = once()
                s.synchronize()
            bad.extend(i for i, (a, b) in enumerate(zip(want, got)) if not torch.equal(a, b))
        except Exception as e:      # reported by the main thread
            bad.append(e)
    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=60)
    assert not any(t.is_alive() for t in threads) and not bad, bad

