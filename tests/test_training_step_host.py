"""Cross entropy and AdamW without a GPU: refusals of the C entries before any
CUDA call, workspace sizes, and that the binding refuses host tensors."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

import fp8_scaled_gemm_gb300 as fm
from fp8_scaled_gemm_gb300 import _build

P = ctypes.c_void_p
AT = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fm.load()


def p(v):
    return P(v) if v else None


def loss(lib, **kw):
    a = dict(A=AT + (1 << 14), at=0, B=AT + (1 << 15), bt=0, sa=AT, sb=AT + 16, mode=1, bias=AT + 272, bias_t=2, t=AT + 528, ignore=-100,
             loss=AT + 768, lse=AT + 1024, M=4, N=64, K=64, ws=AT + (1 << 20), wb=1 << 30) | kw
    return lib.fp8_cross_entropy(p(a["A"]), a["at"], p(a["B"]), a["bt"], p(a["sa"]), p(a["sb"]), a["mode"], p(a["bias"]),
                                 a["bias_t"], p(a["t"]), a["ignore"], p(a["loss"]), p(a["lse"]), a["M"], a["N"], a["K"],
                                 p(a["ws"]), a["wb"], None)


COMMON = [
    (dict(mode=2), -4), (dict(mode=-1), -4), (dict(at=2), -4), (dict(bt=-1), -4), (dict(bias_t=3), -4),
    (dict(M=-1), -2), (dict(N=0), -2), (dict(N=-1), -2), (dict(K=0), -2), (dict(K=8), -2), (dict(K=24), -2),
    (dict(K=(1 << 24) + 16), -2), (dict(M=1 << 31), -2), (dict(N=1 << 31), -2), (dict(M=1 << 20, N=1 << 21), -2),
    (dict(A=None), -1), (dict(B=None), -1), (dict(sa=None), -1), (dict(sb=None), -1), (dict(t=None), -1),
    (dict(A=AT + 8), -3), (dict(B=AT + 1), -3), (dict(sa=AT + 2), -3), (dict(sb=AT + 1), -3), (dict(bias=AT + 2), -3),
    (dict(bias=AT + 1, bias_t=0), -3), (dict(t=AT + 4), -3), (dict(lse=AT + 2), -3), (dict(ws=AT + 8), -3),
    (dict(lse=None), -1), (dict(ws=None), -1),
]


@pytest.mark.parametrize("kw,code", COMMON + [(dict(loss=None), -1), (dict(loss=AT + 2), -3), (dict(loss=AT + 1024), -4),
                                             (dict(lse=AT + 528), -4), (dict(loss=AT + (1 << 15) + 4092), -4), (dict(ws=AT), -4),
                                             (dict(N=(1 << 31) - 1000, M=1), -2), (dict(wb=4 * 4 * 8 - 1), -2)])
def test_loss_refusals(lib, kw, code):
    assert loss(lib, **kw) == code


def test_no_rows_is_a_noop(lib):
    assert loss(lib, M=0, A=None, t=None, ws=None, loss=None) == 0


def grad(lib, **kw):
    a = dict(A=AT + (1 << 14), at=0, B=AT + (1 << 15), bt=0, sa=AT, sb=AT + 16, mode=1, bias=AT + 272, bias_t=2, t=AT + 528, ignore=-100,
             lse=AT + 768, dl=AT + 1024, dn=4, da=AT + (1 << 16), db=AT + (1 << 17), ot=0, dbias=AT + (1 << 18), M=4, N=64,
             K=64, ws=AT + (1 << 20), wb=1 << 30) | kw
    return lib.fp8_cross_entropy_grad(p(a["A"]), a["at"], p(a["B"]), a["bt"], p(a["sa"]), p(a["sb"]), a["mode"], p(a["bias"]),
                                      a["bias_t"], p(a["t"]), a["ignore"], p(a["lse"]), p(a["dl"]), a["dn"], p(a["da"]),
                                      p(a["db"]), a["ot"], p(a["dbias"]), a["M"], a["N"], a["K"], p(a["ws"]), a["wb"], None)


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(ot=3), -4), (dict(ot=-1), -4), (dict(dn=3), -2), (dict(dn=0), -2), (dict(dn=5), -2), (dict(dl=None), -1),
    (dict(dl=AT + 2), -3), (dict(da=AT + 8), -3), (dict(db=AT + 2), -3), (dict(dbias=AT + 2), -3),
    (dict(db=AT + (1 << 16)), -4), (dict(da=AT + (1 << 17) + 8176), -4), (dict(db=AT + (1 << 15)), -4), (dict(dbias=AT + 768), -4),
    (dict(dbias=AT + (1 << 17)), -4), (dict(da=AT + (1 << 20)), -4), (dict(lse=AT + (1 << 16)), -4),
])
def test_grad_refusals(lib, kw, code):
    if "M" in kw:
        kw = kw | {"dn": 1}
    assert grad(lib, **kw) == code


def test_grad_of_nothing_is_a_noop(lib):
    assert grad(lib, da=None, db=None, dbias=None) == 0


def test_workspace_sizes(lib):
    assert lib.fp8_cross_entropy_workspace(0, 10) == 0
    assert lib.fp8_cross_entropy_workspace(1, 0) == -2 and lib.fp8_cross_entropy_workspace(-1, 5) == -2
    assert lib.fp8_cross_entropy_workspace(1 << 20, 1 << 21) == -2
    # 8 bytes for each row and 32 columns, 4 for each row; of many tiles a 64th of the logits in fp32 at most
    for M, N in ((1, 1), (7, 1000)):
        need = -(-N // 128) * M * 32 + M * 4
        assert need <= lib.fp8_cross_entropy_workspace(M, N) < need + 512
    for M, N in ((8192, 131072), (16384, 50257), (3000, 200001)):
        assert 0 < lib.fp8_cross_entropy_workspace(M, N) < M * N * 4 // 64
    assert lib.fp8_cross_entropy_grad_workspace(0, 10, 16, 1, 1, 1) == 0
    assert lib.fp8_cross_entropy_grad_workspace(5, 10, 16, 0, 0, 0) == 0
    for bad in ((-1, 10, 16), (5, 0, 16), (5, 10, 8), (5, 10, 24)):
        assert lib.fp8_cross_entropy_grad_workspace(*bad, 1, 1, 1) == -2


def tensor(**kw):
    a = dict(param=AT, grad=AT + (1 << 12), master=None, exp_avg=AT + (2 << 12), exp_avg_sq=AT + (3 << 12), exp_avg_scale=None,
             exp_avg_sq_scale=None, count=100) | kw
    return fm.AdamwTensor(*(a[k] for k, _ in fm.AdamwTensor._fields_))


def adamw(lib, tensors, n=None, **kw):
    a = dict(param_type=2, grad_type=2, state_bits=32, lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, step=1,
             lr_device=None, step_device=None, grad_scale=None) | kw
    options = fm.AdamwOptions(*(a[k] for k, _ in fm.AdamwOptions._fields_))
    array = (fm.AdamwTensor * max(1, len(tensors)))(*tensors)
    return lib.fp8_adamw(array, len(tensors) if n is None else n, ctypes.byref(options), None)


@pytest.mark.parametrize("kw,code", [
    (dict(param_type=3), -4), (dict(grad_type=-1), -4), (dict(state_bits=16), -4), (dict(state_bits=0), -4),
    (dict(n=-1), -2), (dict(n=1 << 61), -2), (dict(n=(1 << 63) - 1), -2), (dict(step=0), -2), (dict(step=-5), -2), (dict(lr=math.nan), -2), (dict(lr=math.inf), -2),
    (dict(beta1=1.0), -2), (dict(beta1=-0.5), -2), (dict(beta2=1.0), -2), (dict(beta2=math.nan), -2), (dict(eps=-1.0), -2),
    (dict(eps=math.nan), -2), (dict(weight_decay=math.inf), -2), (dict(lr_device=AT + 2), -3), (dict(step_device=AT + 4), -3),
    (dict(grad_scale=AT + 1), -3), (dict(state_bits=8), -1),
])
def test_adamw_refuses_options(lib, kw, code):
    assert adamw(lib, [tensor()], **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(count=-1), -2), (dict(count=1 << 41), -2), (dict(param=None), -1), (dict(grad=None), -1), (dict(exp_avg=None), -1),
    (dict(exp_avg_sq=None), -1), (dict(param=AT + 2), -3), (dict(grad=AT + 1), -3), (dict(master=AT + (9 << 12) + 2), -3),
    (dict(exp_avg=AT + 1), -3), (dict(exp_avg_sq=AT + 6), -3), (dict(exp_avg=AT), -4), (dict(exp_avg=AT + 396), -4),
    (dict(grad=AT + 396), -4), (dict(grad=AT), -4), (dict(master=AT), -4), (dict(exp_avg_sq=AT + (2 << 12) - 396), -4),
])
def test_adamw_refuses_a_tensor(lib, kw, code):
    assert adamw(lib, [tensor(**kw)]) == code


def test_adamw_refuses_tensors_together(lib):
    apart = dict(param=AT + (16 << 12), exp_avg=AT + (18 << 12), exp_avg_sq=AT + (19 << 12))
    assert adamw(lib, [tensor(), tensor()]) == -4
    assert adamw(lib, [tensor(), tensor(**{**apart, "param": AT + 396})]) == -4
    # a master for one of them only
    assert adamw(lib, [tensor(), tensor(**apart, master=AT + (20 << 12))]) == -4
    # scales of 8-bit states: one block here
    eight = dict(exp_avg_scale=AT + (4 << 12), exp_avg_sq_scale=AT + (5 << 12))
    assert adamw(lib, [tensor(**{**eight, "exp_avg_sq_scale": AT + (4 << 12)})], state_bits=8) == -4
    assert adamw(lib, [tensor(**{**eight, "exp_avg_scale": AT + 2})], state_bits=8) == -3


@pytest.mark.parametrize("what", ["lr_device", "step_device", "grad_scale"])
def test_adamw_refuses_options_in_what_it_writes(lib, what):
    assert adamw(lib, [tensor()], **{what: AT + 392}) == -4
    assert adamw(lib, [tensor()], **{what: AT + (2 << 12)}) == -4


def test_adamw_of_nothing_is_a_noop(lib):
    assert adamw(lib, []) == 0
    assert adamw(lib, [tensor(count=0, param=None, grad=None)]) == 0
    assert lib.fp8_adamw(None, 3, ctypes.byref(fm.AdamwOptions(2, 2, 32)), None) == -1
    assert lib.fp8_adamw(None, 0, None, None) == -1


def test_binding_refuses_host_tensors(lib):
    A, Bt = torch.zeros(4, 16).to(torch.float8_e4m3fn), torch.zeros(8, 16).to(torch.float8_e4m3fn)
    one, t = torch.ones(1), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        fm.fp8_cross_entropy(A, Bt.t(), one, one, 0, t)
    with pytest.raises(ValueError):
        fm.fp8_cross_entropy_grad(A, Bt.t(), one, one, 0, t, torch.zeros(4), one)
    x = [torch.zeros(4)]
    with pytest.raises(ValueError):
        fm.fp8_adamw(x, x, x, x, 1)
    fm.fp8_adamw([], [], [], [], 1)
