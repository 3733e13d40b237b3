"""The product's extended epilogue on the GPU (activation, residual, stored
pre-activation; activation gradient) against 64-bit formulas, for every
kernel family and output type.

Tolerance beside the output's own rounding: the product's accumulation,
2^-20 of sum |a b| in scaled units (the bound of the plain product's tests),
through an activation whose slope stays below 1.13 (and is at least -0.13);
the fp32 activation's error; and one fp32 rounding of the sum with the
residual.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from fp8_scaled_gemm_gb300.inputs import make_inputs
from tests import _reference64 as r64

pytestmark = pytest.mark.gpu

AUTO, TILE, SWAP, PAIR, SWAPK, SWAPPAIR = 0, 1, 2, 3, 4, 5
AUX = {torch.bfloat16: torch.bfloat16, torch.float16: torch.float16, torch.float32: torch.float32,
       torch.float8_e4m3fn: torch.bfloat16}


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def problem(M, N, K, rowwise, seed, a_dtype="e4m3"):
    inp = make_inputs(M, N, K, int(rowwise), seed, a_dtype=a_dtype)
    # scales that bring z to a spread of about 1.5, over both ends of an activation
    gain = 1.5 / np.sqrt(K)
    return inp.a_q, inp.bt_q, inp.scale_a * gain, inp.scale_b


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def strided(t, ld, shift=0):
    """t [M, N] on the GPU with row stride ld, `shift` elements into its buffer."""
    M, N = t.shape
    buf = torch.full((shift + M * ld + 8,), 7.0, dtype=t.dtype, device="cuda")
    v = buf[shift:shift + M * ld].view(M, ld)[:, :N]
    v.copy_(t)
    return v


def forward(M, N, K, *, rowwise=True, act="gelu", bias=True, residual=True, preact=True, dtype=torch.bfloat16,
            a_dtype="e4m3", variant=AUTO, tile_n=0, split_k=0, ldr=None, ldp=None, ldo=None, shift=0, in_place=False,
            seed=3, rshift=0):
    import fp8_scaled_gemm_gb300 as fm
    A, Bt, sa, sb = problem(M, N, K, rowwise, seed, a_dtype)
    aux = AUX[dtype]
    b = randn((N,), aux, seed + 1, 0.3) if bias else None
    r = randn((M, N), aux, seed + 2, 1.5) if residual else None
    z, absum = r64.product(A, Bt, sa, sb, rowwise)
    if bias:
        z = z + r64.f64(b)[None, :]
    want = r64.act(z, act) + (r64.f64(r) if residual else 0.0)
    zt = 2.0 ** -20 * absum + 2.0 ** -23 * np.abs(z)
    tol = 1.13 * zt + r64.ACT_ERR * np.abs(z) + 2.0 ** -23 * np.abs(want)
    if dtype == torch.float8_e4m3fn:
        want = np.clip(want, -448, 448)

    d = lambda t: None if t is None else t.cuda()
    out = strided(torch.zeros((M, N)).to(dtype), ldo or N, shift) if (ldo or shift) else \
        torch.zeros((M, N), device="cuda").to(dtype)
    if in_place:
        out.copy_(r)
        rg = out
    else:
        rg = strided(r, ldr or N, shift + rshift) if residual else None
    pg = strided(torch.full((M, N), float("nan")).to(aux), ldp or N, shift) if preact else None
    ret = fm.fp8_scaled_mm_epilogue(A.cuda(), Bt.cuda().t(), sa.cuda(), sb.cuda(), int(rowwise), bias=d(b),
                                    activation=r64.ACTS[act], residual=rg, preact=pg, out=out, variant=variant,
                                    tile_n=tile_n, split_k=split_k)
    assert ret is out
    assert fm.fp8mm_device_status() == 0, fm.fp8mm_last_error()
    r64.assert_close(out, want, tol, "out")
    if preact:
        r64.assert_close(pg, z, zt, "preact")


FAMILIES = [
    # variant, tile_n, split, M, N, K: each with ragged edges in M and N
    (TILE, 128, 1, 200, 328, 400), (TILE, 128, 3, 200, 328, 1040), (TILE, 256, 1, 300, 600, 256),
    (TILE, 256, 1, 300, 600, 1040), (TILE, 256, 2, 130, 600, 1040),
    (SWAP, 16, 1, 13, 328, 400), (SWAP, 32, 1, 40, 328, 400), (SWAP, 64, 2, 50, 328, 1040),
    (SWAP, 128, 1, 100, 328, 400), (SWAP, 32, 3, 40, 328, 1040),
    (PAIR, 256, 1, 300, 600, 400), (PAIR, 128, 1, 300, 328, 400), (PAIR, 256, 2, 300, 600, 1040),
    (PAIR, 256, -1, 300, 2600, 4112),
    (SWAPK, 16, 2, 13, 328, 1040), (SWAPK, 32, 4, 40, 328, 1040), (SWAPK, 64, 8, 50, 328, 2064),
    (SWAPK, 128, 4, 100, 328, 1040), (SWAPPAIR, 32, 1, 40, 328, 400), (SWAPPAIR, 128, 1, 100, 600, 400),
]


@pytest.mark.parametrize("variant,tile_n,split,M,N,K", FAMILIES)
def test_forward_every_kernel_family(variant, tile_n, split, M, N, K):
    _need_gpu()
    forward(M, N, K, variant=variant, tile_n=tile_n, split_k=split)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn])
@pytest.mark.parametrize("M,N", [(7, 200), (200, 264)])
def test_forward_activations_and_types(act, dtype, M, N):
    _need_gpu()
    forward(M, N, 272, act=act, dtype=dtype, a_dtype="e5m2" if act == "silu" else "e4m3")


@pytest.mark.parametrize("bias,residual,preact", [(b, r, p) for b in (0, 1) for r in (0, 1) for p in (0, 1)])
@pytest.mark.parametrize("rowwise", [False, True])
def test_forward_parts(bias, residual, preact, rowwise):
    _need_gpu()
    forward(150, 200, 272, act="silu", bias=bool(bias), residual=bool(residual), preact=bool(preact), rowwise=rowwise)


@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 257, 16), (129, 1, 32), (2, 8, 144), (255, 511, 48),
                                   (257, 255, 16), (1, 4096, 4096), (129, 4099, 1040)])
def test_forward_edge_sizes(M, N, K):
    _need_gpu()
    forward(M, N, K, act="gelu_tanh")


@pytest.mark.parametrize("variant,tile_n,M", [(TILE, 128, 150), (TILE, 256, 150), (PAIR, 256, 300), (SWAP, 32, 40),
                                              (SWAPK, 32, 40), (SWAPPAIR, 32, 40)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,ldr,ldp,ldo,shift", [(201, None, None, None, 0), (200, 203, 211, 206, 0),
                                                 (200, 208, 216, 224, 0), (200, None, None, None, 1)])
def test_forward_strides_and_alignment(variant, tile_n, M, dtype, N, ldr, ldp, ldo, shift):
    """Odd widths, leading dimensions of their own, and bases off 16 bytes."""
    _need_gpu()
    forward(M, N, 272, act="relu", dtype=dtype, variant=variant, tile_n=tile_n, ldr=ldr, ldp=ldp, ldo=ldo,
            shift=shift if dtype == torch.float32 else 2 * shift)


@pytest.mark.parametrize("variant,tile_n,split,M,N", [(PAIR, 256, 1, 300, 600), (PAIR, 256, 2, 300, 600),
                                                      (TILE, 256, 1, 300, 605), (SWAP, 32, 1, 40, 328),
                                                      (SWAPK, 32, 4, 40, 328)])
def test_forward_in_place_residual(variant, tile_n, split, M, N):
    _need_gpu()
    forward(M, N, 1040, act="none", in_place=True, preact=False, variant=variant, tile_n=tile_n, split_k=split)


@pytest.mark.parametrize("M", [40, 300])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_forward_non_finite_values(M, act):
    """NaN and infinities arriving by the bias and by the residual."""
    _need_gpu()
    import fp8_scaled_gemm_gb300 as fm
    N, K = 72, 64
    A, Bt, sa, sb = problem(M, N, K, True, 5)
    b = torch.zeros(N, dtype=torch.bfloat16)
    b[3], b[10], b[20], b[30], b[31] = float("nan"), float("inf"), -float("inf"), 200.0, -200.0
    r = randn((M, N), torch.bfloat16, 6)
    r[:, 40], r[:, 41], r[1, 42] = float("inf"), -float("inf"), float("nan")
    z = r64.product(A, Bt, sa, sb, True)[0] + r64.f64(b)[None, :]
    want = r64.act(z, act) + r64.f64(r)
    out, pre = fm.fp8_scaled_mm_epilogue(A.cuda(), Bt.cuda().t(), sa.cuda(), sb.cuda(), 1, bias=b.cuda(),
                                         activation=r64.ACTS[act], residual=r.cuda(), return_preact=True)
    r64.assert_close(out, want, 1e-4, "out")
    r64.assert_close(pre, z, 1e-4, "preact")


def gradient(M, N, K, *, act="gelu", dtype=torch.bfloat16, rowwise=True, variant=AUTO, tile_n=0, split_k=0, ldz=None,
             seed=11, in_place=False, zshift=0):
    import fp8_scaled_gemm_gb300 as fm
    A, Bt, sa, sb = problem(M, N, K, rowwise, seed, "e5m2")
    z = randn((M, N), AUX[dtype], seed + 1, 2.0)
    acc, absum = r64.product(A, Bt, sa, sb, rowwise)
    d = r64.slope(r64.f64(z), act)
    want = acc * d
    tol = 1.13 * 2.0 ** -20 * absum + r64.ACT_ERR * np.abs(acc) + 2.0 ** -22 * np.abs(want)
    zg = strided(z, ldz or N, zshift)
    out = zg if in_place else None
    got = fm.fp8_scaled_mm_act_grad(A.cuda(), Bt.cuda().t(), sa.cuda(), sb.cuda(), int(rowwise), zg, r64.ACTS[act],
                                    out=out, out_dtype=dtype, variant=variant, tile_n=tile_n, split_k=split_k)
    assert fm.fp8mm_device_status() == 0, fm.fp8mm_last_error()
    if dtype == torch.float8_e4m3fn:
        want = np.clip(want, -448, 448)
    r64.assert_close(got, want, tol, "dz")


@pytest.mark.parametrize("variant,tile_n,split,M,N,K", FAMILIES)
def test_gradient_every_kernel_family(variant, tile_n, split, M, N, K):
    _need_gpu()
    gradient(M, N, K, act="silu", variant=variant, tile_n=tile_n, split_k=split)


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn])
@pytest.mark.parametrize("M,N,ldz", [(7, 203, None), (200, 264, 272), (200, 264, 265)])
def test_gradient_activations_and_types(act, dtype, M, N, ldz):
    _need_gpu()
    gradient(M, N, 272, act=act, dtype=dtype, ldz=ldz, rowwise=act != "relu")


@pytest.mark.parametrize("variant,tile_n,M", [(PAIR, 256, 300), (SWAP, 32, 40), (SWAPK, 32, 40)])
def test_gradient_in_place(variant, tile_n, M):
    _need_gpu()
    gradient(M, 328, 1040, variant=variant, tile_n=tile_n, in_place=True)


@pytest.mark.parametrize("M", [40, 300])
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_gradient_at_non_finite_z(M, act):
    """Slopes at infinities are the limits 0 and 1, at NaN NaN."""
    _need_gpu()
    import fp8_scaled_gemm_gb300 as fm
    N, K = 72, 64
    A, Bt, sa, sb = problem(M, N, K, True, 5)
    z = randn((M, N), torch.bfloat16, 6)
    z[:, 3], z[:, 4], z[:, 5], z[:, 6], z[:, 7] = float("nan"), float("inf"), -float("inf"), 0.0, 1e30
    want = r64.product(A, Bt, sa, sb, True)[0] * r64.slope(r64.f64(z), act)
    got = fm.fp8_scaled_mm_act_grad(A.cuda(), Bt.cuda().t(), sa.cuda(), sb.cuda(), 1, z.cuda(), r64.ACTS[act])
    r64.assert_close(got, want, 1e-4, "dz")


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_gradient_against_differences_of_the_forward_pass(act):
    """dz . v against a central difference of sum(act(z + h v)) through the
    forward entry: the forward pass adds h v as the bias of a zero product."""
    _need_gpu()
    import fp8_scaled_gemm_gb300 as fm
    M, N, K, h = 1, 512, 16, 2.0 ** -6
    zero = torch.zeros((M, K), device="cuda").to(torch.float8_e4m3fn)
    W = torch.zeros((N, K), device="cuda").to(torch.float8_e4m3fn)
    one = torch.ones(1, device="cuda")
    z = torch.linspace(-6, 6, N, device="cuda")

    def f(b):
        return fm.fp8_scaled_mm_epilogue(zero, W.t(), one, one, 0, bias=b.contiguous(), activation=r64.ACTS[act],
                                         out_dtype=torch.float32).double()
    diff = (f(z + h) - f(z - h)) / (2 * h)
    # A row of ones times B of ones / K gives acc = 1: the gradient is the slope
    A1 = torch.ones((M, K), device="cuda").to(torch.float8_e4m3fn)
    B1 = torch.ones((N, K), device="cuda").to(torch.float8_e4m3fn)
    got = fm.fp8_scaled_mm_act_grad(A1, B1.t(), one / K, one, 0, z.view(1, N), r64.ACTS[act]).double()
    # third derivatives stay below 2.5: h^2 / 6 of it; values' rounding 2^-21 over h
    assert (diff - got).abs().max().item() < 2.5 * h * h / 6 + 6 * 2.0 ** -20 / h


def test_stray_writes_around_preact_and_out():
    """Bytes between the rows of out and preact, and around them, stay."""
    _need_gpu()
    import fp8_scaled_gemm_gb300 as fm
    for (M, N, variant, tile_n) in [(300, 601, PAIR, 256), (300, 600, PAIR, 256), (150, 200, TILE, 128),
                                    (40, 203, SWAP, 32), (40, 203, SWAPK, 32), (40, 200, SWAPK, 32)]:
        A, Bt, sa, sb = problem(M, N, 272, True, 9)
        r = randn((M, N), torch.bfloat16, 1).cuda()
        bufs = [torch.full((M + 8, N + 24), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        out, pre = (b[4:4 + M, 8:8 + N] for b in bufs)
        fm.fp8_scaled_mm_epilogue(A.cuda(), Bt.cuda().t(), sa.cuda(), sb.cuda(), 1, activation=4, residual=r, out=out,
                                  preact=pre, variant=variant, tile_n=tile_n)
        assert fm.fp8mm_device_status() == 0
        for b in bufs:
            mask = torch.ones_like(b, dtype=torch.bool)
            mask[4:4 + M, 8:8 + N] = False
            assert bool((b[mask] == 9.0).all()), (M, N, variant)
            assert int((b[4:4 + M, 8:8 + N] == 9.0).sum()) < M * N // 50


def test_results_repeat_and_follow_the_callers_stream():
    """The same bits on every call, also on a stream of the caller's own that
    the inputs are made on."""
    _need_gpu()
    import fp8_scaled_gemm_gb300 as fm
    M, N, K = 300, 2600, 4112
    A, Bt, sa, sb = problem(M, N, K, True, 9)
    r = randn((M, N), torch.bfloat16, 1)
    outs = []
    for s in (torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.current_stream()):
        with torch.cuda.stream(s):
            t = [x.cuda() for x in (A, Bt, sa, sb, r)]
            outs.append(fm.fp8_scaled_mm_epilogue(t[0], t[1].t(), t[2], t[3], 1, activation=2, residual=t[4]))
        s.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# Matrices whose rows start between words, between 16-byte pieces, or both in
# turn, over several column blocks and tiles, the last ones cut.
UNALIGNED = [(TILE, 128, 300, 421, 272), (TILE, 256, 300, 803, 272), (TILE, 256, 300, 803, 1040),
             (PAIR, 256, 520, 803, 272), (PAIR, 128, 300, 421, 272), (PAIR, 256, 300, 2600, 4112)]


@pytest.mark.parametrize("variant,tile_n,M,N,K", UNALIGNED)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("pad,rshift", [(0, 0), (1, 0), (1, 1), (2, 1), (5, 3)])
def test_forward_unaligned_residual(variant, tile_n, M, N, K, dtype, pad, rshift):
    _need_gpu()
    split = -1 if K > 4000 else 0
    forward(M, N, K, act="silu", dtype=dtype, preact=pad != 2, ldr=N + pad, rshift=rshift, variant=variant,
            tile_n=tile_n, split_k=split)


@pytest.mark.parametrize("variant,tile_n,M,N,K", UNALIGNED)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_unaligned_in_place(variant, tile_n, M, N, K, dtype):
    _need_gpu()
    forward(M, N | 1, K, act="gelu", dtype=dtype, preact=False, in_place=True, variant=variant, tile_n=tile_n)
    gradient(M, N | 1, K, act="gelu", dtype=dtype, in_place=True, variant=variant, tile_n=tile_n)


@pytest.mark.parametrize("variant,tile_n,M,N,K", UNALIGNED)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,zshift", [(0, 1), (1, 0), (2, 1)])
def test_gradient_unaligned(variant, tile_n, M, N, K, dtype, pad, zshift):
    _need_gpu()
    gradient(M, N, K, act="silu", dtype=dtype, ldz=N + pad, zshift=zshift, variant=variant, tile_n=tile_n)
