"""Products with the extended epilogue on several streams and threads at once:
the automatic choice passes no partial tiles through memory that another stream's
call uses."""
from __future__ import annotations

import os
import subprocess
import sys
import threading

import pytest
import torch

import fp8_scaled_gemm_gb300 as fm

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E4M3 = torch.float8_e4m3fn

# split-K, stream-K, split-K, neither
SHAPES = [(512, 2048, 14336), (3000, 5000, 4112), (256, 4096, 14336), (300, 1000, 512)]


def problem(M, N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    A = torch.randn((M, K), generator=g, device="cuda").to(E4M3)
    B = torch.randn((N, K), generator=g, device="cuda").to(E4M3).t()
    sa, sb = (torch.rand(n, generator=g, device="cuda") / K ** 0.5 for n in (M, N))
    return (A, B, sa, sb, 1), torch.randn((M, N), generator=g, device="cuda").bfloat16()


def both(p):
    mm, r = p
    return [fm.fp8_scaled_mm_epilogue(*mm, activation=fm.ACT_SILU, residual=r),
            fm.fp8_scaled_mm_act_grad(*mm, r, fm.ACT_GELU)]


def test_threads_with_streams_of_their_own():
    """The bits of one thread's calls, with other data in every thread."""
    threads = 4
    problems = [[problem(*s, seed=10 * t + i) for i, s in enumerate(SHAPES)] for t in range(threads)]
    want = [[both(p) for p in ps] for ps in problems]
    torch.cuda.synchronize()
    errors, start = [], threading.Barrier(threads)

    def work(t):
        try:
            s = torch.cuda.Stream()
            start.wait(timeout=60)
            with torch.cuda.stream(s):
                for turn in range(12):
                    got = {(i + turn + t) % len(SHAPES): None for i in range(len(SHAPES))}
                    for i in got:
                        got[i] = both(problems[t][i])
                    s.synchronize()
                    errors.extend((t, turn, SHAPES[i], k) for i in got for k in (0, 1)
                                  if not torch.equal(got[i][k], want[t][i][k]))
        except Exception as e:      # reported by the main thread
            errors.append(e)
    ts = [threading.Thread(target=work, args=(t,)) for t in range(threads)]
    for t in ts:
        t.start()
    for t in ts:
        t.join(timeout=120)
    assert not any(t.is_alive() for t in ts) and errors == [], errors[:5]
    assert fm.fp8mm_device_status() == 0, fm.fp8mm_last_error()


MANY = r"""
import sys
import torch
sys.path.insert(0, sys.argv[1])
import fp8_scaled_gemm_gb300 as fm
from tests.test_epilogue_streams_gpu import SHAPES, both, problem
p = problem(*SHAPES[0], seed=1)
want = both(p)
streams = [torch.cuda.Stream() for _ in range(24)]
torch.cuda.synchronize()
got = []
for s in streams:
    with torch.cuda.stream(s):
        got.append(both(p))
torch.cuda.synchronize()
assert fm.fp8mm_device_status() == 0, fm.fp8mm_last_error()
for g in got:
    for a, b in zip(g, want):
        # one rounding to bf16 apart, and the fp32 sums' order
        assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=2.0 ** -10)
"""


def test_more_streams_than_there_is_scratch_for():
    """Past 16 streams the kernels that need none are taken: the same sums in
    another order. (A process of its own: the workspaces stay.)"""
    r = subprocess.run([sys.executable, "-c", MANY, ROOT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


SCRIPT = r"""
import sys
import torch
sys.path.insert(0, sys.argv[2])
import fp8_scaled_gemm_gb300 as fm
from tests.test_epilogue_streams_gpu import both, problem
both(problem(300, 1000, 512, 0))
p = problem(512, 2048, 14336, 1)
if sys.argv[1] == "capture":
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = both(p)
    others = [torch.cuda.Stream() for _ in range(2)]
    for s in others:
        with torch.cuda.stream(s):
            g.replay()
        s.synchronize()
    for a, b in zip(got, both(p)):
        assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=2.0 ** -10)
else:
    both(p)
torch.cuda.synchronize()
assert fm.fp8mm_device_status() == 0
"""


@pytest.mark.parametrize("how,splits", [("eager", True), ("capture", False)])
def test_a_captured_call_takes_no_scratch(how, splits):
    """A graph can be replayed on any stream, beside calls on the one it was
    captured on."""
    r = subprocess.run([sys.executable, "-c", SCRIPT, how, ROOT], cwd=ROOT, env=dict(os.environ, FP8MM_LOG="1"),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    line = [ln for ln in r.stderr.splitlines() if ln.startswith("fp8mm: ") and "512x2048x14336" in ln][0]
    assert (" split=2 " in line) == splits, line


@pytest.mark.parametrize("M,N,K,variant,tile_n,split,stop", [(300, 520, 1024, fm.VARIANT_TILE, 128, 3, 1),
                                                             (2304, 2560, 1296, fm.VARIANT_PAIR, 256, -1, 0)])
def test_a_wait_that_runs_out_leaves_the_streams_workspace_usable(M, N, K, variant, tile_n, split, stop):
    """The status read clears the arrivals and flags of every stream's workspace."""
    mm, r = problem(M, N, K, seed=3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def call():
        with torch.cuda.stream(s):
            out = fm.fp8_scaled_mm_epilogue(*mm, activation=fm.ACT_GELU, residual=r, variant=variant, tile_n=tile_n,
                                            split_k=split)
        s.synchronize()
        return out
    want = call()
    assert fm.fp8mm_device_status(s) == 0
    fm.fp8mm_debug_inject(stop_after_kblocks=stop, wait_limit_cycles=1 << 22)
    try:
        call()
        status = fm.fp8mm_device_status(s)
    finally:
        fm.fp8mm_debug_inject(-1, 0)
    assert status == -7
    assert torch.equal(call(), want) and torch.equal(call(), want)
    assert fm.fp8mm_device_status(s) == 0
