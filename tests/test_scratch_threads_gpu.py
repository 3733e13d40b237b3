"""Split-K and stream-K products of several host threads: the device memory
they pass partial tiles through is not freed under a launch of another thread."""
from __future__ import annotations

import threading

import pytest
import torch

import fp8_scaled_gemm_gb300 as fm

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def problem(M, N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    A = torch.randn((M, K), generator=g, device="cuda").to(E4M3)
    B = torch.randn((N, K), generator=g, device="cuda").to(E4M3).t()
    sa, sb = (torch.rand(n, generator=g, device="cuda") / K ** 0.5 for n in (M, N))
    return A, B, sa, sb, 1


def in_threads(works):
    """Runs the functions at once; the exceptions they raised."""
    errors, start = [], threading.Barrier(len(works))

    def run(f):
        try:
            start.wait(timeout=60)
            f()
        except Exception as e:      # reported by the caller
            errors.append(e)
    threads = [threading.Thread(target=run, args=(f,)) for f in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=120)
    assert not any(t.is_alive() for t in threads)
    return errors


def test_growing_the_workspace_beside_launches_of_other_threads():
    """One stream, so the launches follow one another; every thread asks for
    larger workspaces in its own order."""
    shapes = [(128 * i, 128 * j, 1024) for i in (1, 2, 5, 9) for j in (3, 7)]
    problems = [problem(*s, seed=i) for i, s in enumerate(shapes)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())

    def products(order):
        with torch.cuda.stream(stream):
            return {i: [fm.fp8_scaled_mm_config(*problems[i], variant=fm.VARIANT_TILE, tile_n=128, split_k=s)
                        for s in (2, 3)] for i in order}
    n = len(shapes)
    got = [None] * 4

    def work(t):
        def f():
            for _ in range(5):
                got[t] = products([(i * (2 * t + 1) + t) % n for i in range(n)])
        return f
    assert in_threads([work(t) for t in range(4)]) == []
    want = products(range(n))
    torch.cuda.synchronize()
    assert fm.fp8mm_device_status() == 0, fm.fp8mm_last_error()
    for g in got:
        for i in range(n):
            for a, b in zip(g[i], want[i]):
                assert torch.equal(a, b), shapes[i]
