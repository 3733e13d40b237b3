"""The extended epilogue's kernel choice is its own: a tuned entry of the plain
product's shape does not replace it."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r"""
import sys
import torch
import fp8_scaled_gemm_gb300 as fm
M, N, K = (int(v) for v in sys.argv[4:])
p = torch.cuda.get_device_properties(0)
with open(sys.argv[1], "w") as f:      # swap, 16 columns
    f.write(f"{p.major} {p.minor} {p.multi_processor_count} 1 {M} {N} {K} 1 0 0 0 2 16 1 1.0\n")
if sys.argv[2] == "tuned":
    assert fm.fp8mm_autotune_load(sys.argv[1]) == 1
A = torch.randn((M, K), device="cuda").to(torch.float8_e4m3fn)
B = torch.randn((N, K), device="cuda").to(torch.float8_e4m3fn).t()
sa, sb = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
z = torch.randn((M, N), device="cuda").bfloat16()
calls = {"plain": lambda: fm.fp8_scaled_mm(A, B, sa, sb, 1),
         "epilogue": lambda: fm.fp8_scaled_mm_epilogue(A, B, sa, sb, 1, activation=fm.ACT_GELU, residual=z),
         "gradient": lambda: fm.fp8_scaled_mm_act_grad(A, B, sa, sb, 1, z, fm.ACT_GELU)}
calls[sys.argv[3]]()
torch.cuda.synchronize()
"""


def choice(path, table, call, shape=(256, 512, 512)):
    """The log line of one call: after the types, "<kernel> (<where the choice came from>)"."""
    env = dict(os.environ, FP8MM_LOG="1", PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", SCRIPT, str(path), table, call, *map(str, shape)], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    lines = [ln for ln in r.stderr.splitlines() if ln.startswith("fp8mm: ")]
    assert len(lines) == 1, r.stderr
    return lines[0].split(": ")[-1]


def test_a_tuned_entry_of_the_plain_product_is_not_the_epilogues(tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    path = tmp_path / "tuned.txt"
    assert choice(path, "tuned", "plain").startswith("swap tile_n=16 ")
    assert choice(path, "tuned", "plain").endswith("(tuned)")
    for call in ("epilogue", "gradient"):
        got = choice(path, "tuned", call)
        assert got == choice(path, "none", call) and got.endswith("(model)")


def test_the_log_names_the_epilogues_kernel(tmp_path):
    """The 256-wide tiles run 16 epilogue warps up to K = 512 for the plain
    product, up to 1024 for the extended epilogue."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    shape = (2560, 4096, 1024)
    plain = choice(tmp_path / "t", "none", "plain", shape)
    assert plain.startswith("tile tile_n=256 ") and "epilogue_warps=16" not in plain
    assert "epilogue_warps=16" in choice(tmp_path / "t", "none", "epilogue", shape)
