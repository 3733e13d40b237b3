"""The build without its compilers: stand-ins write the output files."""
from __future__ import annotations

import os
import stat
import subprocess

import pytest
import torch

import fp8_scaled_gemm_gb300 as fm
from fp8_scaled_gemm_gb300 import _build

COMPILER = """#!/bin/sh
# writes the file after -o; fails where the file STAND_IN_FAILS names occurs in the arguments
while [ $# -gt 0 ]; do
  if [ -n "$STAND_IN_FAILS" ]; then case "$1" in *"$STAND_IN_FAILS") exit 3;; esac; fi
  if [ "$1" = "-o" ]; then echo built > "$2"; exit 0; fi
  shift
done
"""


@pytest.fixture
def stand_ins(tmp_path, monkeypatch):
    """Compilers that only make their output files, and a build folder of its own."""
    cc = tmp_path / "cc"
    cc.write_text(COMPILER)
    cc.chmod(cc.stat().st_mode | stat.S_IXUSR)
    out = tmp_path / "build"
    monkeypatch.setattr(_build, "nvcc_path", lambda: str(cc))
    monkeypatch.setattr(_build, "BUILD_DIR", str(out))
    monkeypatch.setattr(_build, "LIB_PATH", str(out / "libfp8mm.so"))
    monkeypatch.setattr(_build, "BINDING_PATH", str(out / "_fp8mm_torch.so"))
    monkeypatch.setenv("CXX", str(cc))
    monkeypatch.delenv("STAND_IN_FAILS", raising=False)
    return out


def test_both_are_built(stand_ins):
    assert not _build.up_to_date()
    assert _build.build() == _build.LIB_PATH
    assert os.path.exists(_build.LIB_PATH) and os.path.exists(_build.BINDING_PATH) and _build.up_to_date()
    assert sorted(f for f in os.listdir(stand_ins) if f.endswith(".so")) == ["_fp8mm_torch.so", "libfp8mm.so"]


def no_compiler(monkeypatch):
    monkeypatch.setenv("CXX", "/nonexistent/compiler")


def no_torch(monkeypatch):
    def command(out):
        raise ImportError("No module named 'torch'")
    monkeypatch.setattr(_build, "_binding_command", command)


def no_headers(monkeypatch):
    monkeypatch.setattr(_build, "_binding_command", lambda out: ["/bin/false", "Python.h"])


@pytest.mark.parametrize("missing,error", [(no_compiler, RuntimeError), (no_torch, RuntimeError),
                                           (no_headers, subprocess.CalledProcessError)])
def test_the_library_is_built_where_the_module_cannot_be(stand_ins, monkeypatch, missing, error):
    missing(monkeypatch)
    with pytest.raises(error):
        _build.build()
    assert os.path.exists(_build.LIB_PATH) and not os.path.exists(_build.BINDING_PATH)
    assert not _build.up_to_date()      # the next build tries the module again


def test_a_failed_source_leaves_no_library(stand_ins, monkeypatch):
    monkeypatch.setenv("STAND_IN_FAILS", "fp8mm_norm.cu")
    with pytest.raises(subprocess.CalledProcessError):
        _build.build()
    assert not os.path.exists(_build.LIB_PATH)


def test_a_module_of_another_pytorch_is_stale(stand_ins, monkeypatch):
    _build.build()
    os.utime(_build.BINDING_PATH, (1e9, 1e9))
    assert not _build.up_to_date()
    _build.build()
    assert _build.up_to_date()
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    assert not _build.up_to_date()
    _build.build()
    assert _build.up_to_date()


def test_a_module_of_another_pytorch_is_not_loaded(monkeypatch):
    _build.build()
    monkeypatch.setattr(fm, "_native", None)
    monkeypatch.setattr(_build, "binding_abi", lambda: "0.0.1+other")
    with pytest.raises(RuntimeError, match="build it again"):
        fm._load_native()
