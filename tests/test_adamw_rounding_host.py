"""The rounding of fp8_adamw's 8-bit first moments: refusals of the C entry before
any CUDA call, and of the binding."""
from __future__ import annotations

import ctypes
import os
import re

import pytest

import fp8_scaled_gemm_gb300 as fm
from fp8_scaled_gemm_gb300 import _build

AT = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fm.load()


def stochastic():
    with open(os.path.join(_build.INCLUDE, "fp8mm.h")) as f:
        return int(re.search(r"#define FP8MM_STOCHASTIC_EXP_AVG (\d+)", f.read()).group(1))


@pytest.mark.parametrize("bits,code", [(8, -1), (32, -4), (16, -4), (0, -4), (40, -4)])
def test_it_goes_with_8_bits_only(lib, bits, code):
    t = fm.AdamwTensor(AT, AT + (1 << 12), None, AT + (2 << 12), AT + (3 << 12), None, None, 100)
    o = fm.AdamwOptions(2, 2, bits | stochastic(), 1e-3, 0.9, 0.99, 1e-8, 0.0, 1, None, None, None)
    # (8 bits without scales: what is missing is seen after the type of the states)
    assert lib.fp8_adamw(ctypes.byref(t), 1, ctypes.byref(o), None) == code


def test_the_binding_knows_its_names(lib):
    for name in ("up", "", 1, True):
        with pytest.raises(ValueError, match="exp_avg_rounding"):
            fm.fp8_adamw([], [], [], [], 1, exp_avg_rounding=name)
    for name in (None, "nearest", "stochastic"):
        fm.fp8_adamw([], [], [], [], 1, exp_avg_rounding=name)
