"""Tensors of different devices, or of another than the current one, are refused
before anything is launched. The devices are those of fake tensors, which have no
memory: no GPU."""
from __future__ import annotations

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import fp8_scaled_gemm_gb300 as fm
from fp8_scaled_gemm_gb300 import _build

E4M3, BF16, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32
M, N, K = 4, 16, 32


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def fakes(device):
    with FakeTensorMode():
        def t(*shape, dtype=BF16):
            return torch.empty(shape, dtype=dtype, device=device)
        return dict(A=t(M, K, dtype=E4M3), B=t(N, K, dtype=E4M3).t(), sa=t(M, dtype=F32), sb=t(N, dtype=F32), out=t(M, N),
                    bias=t(N), z=t(M, N), r=t(M, N), pre=t(M, N), dy=t(M, N), dz=t(M, N), dbias=t(N, dtype=F32), x=t(M, N),
                    gamma=t(N, dtype=F32), beta=t(N, dtype=F32), mean=t(M, dtype=F32), rstd=t(M, dtype=F32), y=t(M, N),
                    dx=t(M, N), q=t(M, N, dtype=E4M3), qs=t(M, dtype=F32), xb=t(M, K), wb=t(N, K).t())


# the tensors of each call, the first one first
CALLS = {
    "mm_epilogue": ("A B sa sb bias r pre out", lambda o: fm.fp8_scaled_mm_epilogue(
        o["A"], o["B"], o["sa"], o["sb"], 1, bias=o["bias"], residual=o["r"], preact=o["pre"], out=o["out"])),
    "mm_act_grad": ("A B sa sb z out", lambda o: fm.fp8_scaled_mm_act_grad(
        o["A"], o["B"], o["sa"], o["sb"], 1, o["z"], fm.ACT_GELU, out=o["out"])),
    "act_grad": ("dy z dz dbias", lambda o: fm.fp8_act_grad(o["dy"], o["z"], fm.ACT_GELU, dz=o["dz"], dbias=o["dbias"])),
    "layer_norm": ("x gamma beta y", lambda o: fm.fp8_layer_norm(o["x"], o["gamma"], o["beta"], y=o["y"])),
    "layer_norm_grad": ("dy x gamma mean rstd r dx", lambda o: fm.fp8_layer_norm_grad(
        o["dy"], o["x"], o["gamma"], o["mean"], o["rstd"], residual_grad=o["r"], dx=o["dx"])),
    "mm": ("A B sa sb bias out", lambda o: fm.fp8_scaled_mm(
        o["A"], o["B"], o["sa"], o["sb"], 1, bias=o["bias"], out=o["out"])),
    "mm_ex": ("A B sa sb bias out", lambda o: fm.fp8_scaled_mm_ex(
        o["A"], o["B"], o["sa"], o["sb"], 1, bias=o["bias"], out=o["out"])),
    "config": ("A B sa sb out", lambda o: fm.fp8_scaled_mm_config(o["A"], o["B"], o["sa"], o["sb"], 1, out=o["out"])),
    "noalloc": ("A B sa sb out", lambda o: fm.fp8_scaled_mm_noalloc(o["A"], o["B"], o["sa"], o["sb"], 1, out=o["out"])),
    "layout": ("A B sa sb bias out", lambda o: fm.fp8_scaled_mm_layout(
        o["A"], o["B"], o["sa"], o["sb"], 1, bias=o["bias"], out=o["out"])),
    "bmm": ("A B sa sb out", lambda o: fm.fp8_scaled_bmm(
        o["A"][None], o["B"][None], o["sa"], o["sb"], 1, out=o["out"][None])),
    "quantize": ("x q qs", lambda o: fm.fp8_quantize(o["x"], 1, out=o["q"], scale=o["qs"])),
    "mm_bf16": ("xb wb", lambda o: fm.fp8_scaled_mm_bf16(o["xb"], o["wb"], 1, out=o["out"])),
}
CASES = [(name, other) for name, (names, _) in CALLS.items() for other in names.split()[1:]]


@pytest.mark.parametrize("name,other", CASES)
def test_a_tensor_of_another_device_is_refused(name, other):
    with pytest.raises(ValueError, match="device"):
        CALLS[name][1](fakes("cuda:0") | {other: fakes("cuda:1")[other]})


@pytest.mark.parametrize("name", ["mm", "mm_ex", "config", "noalloc", "layout", "bmm", "quantize"])
def test_the_current_device_is_another_than_the_tensors(name, monkeypatch):
    """The entries that work on the current device only."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    with pytest.raises(ValueError, match="the current device is cuda:0"):
        CALLS[name][1](fakes("cuda:1"))


class StreamOfDevice1:
    device = torch.device("cuda:1")


@pytest.mark.parametrize("name", ["mm_epilogue", "mm_act_grad", "act_grad", "layer_norm", "layer_norm_grad"])
def test_a_stream_of_another_device_is_refused(name):
    o = fakes("cuda:0")
    s = StreamOfDevice1()
    calls = {
        "mm_epilogue": lambda: fm.fp8_scaled_mm_epilogue(o["A"], o["B"], o["sa"], o["sb"], 1, stream=s),
        "mm_act_grad": lambda: fm.fp8_scaled_mm_act_grad(o["A"], o["B"], o["sa"], o["sb"], 1, o["z"], 2, stream=s),
        "act_grad": lambda: fm.fp8_act_grad(o["dy"], o["z"], 2, stream=s),
        "layer_norm": lambda: fm.fp8_layer_norm(o["x"], stream=s),
        "layer_norm_grad": lambda: fm.fp8_layer_norm_grad(o["dy"], o["x"], None, o["mean"], o["rstd"], stream=s),
    }
    with pytest.raises(ValueError, match="the stream is of cuda:1"):
        calls[name]()
