"""Build the sm_103a shared library ``libfp8mm.so`` in-tree with nvcc, and
the extension module that binds the MLP block's operators to PyTorch tensors
(``_fp8mm_torch.so``, host C++ only) with the host compiler.

The library statically links the CUDA runtime and reaches the driver's
tensor-map encoder through the runtime's driver entry-point query, so the
``.so`` has no link-time dependency on libcuda and loads on a host without a
GPU (useful for checking its exported symbols).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libfp8mm.so")
BINDING = "_fp8mm_torch"
BINDING_PATH = os.path.join(BUILD_DIR, BINDING + ".so")

SOURCES = ["fp8mm_epilogue.cu", "fp8mm_epilogue_swap.cu", "fp8mm_api.cu", "fp8mm_norm_grad.cu", "fp8mm_norm.cu", "fp8mm_actgrad.cu"]
GENCODE = "arch=compute_103a,code=sm_103a"


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put the CUDA toolkit on PATH)")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "fp8mm.h"))
    files.append(os.path.abspath(__file__))
    return files


def binding_abi() -> str:
    """What the extension module is bound to: PyTorch's C++ interface, which
    changes from version to version, and Python's."""
    import torch
    return f"{torch.__version__} {sysconfig.get_config_var('SOABI')}"


def binding_is_for() -> str:
    """The binding_abi() the module was built for; "" without a module."""
    try:
        with open(BINDING_PATH + ".abi") as f:
            return f.read() if os.path.exists(BINDING_PATH) else ""
    except OSError:
        return ""


def up_to_date() -> bool:
    if not (os.path.exists(LIB_PATH) and os.path.exists(BINDING_PATH)):
        return False
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(BINDING_PATH))
    return all(os.path.getmtime(f) <= t for f in _inputs()) and binding_is_for() == binding_abi()


def _binding_command(out: str) -> list:
    """The host compiler's command for the extension module. PyTorch's
    libraries are loaded by ``import torch`` before the module is."""
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    include = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            *[f for d in include for f in ("-isystem" if d != INCLUDE else "-I", d)],
            os.path.join(CSRC, "fp8mm_torch.cpp"), "-o", out, "-L", os.path.join(base, "lib"), "-lc10", "-lc10_cuda",
            "-ltorch_cpu", "-ltorch_python"]


def _start_binding(work: str):
    """(path, command, process) of the extension module's compilation; an
    exception in the process's place where it cannot start."""
    module, cmd = os.path.join(work, BINDING + ".so"), []
    try:
        cmd = _binding_command(module)
        return module, cmd, subprocess.Popen(cmd)
    except (ImportError, OSError) as e:     # no PyTorch, no host compiler
        return module, cmd, e


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds what is out of date. The library needs neither PyTorch nor
    Python's headers: it is built and put in place also where the extension
    module cannot be, and the module's failure is raised after that."""
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    flags = ["-gencode", GENCODE, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-cudart", "static",
             "-I", INCLUDE, "-I", CSRC]
    if verbose:
        flags.insert(0, "-Xptxas=-v")
    with tempfile.TemporaryDirectory(dir=BUILD_DIR) as work:
        # one compiler per translation unit, all at once, then the link
        module, module_cmd, binding = _start_binding(work)
        jobs = []
        for src in SOURCES:
            obj = os.path.join(work, src + ".o")
            cmd = [nvcc_path(), *flags, "-c", os.path.join(CSRC, src), "-o", obj]
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            jobs.append((obj, cmd, subprocess.Popen(cmd)))
        failed = [(p.returncode, cmd) for _, cmd, p in jobs if p.wait() != 0]
        module_rc = None if isinstance(binding, Exception) else binding.wait()
        if failed:
            raise subprocess.CalledProcessError(*failed[0])
        subprocess.run([nvcc_path(), *flags, "-shared", *[obj for obj, _, _ in jobs], "-o", tmp], check=True)
        if module_rc == 0:
            with open(module + ".abi", "w") as f:
                f.write(binding_abi())
            os.replace(module, BINDING_PATH)
            os.replace(module + ".abi", BINDING_PATH + ".abi")
        os.replace(tmp, LIB_PATH)
    if module_rc is None:
        raise RuntimeError(f"{LIB_PATH} is built; the extension module {BINDING} cannot be") from binding
    if module_rc != 0:
        raise subprocess.CalledProcessError(module_rc, module_cmd)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
