"""Build libmxq.so (and the matrix-core probe library) in-tree with hipcc
for gfx950, and the torch marshalling module with the host compiler.  The
libraries need neither torch nor a host compiler: without torch the module is
left out (Python callers need both), and an error in its build is raised once
they are written.

Usage: python -m fp8_quantized_linear_mxq_amd.build  (or build() from Python).
Objects go to _build/ at the repository root; the shared library is written
next to this file, where the binding loads it.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmxq.so")
PROBE_SRC = os.path.join(PKG, "probe", "mfma_probe.hip")
PROBE_LIB = os.path.join(PKG, "probe", "libmxq_probe.so")
SOURCES = ["api.cpp", "quantize.hip", "lowrank.hip", "gemm_mx.hip", "gemm_dq.hip", "gemm_dqp.hip",
           "mse.hip", "lowrank_split.hip", "quantize_i8.hip", "gemm_i8.hip", "gemm_few.hip",
           "qk_norm.hip"]
ARCH = "gfx950"
BINDING_SRC = os.path.join(CSRC, "torch_binding.cpp")
BINDING_LIB = os.path.join(PKG, "_torch_binding" + sysconfig.get_config_var("EXT_SUFFIX"))


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the HIP library cannot be built")


def _flags() -> list[str]:
    return [f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
            # packed fp32 VALU ops are kept out of every kernel
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-Wno-unused-command-line-argument",
            "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc(), *_flags(), "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _run(what: str, cmd: list, out: str) -> None:
    """Run the command that writes out.tmp, then move it into place."""
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(out + ".tmp", out)


def _build_binding() -> bool:
    """The Python module that marshals torch tensors (host code only); False
    without torch."""
    try:
        import torch
        from torch.utils import cpp_extension
    except ImportError:
        return False
    inc = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"], os.path.join(ROOT, "include")]
    _run("binding build",
         [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          *(f"-isystem{i}" for i in inc), BINDING_SRC,
          "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch_cpu",
          "-lc10", "-o", BINDING_LIB + ".tmp"], BINDING_LIB)
    return True


def build(verbose: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        binding = ex.submit(_build_binding)
        objs = list(ex.map(_compile, SOURCES))
        _run("link", [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", LIB + ".tmp"], LIB)
        # the matrix-core probes: a separate library, never loaded by the layer
        _run("probe build", [hipcc(), *_flags(), "-shared", PROBE_SRC, "-o", PROBE_LIB + ".tmp"], PROBE_LIB)
        made = [LIB, PROBE_LIB] + ([BINDING_LIB] if binding.result() else [])
    if verbose:
        print("built " + ", ".join(made))
    return LIB


if __name__ == "__main__":
    build()
    sys.exit(0)
