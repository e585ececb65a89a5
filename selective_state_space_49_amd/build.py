"""Build libssmscan.so (HIP kernels for gfx950 + the C ABI) and the _tensor_table extension in
the package directory.

    python -m selective_state_space_49_amd.build

Every HIP translation unit is compiled with floating-point contraction off (the
kernels write their fused multiply-adds explicitly) and with packed fp32 math
disabled. The library is placed next to this file so that it travels with the
source tree.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libssmscan.so")
TABLE = os.path.join(HERE, "_tensor_table.so")
OBJDIR = os.path.join(HERE, "_build")

ARCH = "gfx950"
HIP_SOURCES = ["scan_real.hip", "scan_complex.hip", "step.hip", "scan_bwd.hip", "scan_mimo.hip",
               "input_bwd.hip", "scratch.hip", "gated.hip", "xent.hip", "adamw.hip"]
CPP_SOURCES = ["api.cpp", "api_train.cpp"]
COMMON = ["-O3", "-fPIC", "-std=c++17", f"-I{INCLUDE}", f"-I{CSRC}"]
DEVICE = [f"--offload-arch={ARCH}", "-ffp-contract=off",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def _hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    path = os.path.join(rocm, "bin", "hipcc")
    return path if os.path.exists(path) else "hipcc"


def _compile(src: str, verbose: bool, objdir: str, defines) -> str:
    obj = os.path.join(objdir, os.path.basename(src) + ".o")
    cmd = [_hipcc(), *COMMON, *[f"-D{d}" for d in defines]]
    if src.endswith(".hip"):
        cmd += DEVICE
    cmd += ["-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling {src} failed:\n{r.stdout}\n{r.stderr}")
    return obj


def build_table(verbose: bool = False) -> str:
    """Compile the extension that reads torch tensors for short calls (host code only)."""
    import torch
    root = os.path.dirname(torch.__file__)
    tmp = TABLE + ".tmp"
    cmd = [_hipcc(), "-O2", "-fPIC", "-std=c++17", "-shared", "-w", f"-I{INCLUDE}", f"-I{root}/include",
           f"-I{root}/include/torch/csrc/api/include", f"-I{sysconfig.get_paths()['include']}",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           os.path.join(CSRC, "tensor_table.cpp"), "-o", tmp, f"-L{root}/lib", "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling tensor_table.cpp failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, TABLE)
    return TABLE


def build(verbose: bool = False, out: str = LIB, defines=()) -> str:
    """Compile every source, link libssmscan.so, and build the extension beside it; returns the
    library path.

    out and defines (NAME=VALUE strings, e.g. build-time tuning knobs) allow
    building variants elsewhere; the default is the package's own library.
    """
    objdir = OBJDIR if out == LIB else out + ".objs"
    os.makedirs(objdir, exist_ok=True)
    with ThreadPoolExecutor(max_workers=8) as ex:
        table = ex.submit(build_table, verbose) if out == LIB else None
        objs = list(ex.map(lambda s: _compile(s, verbose, objdir, defines), HIP_SOURCES + CPP_SOURCES))
        if table:
            table.result()
    tmp = out + ".tmp"
    cmd = [_hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking libssmscan.so failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
