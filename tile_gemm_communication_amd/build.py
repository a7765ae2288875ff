"""Build libfluxmi.so (HIP, gfx950 only) and the binding's module in-tree.

Every source under csrc/ is compiled by hipcc for gfx950 and linked into one
shared library next to this file, which the Python binding loads; it needs
hipcc alone.  _fluxmi.so (host code against torch's headers) checks tensors for
the binding and is built where torch is installed.  Packed
fp32 VALU ops are disabled for every device compile.  The compiler's
per-kernel register and scratch figures are kept in
_build/kernel_resources.json, which the CPU tests check.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import json
import os
import re
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfluxmi.so")
MODULE = os.path.join(HERE, "_fluxmi.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

CFLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-I", INCLUDE, "-I", CSRC,
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function", "-Wno-unused-variable",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")))


RESOURCES = os.path.join(BUILD_DIR, "kernel_resources.json")


def _resources(remarks: str) -> list:
    """Per-kernel register and scratch use from hipcc's resource remarks."""
    out, cur = [], None
    for line in remarks.splitlines():
        m = re.search(r"remark:\s+(Function Name|VGPRs|AGPRs|ScratchSize \[bytes/lane\]):\s*(\S+)", line)
        if not m:
            continue
        key, val = m.group(1), m.group(2)
        if key == "Function Name":
            cur = {"name": val}
            out.append(cur)
        elif cur is not None:
            cur[{"VGPRs": "vgpr", "AGPRs": "agpr"}.get(key, "scratch")] = int(val)
    return out


def _compile(src: str):
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = [HIPCC, *CFLAGS, "-Rpass-analysis=kernel-resource-usage", "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, _resources(r.stderr)


def _compile_module() -> str:
    """The host object of fm_python.cpp (torch and Python headers)."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    obj = os.path.join(BUILD_DIR, "fm_python.o")
    flags = [f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
             "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM", "-O2", "-std=c++17", "-fPIC", "-w"]
    dirs = [INCLUDE, sysconfig.get_paths()["include"], *cpp_extension.include_paths(),
            os.path.join(os.path.dirname(os.path.dirname(HIPCC)), "include")]
    cmd = ["g++", *flags, *[x for d in dirs for x in ("-I", d)], "-c",
           os.path.join(CSRC, "fm_python.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for fm_python.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_module(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = MODULE + ".tmp"
    cmd = ["g++", "-shared", "-fPIC", obj, "-o", tmp, "-L", HERE, "-l:libfluxmi.so",
           "-Wl,-rpath,$ORIGIN", "-L", libs, "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MODULE)


def build_library(ex: cf.Executor) -> None:
    """libfluxmi.so and the compiler's resource figures."""
    done = list(ex.map(_compile, sources()))
    with open(RESOURCES, "w") as f:
        json.dump([k for _, ks in done for k in ks], f, indent=0)
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *[o for o, _ in done], "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def have_torch() -> bool:
    return importlib.util.find_spec("torch") is not None


def build_module() -> None:
    """_fluxmi.so beside a library that is built."""
    _link_module(_compile_module())


def build(verbose: bool = True) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    jobs = min(len(sources()) + 1, int(os.environ.get("MAX_JOBS", "8")))
    with cf.ThreadPoolExecutor(max_workers=max(1, jobs)) as ex:
        module = ex.submit(_compile_module) if have_torch() else None
        build_library(ex)
        if module:
            _link_module(module.result())
        else:
            print("torch is not installed: _fluxmi.so, which the Python binding of the router, "
                  "norms, dropout, 4-bit and 8-bit products needs, is not built", file=sys.stderr)
    if verbose:
        print(f"built {LIB}", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    build()
