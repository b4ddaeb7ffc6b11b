"""In-tree build of libbsolve.so (and the arithmetic-throughput probe) with nvcc, and, where torch is
installed, of the row operators' Python module with g++.

Every translation unit is compiled for sm_103a only, in parallel, then linked into a
shared library next to this file. Nothing is installed into site-packages.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import re
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libbsolve.so")
PROBE_LIB = os.path.join(PKG, "libbsolve_probe.so")
ROWCALL = os.path.join(PKG, "_rowcall.so")  # the Python module, against torch's and Python's headers
ROWCALL_SOURCE = "rowcall.cpp"

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--fmad=false", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC]
LIB_SOURCES = ["api.cu", "lu_reg.cu", "lu_reg_f32_row.cu", "lu_reg_f32_col.cu", "lu_reg_f64_row.cu",
               "lu_reg_f64_col.cu", "lu_reg_il_f32_row.cu", "lu_reg_il_f32_col.cu", "lu_reg_il_f64_row.cu",
               "lu_reg_il_f64_col.cu", "lu_rows2.cu", "lu_cta.cu",
               "smem_solvers.cu", "chol_sys.cu", "chol_cluster.cu", "bdsv.cu", "bdmv.cu", "solve.cu",
               "solve_lane.cu", "api_rows.cu", "grec.cu", "grec_bwd.cu", "gnorm.cu",
               "gnorm_f32.cu", "gnorm_bf16.cu", "gnorm_f16.cu",
               "api_delta.cu", "gdelta_prep.cu", "gdelta.cu", "gdelta_step.cu", "gdelta_bwd.cu",
               "gdelta_grad.cu",
               "gnorm_q8_f32.cu", "gnorm_q8_bf16.cu", "gnorm_q8_f16.cu", "gemm_q8.cu"]
PROBE_SOURCES = ["fma_peak.cu"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libbsolve")
    return path


def _cuda() -> str:
    # the toolkit that nvcc belongs to
    return os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))


def _newest_input_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != ROWCALL_SOURCE]
    files.append(os.path.join(INCLUDE, "bsolve.h"))
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files if os.path.isfile(f))


def _torch():
    """(folder, version) of the torch that is installed, without importing it; None where it or the
    headers that the Python module needs are not there."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    base = os.path.dirname(spec.origin)
    headers = [os.path.join(base, "include", "ATen", "core", "Tensor.h"),
               os.path.join(sysconfig.get_paths()["include"], "Python.h")]
    if not all(os.path.exists(h) for h in headers):
        return None
    with open(os.path.join(base, "version.py")) as f:
        return base, re.search(r"^__version__.*= *['\"](.*)['\"]", f.read(), re.M).group(1)


def rowcall_target(torch_version: str) -> str:
    """What the Python module is compiled for: it reads tensors through inline accessors, by the
    object layout of this very torch."""
    return f"torch {torch_version}, {sysconfig.get_config_var('SOABI')}"


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    subprocess.check_call(cmd)
    return obj


def _build_rowcall(force: bool) -> None:
    found = _torch()
    if found is None:  # the C library needs neither; the Python functions say what is missing
        return
    torch_dir, version = found
    inputs = [os.path.join(CSRC, ROWCALL_SOURCE), os.path.join(INCLUDE, "bsolve.h"),
              os.path.abspath(__file__)]
    stamp, target = os.path.join(BUILD, "rowcall.target"), rowcall_target(version)
    if not force and os.path.exists(ROWCALL) and os.path.exists(stamp) and \
            os.path.getmtime(ROWCALL) >= max(os.path.getmtime(f) for f in inputs):
        with open(stamp) as f:
            if f.read() == target + torch_dir:
                return
    import torch
    base, libs = os.path.join(torch_dir, "include"), os.path.join(torch_dir, "lib")
    obj = os.path.join(BUILD, "rowcall.o")
    subprocess.check_call([
        "g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
        f'-DBSOLVE_ROWCALL_TARGET="{target}"', "-I", INCLUDE,
        "-I", sysconfig.get_paths()["include"], "-I", os.path.join(_cuda(), "include"),
        "-isystem", base,
        "-isystem", os.path.join(base, "torch", "csrc", "api", "include"),
        "-c", os.path.join(CSRC, ROWCALL_SOURCE), "-o", obj])
    tmp = ROWCALL + f".tmp{os.getpid()}"
    subprocess.check_call([
        "g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:" + os.path.basename(LIB),
        "-Wl,-rpath,$ORIGIN", "-L", libs, "-ltorch_python", "-ltorch_cpu", "-lc10",
        "-Wl,-rpath," + libs, "-L", os.path.join(_cuda(), "lib64"), "-lcudart"])
    os.replace(tmp, ROWCALL)
    with open(stamp, "w") as f:
        f.write(target + torch_dir)


def _link(objs: list[str], out: str) -> None:
    tmp = out + f".tmp{os.getpid()}"
    subprocess.check_call([nvcc(), *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs])
    os.replace(tmp, out)


def _build_library(verbose_ptxas: bool) -> None:
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    with cf.ThreadPoolExecutor(max_workers=len(LIB_SOURCES) + len(PROBE_SOURCES)) as ex:
        lib_objs = list(ex.map(lambda s: _compile(s, extra), LIB_SOURCES))
        probe_objs = list(ex.map(lambda s: _compile(s, extra), PROBE_SOURCES))
    _link(lib_objs, LIB)
    _link(probe_objs, PROBE_LIB)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile and link libbsolve.so and libbsolve_probe.so if stale, and _rowcall.so if it is stale or
    was compiled for another torch; returns the library's path."""
    os.makedirs(BUILD, exist_ok=True)
    newest = _newest_input_mtime()
    if force or any(
            (not os.path.exists(p)) or os.path.getmtime(p) < newest for p in (LIB, PROBE_LIB)):
        _build_library(verbose_ptxas)
    _build_rowcall(force)
    return LIB
