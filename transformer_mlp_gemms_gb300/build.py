"""Build the in-tree shared library ``_build/libkt_mlp.so`` with nvcc for sm_103a, and the module
``_build/_kt_ops.so`` that hands torch tensors to it (g++, torch's headers).

Each translation unit is compiled in parallel, then linked with ``nvcc -shared``.
The CUDA runtime is linked statically; the driver's tensor-map encoder is looked
up at run time, so the library has no link-time dependency on libcuda.  The library comes first and
needs nothing else; the module is left out, with a line that says so, where this interpreter
has no torch or no headers, and is built anew for another torch or interpreter.

    python -m transformer_mlp_gemms_gb300.build [--force] [--verbose]
"""
from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libkt_mlp.so")
MODULE = os.path.join(BUILD, "_kt_ops.so")
MODULE_OBJ = os.path.join(BUILD, "kt_ops_py.cpp.o")
MODULE_STAMP = os.path.join(BUILD, "_kt_ops.for")  # the torch and interpreter that the module was built for
MODULE_SOURCE = os.path.join(CSRC, "kt_ops_py.cpp")
MODULE_DEPS = [MODULE_SOURCE, os.path.join(INCLUDE, "kt_mlp.h"), os.path.join(INCLUDE, "kt_ops.h")]

SOURCES = ["kt_gemm_act.cu", "kt_gemm_geglu.cu", "kt_gemm_down.cu", "kt_mlp_two_act_f16.cu", "kt_mlp_two_act_bf16.cu",
           "kt_mlp_two_geglu.cu", "kt_fused.cu", "kt_mlp_kernels.cu", "kt_mlp_abi.cpp", "kt_planner.cpp",
           "kt_ln_forward.cu", "kt_ln_backward.cu", "kt_quantize.cu", "kt_linear_i8.cu", "kt_moe.cu",
           "kt_ops_abi.cpp"]
HEADERS = [os.path.join(CSRC, "kt_internal.h"), os.path.join(CSRC, "kt_gemm.cuh"), os.path.join(INCLUDE, "kt_mlp.h"),
           os.path.join(CSRC, "kt_ops_internal.h"), os.path.join(CSRC, "kt_rows.cuh"), os.path.join(INCLUDE, "kt_ops.h")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build the library")


def _flags(src: str):
    common = ["-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]
    if src.endswith(".cu"):
        return ARCH + ["-lineinfo", "--expt-relaxed-constexpr"] + common
    return common


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _module_flags():
    """(compile, link) flags of the Python module: this interpreter's and this torch's headers and
    libraries.  None where they are not there."""
    import sysconfig

    python = sysconfig.get_paths()["include"]
    try:
        import torch
    except ImportError:
        return None
    if not os.path.exists(os.path.join(python, "Python.h")):
        return None
    home = os.path.dirname(os.path.abspath(torch.__file__))
    lib, inc = os.path.join(home, "lib"), os.path.join(home, "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    compile_ = ["-O2", "-std=c++17", "-fPIC", "-I", INCLUDE, "-I", python, "-isystem", inc,
                "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda,
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    link = ["-L", BUILD, "-l:libkt_mlp.so", "-L", lib, "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda",
            "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    return compile_, link


def _module_for() -> str:
    """What the module's binary interface depends on, as text."""
    import torch
    return f"python {sys.version} {sys.implementation.cache_tag}\ntorch {torch.__version__} {os.path.abspath(torch.__file__)}\n"


def _module_is_for(what: str) -> bool:
    try:
        with open(MODULE_STAMP) as f:
            return f.read() == what
    except OSError:
        return False


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    objs, procs = [], []
    for src in SOURCES:
        path = os.path.join(CSRC, src)
        obj = os.path.join(BUILD, src + ".o")
        objs.append(obj)
        if force or _stale(obj, [path] + HEADERS):
            cmd = [cc, "-c", path, "-o", obj] + _flags(src)
            if ptxas_info and src.endswith(".cu"):
                cmd += ["-Xptxas", "-v"]
            if verbose:
                print(" ".join(cmd), flush=True)
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    flags = _module_flags()
    module = None
    if flags is not None and (force or not _module_is_for(_module_for()) or _stale(MODULE_OBJ, MODULE_DEPS)):
        cmd = ["g++", "-c", MODULE_SOURCE, "-o", MODULE_OBJ] + flags[0]
        if verbose:
            print(" ".join(cmd), flush=True)
        module = subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0 or verbose or ptxas_info:
            sys.stdout.write(out)
        if p.returncode != 0:
            failed.append(src)
    if failed:
        raise RuntimeError(f"nvcc failed on {', '.join(failed)}")
    if force or procs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [cc, "-shared", "-o", tmp] + ARCH + objs + ["-lrt", "-lpthread", "-ldl"]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
    if flags is None:
        print(f"{os.path.basename(MODULE)} left out: no torch or no Python.h for this interpreter ({os.path.basename(LIB)} is complete)",
              flush=True)
        return LIB
    if module is not None:
        out, _ = module.communicate()
        if module.returncode != 0:
            raise RuntimeError(f"g++ failed on kt_ops_py.cpp:\n{out}")
    if module is not None or _stale(MODULE, [MODULE_OBJ]):
        tmp = MODULE + f".tmp{os.getpid()}"
        cmd = ["g++", "-shared", "-o", tmp, MODULE_OBJ] + flags[1]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        os.replace(tmp, MODULE)
        with open(MODULE_STAMP, "w") as f:
            f.write(_module_for())
    return LIB


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print -Xptxas -v register / smem usage")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose, ptxas_info=a.ptxas_info))


if __name__ == "__main__":
    main()
