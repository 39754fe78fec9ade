"""Builds libdet_gemm.so in-tree with nvcc for sm_103a (no GPU needed).

Each .cu file under csrc/ (det_gemm) and csrc_ops/ (the mixture-of-experts
operators) is compiled in parallel to an object under ``_build/`` and the
objects are linked into ``libdet_gemm.so`` next to this file. The CUDA runtime
is linked statically, so the library has no load-time dependency on libcuda
(the driver is reached at run time). The native half of _ops.py (binding/) is
built beside it as a Python extension against the installed PyTorch; where
there is no C++ compiler or a header is missing, the library is built alone and
the operators' Python functions say so when they are called.
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
CSRC_OPS = os.path.join(PKG, "csrc_ops")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libdet_gemm.so")
BINDING = os.path.join(PKG, "binding", "ops_native.cpp")
NATIVE = os.path.join(PKG, "_ops_native.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr",
              "-Xptxas", "-warn-spills"] + ARCH


def nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return cand


def sources() -> list[str]:
    return sorted(os.path.join(d, f) for d in (CSRC, CSRC_OPS) for f in os.listdir(d) if f.endswith(".cu"))


def headers() -> list[str]:
    hs = [os.path.join(d, f) for d in (CSRC, CSRC_OPS) for f in os.listdir(d) if f.endswith((".h", ".cuh"))]
    return hs + [os.path.join(INCLUDE, f) for f in ("det_gemm.h", "det_ops.h")]


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, verbose: bool, ptxas_info: bool) -> tuple[str, str]:
    obj = os.path.join(OBJDIR, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-I", CSRC_OPS, "-c", src, "-o", obj]
    if ptxas_info:
        cmd[1:1] = ["-Xptxas", "-v"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
    return obj, r.stdout + r.stderr


def _cxx() -> str:
    return os.environ.get("CXX", "g++")


def _torch_dir() -> str:
    import torch
    return os.path.dirname(torch.__file__)


def _binding_lacks() -> str:
    """What the binding cannot be built without and is not there ('' if nothing)."""
    if shutil.which(_cxx()) is None:
        return "the C++ compiler %s" % _cxx()
    for h in (os.path.join(sysconfig.get_paths()["include"], "Python.h"),
              os.path.join(_torch_dir(), "include", "torch", "csrc", "Exceptions.h")):
        if not os.path.exists(h):
            return h
    return ""


def _compile_binding(verbose: bool) -> str:
    """Compile the Python extension's object (g++, against PyTorch's headers)."""
    import torch
    inc = os.path.join(_torch_dir(), "include")
    obj = os.path.join(OBJDIR, "ops_native.o")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    cmd = [_cxx(), "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI), "-I", INCLUDE, "-I", inc,
           "-I", os.path.join(inc, "torch", "csrc", "api", "include"), "-I", os.path.join(cuda, "include"),
           "-I", sysconfig.get_paths()["include"], "-c", BINDING, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed for %s:\n%s\n%s" % (cmd[0], BINDING, r.stdout, r.stderr))
    return obj


def _link(cmd: list[str], target: str, verbose: bool) -> None:
    """Run a link command whose output goes to a temporary name, then put it in place."""
    tmp = target + ".tmp.%d" % os.getpid()
    cmd = [tmp if c is None else c for c in cmd]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, target)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile (if stale) and link libdet_gemm.so and, where it can be built, the
    binding; returns the library's path."""
    srcs = sources()
    stale = force or ptxas_info or _stale(LIB, srcs + headers())
    declared = [BINDING, os.path.join(INCLUDE, "det_ops.h"), os.path.join(INCLUDE, "det_gemm.h")]
    native = force or stale or _stale(NATIVE, declared)
    if native and _binding_lacks():
        print("the operators' Python binding is not built: no %s" % _binding_lacks(), file=sys.stderr)
        if os.path.exists(NATIVE) and _stale(NATIVE, declared):
            os.remove(NATIVE)                         # made for other declarations than the library's
        native = False
    if not stale and not native:
        return LIB
    os.makedirs(OBJDIR, exist_ok=True)
    logs, objs = [], []
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_compile_binding, verbose) if native else None
        for f in [ex.submit(_compile, s, verbose, ptxas_info) for s in srcs] if stale else []:
            o, log = f.result()
            objs.append(o)
            logs.append(log)
        if stale:
            _link([nvcc(), "-shared", *ARCH, "-o", None, *objs, "-lcudart_static", "-ldl", "-lpthread", "-lrt"], LIB, verbose)
        if native:
            tl = os.path.join(_torch_dir(), "lib")
            _link([_cxx(), "-shared", "-o", None, binding.result(), "-L", PKG, "-l:libdet_gemm.so",
                   "-L", tl, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-ltorch",
                   "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + tl], NATIVE, verbose)
    if ptxas_info:
        sys.stdout.write("".join(logs))
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
