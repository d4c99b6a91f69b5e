"""In-tree build of libokls.so (sm_103a) with nvcc, and of the torch binding of
its language-model operators (_lm_native.so) with the host compiler.

Each translation unit is compiled in parallel, then linked into shared
libraries next to this file.  Used by ``__graft_entry__.build()`` and by the
Python binding when the library is missing and a build is requested.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libokls.so")
SOURCES = ["okls_api.cu", "okls_gemm.cu", "okls_elementwise.cu", "okls_ns_small.cu",
           "okls_soap.cu", "okls_clean.cu", "okls_clean_large.cu",
           "okls_soap_large.cu", "okls_eig.cu", "okls_bjacobi.cu", "okls_tc3.cu",
           "okls_lm_api.cu", "okls_lm_norm.cu", "okls_lm_embed.cu", "okls_lm_score.cu",
           "okls_fp8_quant.cu", "okls_fp8_gemm.cu", "okls_adamw.cu", "okls_int4.cu", "okls_sample.cu"]
BINDING = "lm_torch.cpp"
BINDING_LIB = os.path.join(PKG, "_lm_native.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags(debug: bool = False) -> list[str]:
    f = ARCH + ["-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
                "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    f += ["-O0", "-G"] if debug else ["-O3"]
    return f


def _run(cmd: list[str]) -> None:
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout)
        raise RuntimeError("command failed: " + " ".join(cmd))
    if r.stdout.strip():
        sys.stderr.write(r.stdout)


def _torch_flags() -> tuple[list[str], list[str]]:
    """Compile and link flags of the binding: torch's headers and libraries."""
    import sysconfig

    import torch
    t = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    inc = ["-I" + p for p in (os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
                              os.path.join(cuda, "include"), sysconfig.get_paths()["include"])]
    link = ["-L" + os.path.join(t, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda",
            "-Wl,-rpath," + os.path.join(t, "lib")]
    return ["-O2", "-std=c++17", "-fPIC", "-Wall", "-Wno-sign-compare", "-DTORCH_API_INCLUDE_EXTENSION_H",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI] + inc, link


def _compile_binding() -> tuple[str, str, list[str]]:
    """Compile the torch binding; returns the compiler, the object and the link flags."""
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    flags, link = _torch_flags()
    obj = os.path.join(BUILD, BINDING + ".o")
    _run([cxx, "-c", os.path.join(CSRC, BINDING), "-o", obj] + flags)
    return cxx, obj, link


def build_library(verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every source for sm_103a and link libokls.so, then the torch binding; returns libokls.so's path.

    The C library needs nvcc alone: it is in place before anything of the binding (torch, the host compiler) can fail."""
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def one(src: str) -> str:
        obj = os.path.join(BUILD, src + ".o")
        cmd = [cc, "-c", os.path.join(CSRC, src), "-o", obj] + _flags() + extra
        if verbose:
            print(" ".join(cmd))
        _run(cmd)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        host = ex.submit(_compile_binding)
        objs = list(ex.map(one, SOURCES))
        tmp = LIB + ".tmp"
        _run([cc, "-shared", "-o", tmp] + objs + ARCH + ["--cudart", "static", "-Xcompiler", "-fPIC"])
        os.replace(tmp, LIB)
        try:
            cxx, obj, link = host.result()
            tmp = BINDING_LIB + ".tmp"
            _run([cxx, "-shared", "-o", tmp, obj, "-L" + PKG, "-lokls", "-Wl,-rpath,$ORIGIN"] + link)
            os.replace(tmp, BINDING_LIB)
        except Exception as e:
            raise RuntimeError(f"libokls.so is built, its torch binding (lm.py) is not: {e}") from e
    return LIB


if __name__ == "__main__":
    print(build_library(verbose=True, ptxas_info="-v" in sys.argv))
