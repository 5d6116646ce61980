"""Builds libfa.so in-tree with nvcc for sm_103a (no CMake, no torch extension machinery), and the
Python binding's compiled part, _fa_binding.so, with g++ against the installed PyTorch's headers.

The translation units compile in parallel; libfa.so links the CUDA runtime
statically, so it depends only on the driver.  The binding links libfa.so and
PyTorch.
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(PKG, "_build")
LIB = os.path.join(OUT, "libfa.so")
BINDING = os.path.join(OUT, "_fa_binding.so")
BINDING_SRC = os.path.join(CSRC, "fa_binding.cpp")
SOURCES = ["fa_api.cu", "fa_fwd_bf16.cu", "fa_fwd_fp32.cu", "fa_fwd_merge.cu", "fa_decode.cu",
           "fa_decode_noalloc.cu", "fa_bwd.cu", "fa_bwd_fp32.cu",
           "fa_decode_gqa.cu", "fa_fwd_decode.cu", "fa_rope.cu", "fa_paged.cu", "fa_paged_prefix.cu", "fa_paged_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _deps() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h", ".cpp"))]
    files.append(os.path.join(INCLUDE, "fa.h"))
    files.append(os.path.abspath(__file__))
    return files


def is_stale() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(BINDING)):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return any(os.path.getmtime(f) > t for f in _deps())


def _torch_flags() -> tuple[list[str], list[str]]:
    """g++ compile and link flags for an extension of the installed Python and PyTorch."""
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
    lib = os.path.join(root, "lib")
    return ([f"-D_GLIBCXX_USE_CXX11_ABI={abi}", *[f"-I{d}" for d in inc]],
            [f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10_cuda", "-lc10", f"-Wl,-rpath,{lib}"])


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if stale or forced) libfa.so and the binding; returns the path of libfa.so.

    FA_PTXAS_VERBOSE=1 in the environment adds ``-Xptxas -v`` and keeps its
    register / spill report in _build/ptxas.log.
    """
    if not force and not is_stale():
        return LIB
    os.makedirs(OUT, exist_ok=True)
    nvcc = _nvcc()
    ptxas_v = os.environ.get("FA_PTXAS_VERBOSE") == "1"
    flags = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
                    "--expt-relaxed-constexpr"]
    if ptxas_v:
        flags += ["-Xptxas", "-v"]

    def compile_one(src: str):
        obj = os.path.join(OUT, src.replace(".cu", ".o"))
        cmd = [nvcc, *flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    torch_cflags, torch_ldflags = _torch_flags()
    binding_obj = os.path.join(OUT, "fa_binding.o")

    def compile_binding():
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", *torch_cflags, "-c", BINDING_SRC, "-o", binding_obj]
        return "fa_binding.cpp", binding_obj, subprocess.run(cmd, capture_output=True, text=True)

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(compile_binding)
        results = list(ex.map(compile_one, SOURCES))
        bound = binding.result()
    log = []
    for src, _, r in [*results, bound]:
        log.append(f"== {src}\n{r.stdout}{r.stderr}")
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError(f"compiling {src} failed")
    if ptxas_v or verbose:
        with open(os.path.join(OUT, "ptxas.log"), "w") as f:
            f.write("\n".join(log))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *[obj for _, obj, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("nvcc link failed")
    os.replace(tmp, LIB)
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, binding_obj, f"-L{OUT}", "-l:libfa.so", "-Wl,-rpath,$ORIGIN", *torch_ldflags]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("linking the binding failed")
    os.replace(tmp, BINDING)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
