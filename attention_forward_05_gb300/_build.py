"""Builds libfa.so in-tree with nvcc for sm_103a (no CMake, no torch extension machinery), and the
Python binding's compiled part with g++ against the installed PyTorch's headers.

The translation units compile in parallel; libfa.so links the CUDA runtime
statically, so it depends only on the driver, and nvcc with its host compiler is
all it takes to build.
The binding links libfa.so and PyTorch, whose internal C++ interfaces it uses:
its file's name carries the Python ABI and the PyTorch version it was built
for, so another one of either builds its own.
"""
from __future__ import annotations

import os
import re
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(PKG, "_build")
LIB = os.path.join(OUT, "libfa.so")
BINDING_SRC = os.path.join(CSRC, "fa_binding.cpp")
SOURCES = ["fa_api.cu", "fa_fwd_bf16.cu", "fa_fwd_fp32.cu", "fa_fwd_merge.cu", "fa_decode.cu",
           "fa_decode_noalloc.cu", "fa_bwd.cu", "fa_bwd_fp32.cu",
           "fa_decode_gqa.cu", "fa_fwd_decode.cu", "fa_rope.cu", "fa_paged.cu", "fa_paged_prefix.cu", "fa_paged_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _deps() -> list[str]:
    """Sources of libfa.so."""
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h"))]
    files.append(os.path.join(INCLUDE, "fa.h"))
    files.append(os.path.abspath(__file__))
    return files


def _older(target: str, files: list[str]) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(f) > os.path.getmtime(target) for f in files)


def is_stale() -> bool:
    return _older(LIB, _deps())


def binding_path() -> str:
    """The binding for the running Python and its PyTorch."""
    import torch

    version = re.sub(r"[^0-9A-Za-z.]", "_", torch.__version__)
    return os.path.join(OUT, f"_fa_binding.torch{version}{sysconfig.get_config_var('EXT_SUFFIX')}")


def binding_is_stale() -> bool:
    return _older(binding_path(), [BINDING_SRC, os.path.join(INCLUDE, "fa.h"), os.path.abspath(__file__)])


def _torch_flags() -> tuple[list[str], list[str]]:
    """g++ compile and link flags for an extension of the installed Python and PyTorch."""
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
    """Compile libfa.so if it is stale or forced; returns its path.

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

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    log = []
    for src, _, r in results:
        log.append(f"== {src}\n{r.stdout}{r.stderr}")
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError(f"nvcc failed on {src}")
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
    return LIB


def _compile_binding() -> str:
    """The binding's object file.  Raises if it does not compile."""
    os.makedirs(OUT, exist_ok=True)
    obj = binding_path() + f".{os.getpid()}.o"
    r = subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", *_torch_flags()[0], "-c", BINDING_SRC, "-o", obj],
                       capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("g++ failed on fa_binding.cpp")
    return obj


def _link_binding(obj: str) -> str:
    path = binding_path()
    tmp = path + f".tmp{os.getpid()}"
    r = subprocess.run(["g++", "-shared", "-o", tmp, obj, f"-L{OUT}", "-l:libfa.so", "-Wl,-rpath,$ORIGIN", *_torch_flags()[1]],
                       capture_output=True, text=True)
    os.remove(obj)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("linking the binding failed")
    os.replace(tmp, path)
    return path


def build_binding(force: bool = False) -> str:
    """Compile the binding if it is stale or forced; returns its path.  libfa.so must be there (build)."""
    if not force and not binding_is_stale():
        return binding_path()
    return _link_binding(_compile_binding())


def build_all(force: bool = False, verbose: bool = False) -> str:
    """libfa.so and the binding, compiled side by side; returns the path of libfa.so, which is there although the
    binding may have failed (then this raises)."""
    with ThreadPoolExecutor(max_workers=1) as ex:
        obj = ex.submit(_compile_binding) if force or binding_is_stale() else None
        build(force, verbose)
        if obj is not None:
            _link_binding(obj.result())
    return LIB


if __name__ == "__main__":
    print(build_all(force="--force" in sys.argv, verbose=True))
