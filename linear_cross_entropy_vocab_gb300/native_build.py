"""Builds libflce.so in-tree with nvcc for sm_103a (GB300).

The translation units are compiled in parallel and linked into
``linear_cross_entropy_vocab_gb300/_build/libflce.so``; the CUDA runtime is
linked statically and the driver's tensor-map encoder is looked up at run
time, so the library needs no libcuda at link time. Beside it lies
``libflce_torch.so``: the operators that are registered with PyTorch, compiled
by the host compiler against the installed PyTorch and linked to libflce.so. It works with that
PyTorch alone, so ``libflce_torch.json`` says which one it was.
"""
from __future__ import annotations

import concurrent.futures
import json
import os
import shutil
import subprocess
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libflce.so")
TORCH_LIB = os.path.join(BUILD, "libflce_torch.so")
TORCH_SOURCE = "norm_torch.cpp"
TORCH_STAMP = os.path.join(BUILD, "libflce_torch.json")

SOURCES = ["flce_api.cu", "kernels_tc.cu", "kernels_simt.cu", "kernels_rows.cu",
           "grads_api.cu", "kernels_grads.cu", "beam_api.cu", "kernels_beam.cu",
           "int8_api.cu", "kernels_int8.cu", "kernels_qlinear.cu",
           "norm_api.cu", "kernels_norm.cu", "kernels_norm_q.cu", "kernels_norm_bwd.cu",
           "ortho_api.cu", "kernels_ortho.cu", "kernels_ortho_small.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found (need the CUDA 13 toolkit)")
    return cand


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "flce.h"))
    files.append(os.path.abspath(__file__))
    return files


def _installed_torch() -> dict:
    """What libflce_torch.so depends on beside its sources."""
    import torch

    return {"version": str(torch.__version__), "git": torch.version.git_version,
            "cxx11_abi": bool(torch.compiled_with_cxx11_abi())}


def torch_mismatch() -> Optional[str]:
    """Why libflce_torch.so does not go with the installed PyTorch, or None."""
    try:
        with open(TORCH_STAMP) as f:
            built = dict(json.load(f))
    except (OSError, ValueError, TypeError):
        return "it does not say which PyTorch it was built against"
    return ", ".join(f"{k} {built.get(k)} when it was built, {v} here"
                     for k, v in _installed_torch().items() if built.get(k) != v) or None


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(TORCH_LIB)) or torch_mismatch():
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(TORCH_LIB))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _compile_torch() -> str:
    """The object file of the operators that are registered with PyTorch."""
    import torch

    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        raise RuntimeError("no C++ compiler found (g++)")
    include = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    obj = os.path.join(BUILD, "norm_torch.o")
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE, "-isystem", include, "-isystem",
           os.path.join(include, "torch", "csrc", "api", "include"), "-isystem", cuda,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-c",
           os.path.join(CSRC, TORCH_SOURCE), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cxx} failed on {TORCH_SOURCE}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_torch(obj: str) -> None:
    import torch

    tmp = TORCH_LIB + ".tmp"
    cmd = [shutil.which("g++") or shutil.which("c++"), "-shared", "-o", tmp, obj, "-L", BUILD,
           "-lflce", "-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_cpu",
           "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    # the stamp is away while the library and it may disagree
    if os.path.exists(TORCH_STAMP):
        os.remove(TORCH_STAMP)
    os.replace(tmp, TORCH_LIB)
    with open(TORCH_STAMP + ".tmp", "w") as f:
        json.dump(_installed_torch(), f)
    os.replace(TORCH_STAMP + ".tmp", TORCH_STAMP)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile (if stale) and return the path of libflce.so."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *NVCC_FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        torch_obj = ex.submit(_compile_torch)
        objs = list(ex.map(compile_one, SOURCES))
        torch_obj = torch_obj.result()
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_torch(torch_obj)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
