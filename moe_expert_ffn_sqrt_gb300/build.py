"""Builds libmoe.so in-tree with nvcc for sm_103a (one -gencode, translation units in parallel), and the Python binding's
argument marshalling (_native.so) with g++ against the installed torch.

Usage: python -m moe_expert_ffn_sqrt_gb300.build   (or call build()).
"""
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe.so")
NATIVE = os.path.join(PKG, "_native.so")
SOURCES = ["api.cu", "route.cu", "route_noalloc.cu", "permute.cu", "gate.cu", "gemm.cu", "gemm_nv.cu", "gemm_i8.cu", "reduce.cu",
           "train_api.cu", "train_rows.cu", "route_grad.cu", "linear.cu", "norm.cu", "select.cu",
           "rows8.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(OUT_DIR, src.replace(".cu", ".o"))
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    with open(os.path.join(OUT_DIR, src + ".ptxas.txt"), "w") as f:
        f.write(r.stderr)
    if verbose:
        print(f"compiled {src}", file=sys.stderr)
    return obj


def _native(verbose: bool) -> None:
    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = NATIVE + ".tmp"
    cmd = [os.environ.get("CXX") or shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", os.path.join(CSRC, "native.cpp"), "-o", tmp,
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu",
           "-lc10", "-lc10_cuda", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for native.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, NATIVE)
    if verbose:
        print("compiled native.cpp", file=sys.stderr)


def build(verbose: bool = False) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    with ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        native = ex.submit(_native, verbose)
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
        native.result()
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
