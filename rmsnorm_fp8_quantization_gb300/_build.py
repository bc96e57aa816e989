"""Builds libgbnorm.so in-tree from csrc/ with nvcc for sm_103a.

The translation units compile in parallel; the link uses the static CUDA
runtime so the library carries no runtime-library path of this machine.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libgbnorm.so")
BUILD_DIR = os.path.join(PKG, "_build")
# The wrappers' host-side shortcut (csrc/fastcall.cpp), named for this interpreter, and what
# torch it was compiled against.
FAST = os.path.join(PKG, "_fastcall" + sysconfig.get_config_var("EXT_SUFFIX"))
FAST_STAMP = os.path.join(BUILD_DIR, "fastcall.txt")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = ["api.cu", "kernels_f32.cu", "kernels_bf16.cu", "kernels_f16.cu", "finalize.cu",
           "noalloc.cu", "softmax.cu", "rope.cu", "paged_attention.cu",
           "paged_prefill.cu", "attention_bwd.cu",
           "attention_bwd_bf16.cu", "attention_bwd_f16.cu", "dropout.cu"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgbnorm.so")
    return cand


def _inputs():
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "gbnorm.h")]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def torch_tag() -> str:
    """The torch whose object layouts the shortcut has compiled in; another one must not load it."""
    import torch
    return f"{torch.__version__} {torch.version.git_version}"


def fastcall_up_to_date() -> bool:
    try:
        with open(FAST_STAMP) as f:
            return os.path.exists(FAST) and f.read() == torch_tag()
    except OSError:
        return False


def _compile_fastcall() -> str:
    """Compiles FAST; returns why it could not, or an empty string."""
    import torch
    gxx = shutil.which("g++")
    if gxx is None:
        return "no g++"
    try:
        cuda = os.path.dirname(os.path.dirname(_nvcc()))
    except RuntimeError as e:
        return str(e)
    home = os.path.dirname(torch.__file__)
    tmp = FAST + f".tmp{os.getpid()}"
    cmd = [gxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-DNDEBUG",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DGBN_BUILT_FOR="{torch_tag()}"', "-I", INCLUDE,
           "-I", os.path.join(home, "include"),
           "-I", os.path.join(home, "include", "torch", "csrc", "api", "include"),
           "-I", os.path.join(cuda, "include"), "-I", sysconfig.get_paths()["include"],
           os.path.join(CSRC, "fastcall.cpp"), "-o", tmp, "-L", os.path.join(home, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        return r.stderr[-2000:]
    os.replace(tmp, FAST)
    os.makedirs(BUILD_DIR, exist_ok=True)
    with open(FAST_STAMP, "w") as f:
        f.write(torch_tag())
    return ""


def build_fastcall() -> None:
    """The wrappers' host-side shortcut, a small CPython module over torch's C++
    headers.  Without a compiler, the toolkit's headers or torch's it is left out (the
    wrappers then do the same in Python, at 10 to 15 us more host time a call)."""
    try:
        why = _compile_fastcall()
    except OSError as e:
        why = str(e)
    if why:
        sys.stderr.write(f"fastcall.cpp not built (the wrappers work without it): {why}\n")


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if not force and up_to_date():
        if not fastcall_up_to_date():
            build_fastcall()
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    common = [nvcc, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-I", INCLUDE, "-I", CSRC]
    if verbose_ptxas:
        common += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        cmd = common + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        fast = ex.submit(build_fastcall)
        results = list(ex.map(compile_one, SOURCES))
        fast.result()
    if verbose_ptxas:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv)
    print(LIB)
