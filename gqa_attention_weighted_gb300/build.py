"""In-tree build of libgqa_av.so (sm_103a) with nvcc, and of the Python calls around
it that need the tensors' C++ side (_fastcall, with the host compiler). The library
needs neither Python's nor torch's headers; where _fastcall cannot be built the
Python binding does without it.

The translation units compile in parallel; both land next to this file so that
the Python binding loads them from the source tree. Nothing is
installed into site-packages.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIBRARY = os.path.join(PKG, "libgqa_av.so")
FASTCALL = os.path.join(PKG, "_fastcall" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
FASTCALL_TORCH = os.path.join(BUILD_DIR, "fastcall_torch.txt")   # what _fastcall was built against

SOURCES = ["gqa_av_api.cu", "gqa_av_bf16.cu", "gqa_av_fp16.cu", "gqa_av_noalloc.cu", "gqa_qk_api.cu",
           "gqa_attn_api.cu", "gqa_kv_api.cu", "gqa_prefix_api.cu", "gqa_prompt_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                     "-diag-suppress", "1160", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = os.path.join(home, "bin", "nvcc")
    return path if os.path.exists(path) else "nvcc"


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return files


def _newer(built: str) -> bool:
    """Whether a built file is there and no source has changed since."""
    return os.path.exists(built) and all(os.path.getmtime(f) <= os.path.getmtime(built)
                                         for f in _inputs())


def torch_kind() -> str:
    """What an extension built against this torch depends on."""
    import torch

    return f"{torch.__version__} abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}"


def fastcall_fits() -> bool:
    """Whether _fastcall is there and was built against this torch."""
    try:
        with open(FASTCALL_TORCH) as f:
            return os.path.exists(FASTCALL) and f.read() == torch_kind()
    except (OSError, ImportError):
        return False


def fastcall_up_to_date() -> bool:
    return fastcall_fits() and _newer(FASTCALL)


def up_to_date() -> bool:
    return _newer(LIBRARY) and fastcall_up_to_date()


def fastcall_command(out: str) -> list:
    import torch

    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    include = [INCLUDE, os.path.join(home, "include"),
               os.path.join(home, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[x for path in include for x in ("-I", path)],
            os.path.join(CSRC, "gqa_fastcall.cpp"), "-o", out, "-L", os.path.join(home, "lib"),
            "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]


def build_fastcall(verbose: bool = False) -> None:
    """Compile _fastcall; a warning where that fails."""
    try:
        cmd = fastcall_command(FASTCALL + ".tmp")
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        r = subprocess.run(cmd, capture_output=True, text=True)
        error = r.stdout + r.stderr if r.returncode else ""
    except (ImportError, OSError) as e:
        error = str(e)
    if error:
        warnings.warn(f"_fastcall was not built, its calls check their tensors in Python:\n{error}")
        return
    os.replace(FASTCALL + ".tmp", FASTCALL)
    with open(FASTCALL_TORCH, "w") as f:
        f.write(torch_kind())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link what is not up to date of libgqa_av.so and _fastcall; returns the
    library's path."""
    if not force and up_to_date():
        return LIBRARY
    os.makedirs(BUILD_DIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=1) as ex:
        fast = None if not force and fastcall_up_to_date() else ex.submit(build_fastcall, verbose)
        if force or not _newer(LIBRARY):
            build_library(verbose)
        if fast:
            fast.result()
    return LIBRARY


def build_library(verbose: bool = False) -> None:
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIBRARY + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIBRARY)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
