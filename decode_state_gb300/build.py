"""Builds the SDM CUDA library ``_build/libsdm.so`` in place with nvcc, for sm_103a only.

Each ``csrc/*.cu`` file compiles to an object in parallel; the objects link into one shared
library that exports the C ABI of ``include/sdm.h`` and links the CUDA runtime dynamically (so a
process that already loaded PyTorch's runtime reuses it). Beside it ``_build/sdm_torch.so`` binds the
operators that are called once a token to PyTorch tensors (``csrc/torch_binding.cpp``, host code
compiled against the installed PyTorch).
"""

from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(OUT_DIR, "libsdm.so")
BINDING_PATH = os.path.join(OUT_DIR, "sdm_torch.so")
BINDING = "torch_binding.cpp"
SOURCES = ["sdm_abi.cu", "sdm_abi_quant.cu", "sdm_abi_train.cu", "decode.cu", "gather.cu", "quant.cu", "qgather.cu", "qgather_ring.cu",
           "qdecode.cu", "route.cu", "balance.cu", "balance_bf16.cu", "balance_f32.cu", "lookup.cu", "row_sums.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise FileNotFoundError("nvcc not found (set NVCC or put the CUDA toolkit on PATH)")


def cuda_lib_dir() -> str:
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "lib64")


def compile_command(src: str, obj: str, extra: list[str] | None = None) -> list[str]:
    return [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
            *(extra or []), "-c", os.path.join(CSRC, src), "-o", obj]


def binding_command(obj: str) -> list[str]:
    import sysconfig

    import torch

    root = os.path.join(os.path.dirname(torch.__file__), "include")
    system = [root, os.path.join(root, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"],
              os.path.join(os.path.dirname(cuda_lib_dir()), "include")]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-Wall", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
            *(f for d in system for f in ("-isystem", d)), "-c", os.path.join(CSRC, BINDING), "-o", obj]


def binding_link_command(obj: str, out: str) -> list[str]:
    import torch

    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    return [os.environ.get("CXX", "g++"), "-shared", "-o", out, obj, LIB_PATH, "-L", libs, "-ltorch_python", "-ltorch_cuda",
            "-ltorch_cpu", "-lc10_cuda", "-lc10", "-L", cuda_lib_dir(), "-lcudart", "-Wl,-rpath,$ORIGIN",
            f"-Wl,-rpath,{libs}", f"-Wl,-rpath,{cuda_lib_dir()}"]


def _link(cmd: list[str], path: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        print(" ".join(cmd))
        print(r.stdout + r.stderr)
        raise RuntimeError(f"linking {os.path.basename(path)} failed")
    os.replace(cmd[cmd.index("-o") + 1], path)


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    """Compile and link libsdm.so if any source or header is newer; returns its path."""
    os.makedirs(OUT_DIR, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(INCLUDE, "sdm.h"))
    objs = []
    jobs = []
    for src in SOURCES:
        obj = os.path.join(OUT_DIR, src.replace(".cu", ".o"))
        objs.append(obj)
        if force or _stale(obj, [os.path.join(CSRC, src), *headers]):
            jobs.append(compile_command(src, obj, extra))
    binding_obj = os.path.join(OUT_DIR, BINDING.replace(".cpp", ".o"))
    if force or _stale(binding_obj, [os.path.join(CSRC, BINDING), os.path.join(INCLUDE, "sdm.h")]):
        jobs.append(binding_command(binding_obj))
    if jobs:
        with concurrent.futures.ThreadPoolExecutor(max_workers=len(jobs)) as ex:
            results = list(ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs))
        for cmd, r in zip(jobs, results):
            if verbose or r.returncode != 0:
                print(" ".join(cmd))
                print(r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError(f"compiling {cmd[-3]} failed")
    if force or jobs or _stale(LIB_PATH, objs):
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        _link([nvcc(), *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs, "-Xlinker", f"-rpath,{cuda_lib_dir()}",
               "-Xlinker", "-soname,libsdm.so"], LIB_PATH)
    if force or jobs or _stale(BINDING_PATH, [binding_obj, LIB_PATH]):
        tmp = BINDING_PATH + f".tmp{os.getpid()}"
        _link(binding_link_command(binding_obj, tmp), BINDING_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))
