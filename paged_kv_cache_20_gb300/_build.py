"""Build libpagedattn.so in-tree with nvcc for sm_103a.

Each .cu file compiles to an object in parallel, then one link step produces
``paged_kv_cache_20_gb300/libpagedattn.so``.  The library links the shared CUDA
runtime so it shares one runtime instance with PyTorch in the same process.  The
binding's checked calls (``csrc/pa_calls.cpp``, host code against torch's headers) go
into ``paged_kv_cache_20_gb300/_calls.so`` beside it; where they cannot be built the
binding makes the same calls without them.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIBRARY = os.path.join(HERE, "libpagedattn.so")
CALLS = os.path.join(HERE, "_calls.so")   # the binding's checked calls (host code only)

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden", "-I", INCLUDE, "--threads", "2"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "pagedattn.h"))
    files.append(__file__)
    return files


def _calls_record() -> str:
    """File that says for which torch the checked calls were last built, or tried."""
    return os.path.join(BUILD_DIR, "calls.txt")


def needs_build() -> bool:
    import torch
    if not os.path.exists(LIBRARY) or not os.path.exists(_calls_record()):
        return True
    with open(_calls_record()) as f:
        outcome, version = f.read().split()
    if version != torch.__version__ or (outcome == "built" and not os.path.exists(CALLS)):
        return True
    t = min(os.path.getmtime(LIBRARY), os.path.getmtime(_calls_record()))
    return any(os.path.getmtime(f) > t for f in _deps())


def calls_command(out: str) -> list[str]:
    import sysconfig

    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f'-DPA_TORCH_VERSION="{torch.__version__}"',
            "-I", sysconfig.get_paths()["include"], "-I", os.path.join(root, "include"),
            "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
            "-I", os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include"),
            os.path.join(CSRC, "pa_calls.cpp"), "-o", out, "-L", os.path.join(root, "lib"),
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-L", HERE, "-l:libpagedattn.so",
            "-Wl,-rpath,$ORIGIN"]


def build_calls() -> None:
    """The checked calls, after the library.  They only shorten calls: where they cannot be
    built (no headers of Python or torch) that is a warning, and none are left behind."""
    import torch
    tmp = CALLS + ".tmp"
    cmd = calls_command(tmp)
    try:
        res = subprocess.run(cmd, capture_output=True, text=True)
        failure = res.stdout + res.stderr if res.returncode != 0 else None
    except OSError as e:
        failure = str(e)
    if failure is None:
        os.replace(tmp, CALLS)
    else:
        if os.path.exists(CALLS):
            os.remove(CALLS)
        warnings.warn(f"_calls.so not built, calls are checked in Python: {' '.join(cmd)}\n{failure}",
                      RuntimeWarning, stacklevel=2)
    with open(_calls_record(), "w") as f:
        f.write(f"{'failed' if failure is not None else 'built'} {torch.__version__}\n")


def build(verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed: {' '.join(cmd)}\n{res.stdout}{res.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(res.stdout + res.stderr)
        return obj

    srcs = sources()
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIBRARY + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-cudart", "shared", *objs, "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{res.stdout}{res.stderr}")
    os.replace(tmp, LIBRARY)
    build_calls()
    return LIBRARY


if __name__ == "__main__":
    print(build(verbose=True, ptxas_info="-v" in sys.argv))
