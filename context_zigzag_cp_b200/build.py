"""Build libcpattn.so with nvcc for sm_100a and _calls.so, the binding's native part, in-tree
(python -m context_zigzag_cp_b200.build)."""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig
import warnings

_HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(_HERE)
LIB = os.path.join(_HERE, "libcpattn.so")
SRC = os.path.join(_HERE, "csrc", "cp_attn.cu")
CALLS = os.path.join(_HERE, "_calls.so")
CALLS_SRC = os.path.join(_HERE, "csrc", "calls.cpp")

NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
              "-Xptxas", "-v", "-shared", "-Xcompiler", "-fPIC", "-Xcompiler",
              "-fvisibility=hidden", "-cudart", "static"]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return [SRC] + sorted(glob.glob(os.path.join(_HERE, "csrc", "*.cuh")) +
                          glob.glob(os.path.join(_HERE, "csrc", "*.h")) +
                          [os.path.join(ROOT, "include", "cp_attn.h")])


def _newer(target, srcs) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(s) <= os.path.getmtime(target) for s in srcs)


def up_to_date() -> bool:
    return _newer(LIB, sources())


def _run(cmd, target, verbose):
    tmp = target + ".tmp%d" % os.getpid()
    res = subprocess.run(cmd + ["-o", tmp], capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed building {os.path.basename(target)}")
    if verbose:
        sys.stderr.write(res.stderr)
    os.replace(tmp, target)


def calls_mark() -> str:
    """What _calls.so says of the torch that it was built against: its classes are that torch's alone."""
    import torch
    return f"built for torch {torch.__version__}"


def calls_up_to_date() -> bool:
    if not _newer(CALLS, [CALLS_SRC, os.path.join(ROOT, "include", "cp_attn.h")]):
        return False
    with open(CALLS, "rb") as f:
        return calls_mark().encode() + b"\0" in f.read()


def _build_calls(verbose: bool) -> None:
    """_calls.so against the installed torch, whose allocator and streams it uses."""
    import torch
    root = os.path.dirname(torch.__file__)
    nvcc = _nvcc()
    cuda = os.path.dirname(os.path.dirname(nvcc)) if os.path.isabs(nvcc) else "/usr/local/cuda"
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"], os.path.join(ROOT, "include")]
    libs = os.path.join(root, "lib")
    _run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DCALLS_MARK="{calls_mark()}"'] + ["-I" + i for i in inc] +
         [CALLS_SRC, "-L" + libs, "-Wl,-rpath," + libs, "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"],
         CALLS, verbose)


def build(force: bool = False, verbose: bool = False) -> str:
    if force or not up_to_date():
        _run([_nvcc()] + NVCC_FLAGS + ["-I", os.path.join(ROOT, "include"), SRC], LIB, verbose)
    if force or not calls_up_to_date():
        try:
            _build_calls(verbose)
        except (RuntimeError, OSError) as e:   # no g++, no headers of torch: the library itself does without
            warnings.warn(f"_calls.so: {e}; the decoding calls go through Python, some 25 us slower")
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
