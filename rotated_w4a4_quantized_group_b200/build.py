"""Build the CUDA library libck.so (sm_100a) in-tree, next to this file.

    python -m rotated_w4a4_quantized_group_b200.build [--force]

Compiles every csrc/*.cu with nvcc for sm_100a and links them into one shared
library exporting the C ABI declared in include/ck.h.  It also builds
libck_test_waits.so, the same sources with every role wait limited to zero cycles,
which the bounded-wait expiry test loads to drive each kernel through its timeout path, and
_ck_bind.so, the host side of the fp4 calls (csrc/ck_bind.cpp, against torch's headers).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libck.so")
# variant name -> (output library, extra nvcc flags)
VARIANTS = {
    None: (LIB, []),
    "test_waits": (os.path.join(HERE, "libck_test_waits.so"), ["-DCK_ROLE_WAIT_LIMIT_CYCLES=0"]),
}

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC,
              "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libck.so")
    return p


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]


def needs_build(variant=None) -> bool:
    lib = VARIANTS[variant][0]
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(p) > t for p in _deps())


def _compile(src: str, out_dir: str, extra: list) -> str:
    obj = os.path.join(out_dir, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def build(force: bool = False, variant=None) -> str:
    lib, extra = VARIANTS[variant]
    if not force and not needs_build(variant):
        return lib
    out_dir = BUILD_DIR if variant is None else os.path.join(BUILD_DIR, variant)
    os.makedirs(out_dir, exist_ok=True)
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, out_dir, extra), srcs))
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-Xcompiler", "-fPIC"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


BIND_SRC = os.path.join(CSRC, "ck_bind.cpp")
BIND = os.path.join(HERE, "_ck_bind" + sysconfig.get_config_var("EXT_SUFFIX"))
BIND_TORCH = "ck_bind.torch"    # in BUILD_DIR: the torch version that BIND was built against


def build_bind(force: bool = False) -> str:
    """The Python extension _ck_bind, which loads libck.so when it is told where.  Built again for another
    torch, whose types and symbols may differ."""
    import torch

    deps = [BIND_SRC, __file__] + glob.glob(os.path.join(INCLUDE, "*.h"))
    stamp = os.path.join(BUILD_DIR, BIND_TORCH)
    built_for = open(stamp).read() if os.path.exists(stamp) else None
    if not force and built_for == str(torch.__version__) and os.path.exists(BIND) and \
            all(os.path.getmtime(p) <= os.path.getmtime(BIND) for p in deps):
        return BIND
    t = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = BIND + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DCK_TORCH_VERSION="{torch.__version__}"', "-I" + INCLUDE,
           "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(t, "include"),
           "-I" + os.path.join(t, "include", "torch", "csrc", "api", "include"),
           "-I" + os.path.join(cuda, "include"), BIND_SRC, "-o", tmp, "-L" + os.path.join(t, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BIND_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BIND)
    os.makedirs(BUILD_DIR, exist_ok=True)
    with open(stamp, "w") as f:
        f.write(torch.__version__)
    return BIND


def build_all(force: bool = False) -> list:
    return [build(force, v) for v in VARIANTS] + [build_bind(force)]


if __name__ == "__main__":
    print(build_all(force="--force" in sys.argv))
