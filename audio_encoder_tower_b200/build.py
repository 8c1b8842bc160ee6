"""Build the encoder library (libenc_b200.so) in-tree with nvcc for sm_100a.

    python -m audio_encoder_tower_b200.build [--force] [--verbose]

Every .cu file under csrc/ is compiled for sm_100a (compute_100a) into
_build/, then linked into audio_encoder_tower_b200/libenc_b200.so with the
CUDA runtime linked statically. Where PyTorch is installed, csrc/fastcall.cpp is
compiled as well (g++, no CUDA code): the short way from torch tensors to the
8-bit operators' C calls. Without it the same calls go through ctypes, so a
machine where it does not compile (no g++, a PyTorch without CUDA) gets a warning
and the library.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libenc_b200.so")
FASTCALL_SRC = os.path.join(CSRC, "fastcall.cpp")
FASTCALL = os.path.join(HERE, "_fastcall" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
FASTCALL_STAMP = os.path.join(BUILD, "fastcall.torch")   # the PyTorch version that it was built against

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", INCLUDE]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the encoder library needs the CUDA 12.9 toolkit")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _torch_version(torch_dir: str) -> str:
    """torch.__version__ of an installed PyTorch, without importing it."""
    with open(os.path.join(torch_dir, "version.py")) as f:
        m = re.search(r"^__version__ = ['\"](.*)['\"]", f.read(), re.M)
    return m.group(1) if m else ""


def build_fastcall(force: bool = False) -> str | None:
    """Compile csrc/fastcall.cpp against the installed PyTorch; None where there is none.

    The module reads PyTorch's C++ objects, whose layout changes between versions: it is built
    again for another version, and binding.py uses it only with the version that it names.
    """
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    version = _torch_version(spec.submodule_search_locations[0])
    deps = [FASTCALL_SRC, os.path.join(INCLUDE, "enc_fp8.h"), os.path.join(INCLUDE, "enc.h")]
    if not force and os.path.exists(FASTCALL) and os.path.exists(FASTCALL_STAMP) and \
            all(os.path.getmtime(p) <= os.path.getmtime(FASTCALL) for p in deps):
        with open(FASTCALL_STAMP) as f:
            if f.read() == version:
                return FASTCALL
    torch = spec.submodule_search_locations[0]
    inc = [INCLUDE, os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_path("include"), os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    tmp = FASTCALL + f".{os.getpid()}.tmp"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f'-DENC_TORCH_VERSION="{version}"', *(x for d in inc for x in ("-isystem", d)), FASTCALL_SRC, "-o", tmp, "-L", HERE, "-lenc_b200",
           "-Wl,-rpath,$ORIGIN", "-L", os.path.join(torch, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on fastcall.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, FASTCALL)
    os.makedirs(BUILD, exist_ok=True)
    with open(FASTCALL_STAMP, "w") as f:
        f.write(version)
    return FASTCALL


def _try_fastcall(force: bool = False):
    """build_fastcall, whose failure leaves the library usable: a warning, and no module of another build."""
    try:
        build_fastcall(force)
    except (OSError, RuntimeError) as e:
        if os.path.exists(FASTCALL):
            os.remove(FASTCALL)
        warnings.warn(f"the short call of the 8-bit operators was not built, they go through ctypes: {e}")


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    if not force and up_to_date():
        _try_fastcall()
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    flags = NVCC_FLAGS + (extra_flags or [])
    if verbose:
        flags = flags + ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _try_fastcall(force)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
