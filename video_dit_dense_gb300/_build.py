"""Build libh3attn.so in-tree with nvcc for sm_103a, and _step.so, the Python
binding's host path of the generation operators, with g++ against torch (where
there is one: the C library needs the CUDA toolkit alone).

Translation units compile in parallel; the CUDA runtime is linked
statically so the library loads without a CUDA toolkit on the library path.
A stamp of the sources and flags skips rebuilds when nothing changed.
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libh3attn.so")
STEP_LIB = os.path.join(HERE, "_step.so")
STEP_SOURCE = "step.cpp"
BUILD_DIR = os.path.join(HERE, "_build")
SOURCES = ["api.cu", "api_generate.cu", "qk_norm_rope.cu", "attn_fwd.cu", "rmsnorm_modulate.cu", "add_rmsnorm.cu",
           "rope_table.cu", "norm_rope_append.cu", "paged_decode.cu", "paged_decode_q4.cu", "decode_weights.cu", "paged_read.cu",
           "paged_evict.cu"]
HEADERS = ["ptx.cuh", "internal.h", "api_common.h", "generate.h", "cache4.cuh", "decode_common.cuh", "attn_pipe.cuh", "attn_persist.cuh", "attn_wide.cuh", "attn_chain.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
                     "--expt-relaxed-constexpr", f"-I{INCLUDE}"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: libh3attn needs the CUDA toolkit to build")


def _stamp() -> str:
    h = hashlib.sha256()
    for name in SOURCES + HEADERS:
        with open(os.path.join(CSRC, name), "rb") as f:
            h.update(name.encode() + f.read())
    with open(os.path.join(INCLUDE, "h3attn.h"), "rb") as f:
        h.update(f.read())
    h.update(" ".join(NVCC_FLAGS).encode())
    return h.hexdigest()[:20]


def _torch():
    """The torch that the Python binding's host path is built against: None where there is none with CUDA.  The C library
    needs neither torch nor Python."""
    try:
        import torch
    except (ImportError, OSError):  # none, or one whose libraries do not load
        return None
    return torch if torch.version.cuda is not None else None


def _step_flags(torch) -> list[str]:
    return ["-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]


def _step_command(torch, out: str) -> list[str]:
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    includes = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    return ["g++", *_step_flags(torch), *(f"-isystem{i}" for i in includes), os.path.join(CSRC, STEP_SOURCE), "-o", out,
            "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


def step_versions(torch) -> str:
    """What the host path is compiled for and loads with, no other: neither has a stable binary interface."""
    return f"torch {torch.__version__}, Python {sys.version_info.major}.{sys.version_info.minor}"


def step_built_for() -> str:
    """step_versions() of the host path that is there ("" where that is not known)."""
    if not os.path.exists(STEP_LIB + ".stamp"):
        return ""
    with open(STEP_LIB + ".stamp") as f:
        return f.read().strip().partition(" ")[2]


def _step_stamp(torch) -> str:
    """Of the sources, the flags and the versions, not of the toolkit: what is current needs no nvcc."""
    h = hashlib.sha256(" ".join(_step_flags(torch)).encode())
    for path in (os.path.join(CSRC, STEP_SOURCE), os.path.join(INCLUDE, "h3attn.h")):
        with open(path, "rb") as f:
            h.update(f.read())
    return f"{h.hexdigest()[:20]} {step_versions(torch)}"


def _current(lib: str, stamp: str) -> bool:
    if not os.path.exists(lib) or not os.path.exists(lib + ".stamp"):
        return False
    with open(lib + ".stamp") as f:
        return f.read().strip() == stamp


def _build_step(torch, stamp: str) -> None:
    tmp = STEP_LIB + f".tmp{os.getpid()}"
    r = subprocess.run(_step_command(torch, tmp), capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {STEP_SOURCE}:\n{r.stderr}")
    os.replace(tmp, STEP_LIB)
    with open(STEP_LIB + ".stamp", "w") as f:
        f.write(stamp)


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds what is not current, and returns the C library's path.  Without a torch the binding's host path is left out
    (its functions say so when they are called); where it does not compile, the C library is built before that is raised."""
    torch = _torch()
    st, step_stamp = _stamp(), _step_stamp(torch) if torch else None
    step_needed = torch is not None and (force or not _current(STEP_LIB, step_stamp))
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        step = ex.submit(_build_step, torch, step_stamp) if step_needed else None
        if force or not _current(LIB, st):
            _build_lib(st, verbose)
        if step is not None:
            step.result()
    return LIB


def _build_lib(stamp: str, verbose: bool) -> None:
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [nvcc] + NVCC_FLAGS + (["-Xptxas", "-v"] if verbose else []) + [
            "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    with open(LIB + ".stamp", "w") as f:
        f.write(stamp)


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
