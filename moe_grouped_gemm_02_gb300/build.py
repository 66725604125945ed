"""Builds libdg.so in-tree: every csrc/*.cu compiled for sm_103a in parallel, then linked; and beside it
the Python binding dg_binding.so (csrc/dg_binding.cpp, against the installed torch).

    python -m moe_grouped_gemm_02_gb300.build [--force] [--verbose]

--verbose adds `-Xptxas -v` (registers, spills, shared memory per kernel).
"""
from __future__ import annotations

import concurrent.futures
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
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libdg.so")
BINDING_SRC = os.path.join(CSRC, "dg_binding.cpp")
BINDING_OBJ = os.path.join(BUILD_DIR, "dg_binding.o")
BINDING_PATH = os.path.join(HERE, "dg_binding.so")

GENCODE = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale(obj: str, src: str) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(p) > t for p in [src] + _headers())


def _older(out: str, parts) -> bool:
    """Whether `out` is missing or was linked before one of its parts was compiled."""
    return not os.path.exists(out) or any(os.path.getmtime(p) > os.path.getmtime(out) for p in parts)


def _run(cmd, what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(what)


def _compile_binding() -> None:
    """dg_binding.cpp with the host compiler, against the headers of Python, torch and CUDA."""
    from torch.utils import cpp_extension
    import torch
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    inc = [sysconfig.get_paths()["include"], *cpp_extension.include_paths(), cuda, INCLUDE]
    _run(["g++", "-O2", "-std=c++20" if tuple(map(int, torch.__version__.split(".")[:2])) >= (2, 10) else "-std=c++17",
          "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[x for i in inc for x in ("-isystem", i)],
          "-c", BINDING_SRC, "-o", BINDING_OBJ], "g++ failed on dg_binding.cpp")


def _link_binding() -> None:
    """dg_binding.so: libdg.so from its own folder, torch's libraries as the process has loaded them."""
    from torch.utils import cpp_extension
    libs = [x for p in cpp_extension.library_paths() for x in ("-L", p)]
    _run(["g++", "-shared", "-o", BINDING_PATH + ".tmp", BINDING_OBJ, LIB_PATH, *libs, "-lc10", "-lc10_cuda", "-ltorch_cpu",
          "-ltorch_python", "-Wl,-rpath,$ORIGIN"], "link of dg_binding.so failed")
    os.replace(BINDING_PATH + ".tmp", BINDING_PATH)


def build(force: bool = False, verbose: bool = False) -> str:
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    objs = [os.path.join(BUILD_DIR, os.path.basename(s)[:-3] + ".o") for s in sources]
    todo = [(s, o) for s, o in zip(sources, objs) if force or _stale(o, s)]
    extra = ["-Xptxas", "-v"] if verbose else []

    def compile_one(so):
        src, obj = so
        cmd = [nvcc, *GENCODE, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, r.returncode, r.stdout + r.stderr

    binding = force or _stale(BINDING_OBJ, BINDING_SRC)
    if todo or binding:
        with concurrent.futures.ThreadPoolExecutor(max_workers=min(len(todo) + 1, os.cpu_count() or 4)) as ex:
            done = ex.submit(_compile_binding) if binding else None
            for src, rc, out in ex.map(compile_one, todo):
                if verbose or rc != 0:
                    sys.stderr.write(out)
                if rc != 0:
                    raise RuntimeError(f"nvcc failed on {os.path.basename(src)}")
            if done is not None:
                done.result()
    # (by the files, not by what was compiled just now: a build that failed halfway left parts behind)
    if _older(LIB_PATH, objs):
        tmp = LIB_PATH + ".tmp"
        # (the soname is what dg_binding.so records: it finds the library in its own folder)
        cmd = [nvcc, *GENCODE, "-shared", "-Xlinker", "-soname=libdg.so", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link of libdg.so failed")
        os.replace(tmp, LIB_PATH)
    if _older(BINDING_PATH, [BINDING_OBJ]):
        _link_binding()
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
