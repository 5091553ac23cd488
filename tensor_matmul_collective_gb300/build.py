"""Build libcoc.so in-tree: nvcc for sm_103a only, the translation units
compiled in parallel, linked with the static CUDA runtime; and beside it
_coc_marshal.so, the decode-step calls' argument marshalling (host code against
this PyTorch's headers)."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libcoc.so")
SOURCES = ["coc_api.cu", "coc_kernel.cu", "coc_slab.cu", "coc_w8_ts.cu", "coc_noalloc.cu", "coc_w8_prepass.cu", "coc_moe.cu",
           "coc_kv_append.cu", "coc_kv_attention.cu", "coc_w4.cu"]
HEADERS = ["coc_internal.h", "coc_dequant.cuh", "coc_ptx.cuh", "coc_kv.cuh", "coc_kv_units.h", os.path.join("..", "..", "include", "coc.h")]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr"]


MARSHAL_SRC = os.path.join(CSRC, "coc_marshal.cpp")
MARSHAL = os.path.join(HERE, "_coc_marshal.so")
MARSHAL_FOR = os.path.join(BUILD, "marshal_for.txt")      # what it was built against


def _marshal_command():
    """The compiler call for _coc_marshal.so, None where there is nothing to build it against."""
    import torch
    inc, lib = (os.path.join(os.path.dirname(torch.__file__), d) for d in ("include", "lib"))
    py = sysconfig.get_paths()["include"]
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    if not (os.path.exists(os.path.join(py, "Python.h")) and os.path.exists(os.path.join(inc, "ATen", "ATen.h"))):
        return None
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            *[f"-isystem{d}" for d in (inc, os.path.join(inc, "torch", "csrc", "api", "include"), py, cuda)], MARSHAL_SRC, "-o", MARSHAL,
            f"-L{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python", f"-Wl,-rpath,{lib}"]


def _marshal_target() -> str:
    import torch
    return f"torch {torch.__version__}, Python {sys.version}"


def _marshal_stale() -> bool:
    if _stale(MARSHAL, [MARSHAL_SRC, os.path.join(CSRC, HEADERS[-1])]) or not os.path.exists(MARSHAL_FOR):
        return True
    with open(MARSHAL_FOR) as f:
        return f.read() != _marshal_target()


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, h) for h in HEADERS]
    objs, procs = [], []
    marshal = _marshal_command() if force or _marshal_stale() else None
    if marshal is not None:
        marshal = (marshal, subprocess.Popen(marshal, stdout=subprocess.PIPE, stderr=subprocess.STDOUT))
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + headers):
            cmd = [nvcc(), *ARCH, *FLAGS, *extra_flags, "-c", s, "-o", o]
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    for cmd, pr in procs:
        out, _ = pr.communicate()
        if pr.returncode != 0:
            raise RuntimeError(f"nvcc failed: {' '.join(cmd)}\n{out.decode(errors='replace')}")
        if verbose and out:
            print(out.decode(errors="replace"), file=sys.stderr)
    if force or procs or _stale(LIB, objs):
        cmd = [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", *objs, "-o", LIB]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}{r.stderr}")
    if marshal is not None:
        out, _ = marshal[1].communicate()
        if marshal[1].returncode != 0:
            raise RuntimeError(f"g++ failed: {' '.join(marshal[0])}\n{out.decode(errors='replace')}")
        with open(MARSHAL_FOR, "w") as f:
            f.write(_marshal_target())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
