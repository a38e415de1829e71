"""Builds libbitlinear.so (the C-ABI CUDA library) in-tree for sm_103a.

Each .cu file is compiled by nvcc in parallel into bitlinear_w1_a8_gb300/_build/
and linked into bitlinear_w1_a8_gb300/_build/libbitlinear.so.  Needs nvcc but
no GPU (the container cross-compiles; the GPU host rebuilds for its own CPU).
Beside it, _build/bitlinear_marshal-<key>.so (host code, g++ with the headers of
Python and torch) reads the attention calls' tensors faster than the Python binding
can; where it cannot be built the binding does all of it.  The key stands for its
source, the library's header and the Python and torch it was compiled against.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(BUILD, "libbitlinear.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + [
    "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
    "--fmad=false",          # quantisation arithmetic is unfused IEEE fp32 everywhere
    "-prec-div=true", "-prec-sqrt=true",
    "-I", INCLUDE, "-I", CSRC,
]
SOURCES = ["abi.cu", "wquant.cu", "aquant.cu", "decode.cu", "prefill.cu", "wide.cu", "argmax.cu",
           "rope_kv.cu", "attention.cu"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the BitLinear CUDA library cannot be built")


def _stale(out: str, deps: list[str]) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _marshal_command(out: str) -> list[str] | None:
    """The compile command of marshal.cpp, or None without torch or the headers it takes."""
    try:
        import torch
    except Exception:  # missing, or broken: the library needs none
        return None
    at, python = os.path.dirname(torch.__file__), sysconfig.get_paths()["include"]
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    if not (os.path.exists(os.path.join(python, "Python.h"))
            and os.path.exists(os.path.join(at, "include", "torch", "csrc", "autograd", "python_variable.h"))
            and shutil.which("g++")):
        return None
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", INCLUDE, "-I", os.path.join(at, "include"),
            "-I", os.path.join(at, "include", "torch", "csrc", "api", "include"), "-I", cuda, "-I", python,
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", os.path.join(CSRC, "marshal.cpp"),
            "-o", out, "-L", os.path.join(at, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


def marshal_path() -> str | None:
    """Where the module is that belongs to the sources as they are and to this Python and torch; None
    without torch.  It holds torch's and Python's layouts and the C ABI's, so no other may be loaded."""
    try:
        import torch
    except Exception:  # missing, or broken: the library needs none
        return None
    key = hashlib.sha256()
    for at in (os.path.join(CSRC, "marshal.cpp"), os.path.join(INCLUDE, "bitlinear.h")):
        with open(at, "rb") as f:
            key.update(hashlib.sha256(f.read()).digest())
    key.update(repr((torch.__version__, torch.version.git_version, sysconfig.get_config_var("SOABI"))).encode())
    return os.path.join(BUILD, f"bitlinear_marshal-{key.hexdigest()[:16]}.so")


def _build_marshal(force: bool, verbose: bool) -> tuple[str, str] | None:
    """Compiles the module unless it is there -> (the new file, its place), or None.  Those of other
    sources or versions are removed first, whatever becomes of this one."""
    at = marshal_path()
    if at is None:
        return None
    for old in glob.glob(os.path.join(glob.escape(BUILD), "bitlinear_marshal*.so")):
        if force or old != at:
            try:
                os.unlink(old)
            except FileNotFoundError:  # another build was faster
                pass
    if os.path.exists(at):
        return None
    tmp = at + f".{os.getpid()}.tmp"
    cmd = _marshal_command(tmp)
    if cmd is None:
        return None
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(f"bitlinear_marshal not built, the Python binding does its work:\n{r.stderr[-2000:]}\n")
        return None
    return tmp, at


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(INCLUDE, "bitlinear.h"))
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s, *headers, __file__]):
            cmd = [nvcc, *NVCC_FLAGS, "-c", s, "-o", o]
            if ptxas_verbose:
                cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        return r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(8, 1 + len(jobs))) as ex:
        marshal = ex.submit(_build_marshal, force, verbose)
        for err in ex.map(run, jobs):
            if ptxas_verbose and err:
                sys.stderr.write(err)
        built = marshal.result()
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".{os.getpid()}.tmp"
        run([nvcc, *ARCH, "-shared", "-Xlinker", "--no-undefined", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    if built:  # once the library that it calls is there
        os.replace(*built)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv))
