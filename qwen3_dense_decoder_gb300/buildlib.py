"""Build the sm_103a CUDA library (libq3.so) in-tree with nvcc.

Each translation unit under csrc/ compiles in parallel for
``-gencode arch=compute_103a,code=sm_103a``; the objects link into one shared
library with the CUDA runtime linked statically, so the library loads on a
host without a GPU (the CPU tests check its exported symbols).  The host
compiler builds csrc/bind.cpp, the asynchronous operators' Python side, into
the extension module _ops beside it.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libq3.so")
OPS = os.path.join(HERE, "_ops.so")

SOURCES = ["runtime.cu", "k_gemm.cu", "k_gemv.cu", "k_attn.cu", "k_attn_prefill.cu", "k_misc.cu",
           "noalloc.cu", "k_decode.cu", "k_attn_tc.cu", "k_gemv_a4.cu",
           "k_kv4.cu", "k_kv4_prefill.cu", "k_logprobs.cu",
           "k_i8_rows.cu", "k_i8_norm.cu", "k_i8_few.cu", "k_i8_matmul.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libq3.so")
    return path


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "q3.h"))
    return max(os.path.getmtime(f) for f in files)


def torch_dir() -> str:
    return os.path.dirname(importlib.util.find_spec("torch").origin)


def ops_stamp() -> str:
    """What _ops.so's binary interface depends on: this Python's and the installed torch's."""
    try:
        with open(os.path.join(torch_dir(), "version.py")) as f:
            version = f.read()
    except OSError:
        version = ""
    return f"{sysconfig.get_config_var('EXT_SUFFIX')}\n{torch_dir()}\n{version}"


def ops_stale(newest: float) -> bool:
    """Whether _ops.so is missing, older than its sources or made for another torch or Python."""
    if not os.path.exists(OPS) or os.path.getmtime(OPS) < newest:
        return True
    try:
        with open(OPS + ".stamp") as f:
            return f.read() != ops_stamp()
    except OSError:
        return True


def compile_ops() -> None:
    """csrc/bind.cpp into _ops.so, against the headers and libraries of the torch that will load it."""
    torch = torch_dir()
    libs = os.path.join(torch, "lib")
    includes = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
                os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include"),
                sysconfig.get_paths()["include"]]
    tmp = OPS + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-I", INCLUDE,
           *(x for d in includes for x in ("-isystem", d)), os.path.join(CSRC, "bind.cpp"), "-o", tmp,
           "-L", libs, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{libs}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on bind.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, OPS)
    with open(OPS + ".stamp", "w") as f:
        f.write(ops_stamp())


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    """Compile csrc/*.cu into libq3.so and csrc/bind.cpp into _ops.so (each skipped when up to date).

    The library and the model paths need nothing of torch's headers; where the
    extension cannot be built, that is written to stderr, and its operators
    raise when they are called."""
    newest = _deps_mtime()
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        ops = ex.submit(compile_ops) if force or ops_stale(newest) else None
        if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < newest:
            compile_lib(verbose, list(extra or []))
        try:
            if ops:
                ops.result()
        except Exception as e:
            if os.path.exists(OPS):
                os.remove(OPS)
            sys.stderr.write(f"_ops.so was not built: {e}\n")
    return LIB


def compile_lib(verbose: bool, extra: list[str]) -> None:
    """csrc/*.cu into libq3.so."""
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


FAULT_LIB = os.path.join(BUILD, "faults", "libq3_faults.so")


def build_fault_variant(force: bool = False) -> str:
    """The test build of the mutation gate: runtime.cu compiled with
    -DQ3_TEST_FAULTS (the host then plants the addressing fault named by the
    Q3_FAULT environment variable in what it uploads) and linked with the
    product's kernel objects into a separate library.  Never the product."""
    build()
    out_dir = os.path.dirname(FAULT_LIB)
    obj = os.path.join(out_dir, "runtime.o")
    src = os.path.join(CSRC, "runtime.cu")
    if not force and os.path.exists(FAULT_LIB) and os.path.getmtime(FAULT_LIB) >= os.path.getmtime(LIB):
        return FAULT_LIB
    os.makedirs(out_dir, exist_ok=True)
    cc = nvcc()
    r = subprocess.run([cc, *ARCH, *FLAGS, "-DQ3_TEST_FAULTS", "-c", src, "-o", obj], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on runtime.cu (fault build):\n{r.stdout}\n{r.stderr}")
    objs = [obj] + [os.path.join(BUILD, f.replace(".cu", ".o")) for f in SOURCES if f != "runtime.cu"]
    tmp = FAULT_LIB + f".tmp{os.getpid()}"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed (fault build):\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, FAULT_LIB)
    return FAULT_LIB


if __name__ == "__main__":
    v = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas" in sys.argv else None
    print(build(force=True, verbose=v or bool(extra), extra=extra))
