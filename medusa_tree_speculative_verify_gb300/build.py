"""Builds libmedusa_verify.so in-tree with nvcc for sm_103a (GB300).

Each .cu under csrc/ is compiled in parallel into _build/, then linked into
medusa_tree_speculative_verify_gb300/libmedusa_verify.so against the shared
CUDA runtime. Beside it _calls.so, the compiled part of the Python binding, is
made from csrc/calls.cpp with the host compiler and torch's headers. A rebuild
happens only when a source or header is newer than either (or when forced).
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmedusa_verify.so")
CALLS_SRC = os.path.join(CSRC, "calls.cpp")
CALLS = os.path.join(PKG, "_calls.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC,-O2",
         "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmedusa_verify.so")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def torch_dir() -> str:
    """Where torch is installed (it is not imported: that takes seconds)."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        raise RuntimeError("torch not found: the Python binding is compiled against its headers")
    return list(spec.submodule_search_locations)[0]


def calls_commands(obj: str, out: str):
    """The compile and the link of _calls.so."""
    torch = torch_dir()
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    cxx = os.environ.get("CXX") or shutil.which("g++") or "c++"
    include = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
    libs = os.path.join(torch, "lib")
    return ([cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *(f"-I{d}" for d in include), "-c", CALLS_SRC, "-o", obj],
            [cxx, "-shared", obj, "-o", out, f"-L{PKG}", "-l:libmedusa_verify.so", f"-L{libs}", "-lc10", "-lc10_cuda", "-ltorch_cpu",
             "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"])


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(CALLS):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(CALLS))
    deps = [CALLS_SRC] + sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    deps += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)] + [os.path.abspath(__file__)]
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link the library if needed; returns its path."""
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    calls_obj, calls_tmp = os.path.join(BUILD, "calls.cpp.o"), CALLS + ".tmp"
    compile_calls, link_calls = calls_commands(calls_obj, calls_tmp)
    jobs = min(len(sources()) + 1, os.cpu_count() or 4)
    with ThreadPoolExecutor(jobs) as ex:
        calls = ex.submit(subprocess.run, compile_calls, capture_output=True, text=True)
        results = list(ex.map(compile_one, sources()))
        results_calls = [(CALLS_SRC, calls_obj, calls.result())]
    failed = [(s, r) for s, _, r in results + results_calls if r.returncode != 0]
    for s, _, r in results + results_calls:
        if verbose or ptxas_info or r.returncode != 0:
            sys.stderr.write(f"== {os.path.basename(s)}\n{r.stdout}{r.stderr}")
    if failed:
        raise RuntimeError("compilation failed for: " + ", ".join(os.path.basename(s) for s, _ in failed))
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp] + [o for _, o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, LIB)
    r = subprocess.run(link_calls, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    os.replace(calls_tmp, CALLS)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
