"""Builds libmedusa_verify.so in-tree with nvcc for sm_103a (GB300).

Each .cu under csrc/ is compiled in parallel into _build/, then linked into
medusa_tree_speculative_verify_gb300/libmedusa_verify.so against the shared
CUDA runtime; that takes nvcc alone. Beside it _calls-<key>.so, the compiled
part of the Python binding, is made from csrc/calls.cpp with the host compiler
and torch's headers, where torch is installed; its name says for which torch and
interpreter. Each is rebuilt only when one of its own sources or headers is
newer (or when forced).
"""
from __future__ import annotations

import hashlib
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
    """The compile and the link of the binding."""
    torch = torch_dir()
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    cxx = os.environ.get("CXX") or shutil.which("g++") or "c++"
    include = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
    libs = os.path.join(torch, "lib")
    return ([cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *(f"-I{d}" for d in include), "-c", CALLS_SRC, "-o", obj],
            [cxx, "-shared", obj, "-o", out, f"-L{PKG}", "-l:libmedusa_verify.so", f"-L{libs}", "-lc10", "-lc10_cuda", "-ltorch_cpu",
             "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"])


def calls_path() -> str:
    """Where the binding for this torch and this interpreter lies. It has torch's structures and the interpreter's compiled in
    and torch's libraries as its run path, so that one made for others must not be loaded."""
    torch = torch_dir()
    with open(os.path.join(torch, "version.py"), encoding="utf-8") as f:
        made_for = (torch, f.read(), sys.version, sysconfig.get_config_var("EXT_SUFFIX"))
    key = hashlib.sha256(repr(made_for).encode()).hexdigest()[:12]
    return os.path.join(PKG, f"_calls-{key}{made_for[3]}")


def _older(path: str, deps) -> bool:
    return not os.path.exists(path) or any(os.path.getmtime(p) > os.path.getmtime(path) for p in deps)


def _headers():
    return [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)] + [os.path.abspath(__file__)]


def _library_stale() -> bool:
    return _older(LIB, sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + _headers())


def _calls_stale() -> bool:
    return _older(calls_path(), [CALLS_SRC] + _headers())


def _stale() -> bool:
    return _library_stale() or _calls_stale()


def _run(cmd, what: str, verbose: bool = False) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stderr.write(f"== {what}\n{r.stdout}{r.stderr}")
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed")


def build_library(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link the library if needed; returns its path."""
    if not force and not _library_stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    jobs = min(len(sources()), os.cpu_count() or 4)
    with ThreadPoolExecutor(jobs) as ex:
        results = list(ex.map(compile_one, sources()))
    failed = [(s, r) for s, _, r in results if r.returncode != 0]
    for s, _, r in results:
        if verbose or ptxas_info or r.returncode != 0:
            sys.stderr.write(f"== {os.path.basename(s)}\n{r.stdout}{r.stderr}")
    if failed:
        raise RuntimeError("nvcc failed for: " + ", ".join(os.path.basename(s) for s, _ in failed))
    tmp = LIB + ".tmp"
    _run([cc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp] + [o for _, o, _ in results], "link of libmedusa_verify.so")
    os.replace(tmp, LIB)
    return LIB


def _compile_calls(verbose: bool = False):
    """Compiles the binding; returns the link, which wants the library there."""
    os.makedirs(BUILD, exist_ok=True)
    path = calls_path()
    tmp = path + ".tmp"
    compile_cmd, link_cmd = calls_commands(os.path.join(BUILD, os.path.basename(path) + ".o"), tmp)
    _run(compile_cmd, "compilation of calls.cpp", verbose)

    def link():
        _run(link_cmd, f"link of {os.path.basename(path)}")
        os.replace(tmp, path)
    return link


def build_calls(force: bool = False, verbose: bool = False) -> str:
    """Compile and link the compiled part of the binding if needed, beside a library that is there; returns its path."""
    if force or _calls_stale():
        _compile_calls(verbose)()
    return calls_path()


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Build the library and, where torch is installed, the compiled part of the binding, if needed; returns the library's
    path. The library is there even where the binding could not be built."""
    with ThreadPoolExecutor(1) as ex:
        compiled = None
        if importlib.util.find_spec("torch") is not None and (force or _calls_stale()):
            compiled = ex.submit(_compile_calls, verbose)  # beside the library's kernels, which take longer
        build_library(force, verbose, ptxas_info)
    if compiled is not None:
        compiled.result()()
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
