"""Build libspecverify.so in-tree with nvcc for sm_103a (GB300).

Twelve translation units (verification, sampling, the LM-head-fused
verification, tree verification, tree attention, its plan and cache commit,
logits processing, chunk attention, its plan and append, beam selection, the
cache's pages, the benchmark's read probe), one -gencode, no cmake: each
is compiled by its own nvcc process in parallel, then one nvcc call links the
shared library.  The library links the CUDA runtime statically so it only
needs the driver at run time; PyTorch's own runtime is not involved.

Beside them, where PyTorch is installed, g++ compiles the Python binding's short way
into the library (csrc/calls.cpp) against PyTorch's headers.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
SRCS = [os.path.join(CSRC, "spec_verify.cu"), os.path.join(CSRC, "spec_sample.cu"),
        os.path.join(CSRC, "spec_lmhead.cu"), os.path.join(CSRC, "spec_tree.cu"),
        os.path.join(CSRC, "spec_attn.cu"), os.path.join(CSRC, "spec_cache.cu"),
        os.path.join(CSRC, "spec_logits.cu"), os.path.join(CSRC, "spec_chunk.cu"),
        os.path.join(CSRC, "spec_append.cu"), os.path.join(CSRC, "spec_beam.cu"),
        os.path.join(CSRC, "spec_pages.cu"), os.path.join(CSRC, "bench_read.cu")]
DEPS = [os.path.join(CSRC, "device_common.cuh"), os.path.join(CSRC, "attn_plan.cuh"),
        os.path.join(CSRC, "attn_common.cuh"), os.path.join(CSRC, "chunk_plan.cuh"), os.path.join(CSRC, "internal.h"),
        os.path.join(CSRC, "resolve.cuh"), os.path.join(CSRC, "exp2_table.h"),
        os.path.join(CSRC, "row_cut.h"),
        os.path.join(ROOT, "include", "spec_lmhead.h"),
        os.path.join(ROOT, "include", "spec_verify.h"),
        os.path.join(ROOT, "include", "spec_sample.h"),
        os.path.join(ROOT, "include", "spec_bench.h"),
        os.path.join(ROOT, "include", "spec_tree.h"),
        os.path.join(ROOT, "include", "spec_attn.h"),
        os.path.join(ROOT, "include", "spec_logits.h"),
        os.path.join(ROOT, "include", "spec_chunk.h"),
        os.path.join(ROOT, "include", "spec_beam.h"),
        os.path.join(ROOT, "include", "spec_pages.h")]
SRC = SRCS[0]
LIB = os.path.join(PKG, "libspecverify.so")
CALLS_SRC = os.path.join(CSRC, "calls.cpp")
CALLS_HEADER = os.path.join(ROOT, "include", "spec_verify.h")
CALLS = os.path.join(PKG, "_calls.so")
CALLS_FOR = CALLS + ".for"  # what it was compiled for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("CUDA_HOME"), os.environ.get("CUDA_PATH"), "/usr/local/cuda"):
        if cand and os.path.exists(os.path.join(cand, "bin", "nvcc")):
            return os.path.join(cand, "bin", "nvcc")
    found = shutil.which("nvcc")
    if not found:
        raise RuntimeError("nvcc not found: set CUDA_HOME")
    return found


def compile_command(src: str, obj: str, extra=()) -> list:
    return [nvcc_path(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-c",
            "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
            "-I", os.path.join(ROOT, "include"), *extra, "-o", obj, src]


def link_command(objs, out: str) -> list:
    return [nvcc_path(), *ARCH, "--shared", "-cudart", "static", "-o", out, *objs]


def calls_command(out: str):
    """None without PyTorch (which is looked for, not imported)."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    torch = spec.submodule_search_locations[0]
    lib = os.path.join(torch, "lib")
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    return ["g++", "-std=c++17", "-O2", "-Wall", "-fPIC", "-shared", "-fvisibility=hidden",
            "-I", os.path.join(ROOT, "include"), "-I", sysconfig.get_paths()["include"],
            "-isystem", os.path.join(torch, "include"),
            "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
            "-isystem", os.path.join(cuda, "include"), "-o", out, CALLS_SRC, "-L", lib,
            "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10",
            f"-Wl,-rpath,{lib}"]


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in (*SRCS, *DEPS, __file__))


def calls_made_for():
    """What _calls.so depends on besides its sources: PyTorch (whose C++ headers it is compiled
    against, inline functions and all) and this Python.  None without PyTorch."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    torch = spec.submodule_search_locations[0]
    try:
        with open(os.path.join(torch, "version.py")) as f:
            version = f.read()
    except OSError:
        version = ""
    return "\n".join((torch, version, sysconfig.get_config_var("SOABI") or "", ""))


def calls_match() -> bool:
    """Whether _calls.so was compiled for this PyTorch and Python."""
    try:
        with open(CALLS_FOR) as f:
            return os.path.exists(CALLS) and f.read() == calls_made_for()
    except OSError:
        return False


def calls_stale() -> bool:
    if calls_made_for() is None:
        return False
    return not calls_match() or any(os.path.getmtime(p) > os.path.getmtime(CALLS)
                                    for p in (CALLS_SRC, CALLS_HEADER, __file__))


def _run(cmd, verbose):
    res = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or res.returncode != 0:
        print(" ".join(cmd))
        print(res.stdout)
        print(res.stderr)
    return res.returncode


def build_calls(tag: str, verbose: bool) -> bool:
    """Compile the binding's short way.  Where that does not work (a PyTorch without CUDA or without
    headers, no Python.h, no g++) a line says so, an old one is taken away, and calls go through Python:
    the library does not hang on it."""
    tmp = CALLS + tag
    try:
        command = calls_command(tmp)
        if command is None:
            return False
        res = subprocess.run(command, capture_output=True, text=True)
        if verbose:
            print(" ".join(command), res.stdout, res.stderr, sep="\n")
        if res.returncode == 0:
            with open(tmp + ".for", "w") as f:
                f.write(calls_made_for())
            # (in this order: a build that is cut off between leaves none that passes for this one)
            if os.path.exists(CALLS_FOR):
                os.remove(CALLS_FOR)
            os.replace(tmp, CALLS)
            os.replace(tmp + ".for", CALLS_FOR)
            return True
        errors = [x for x in res.stderr.splitlines() if "error" in x] or res.stderr.splitlines()
        why = errors[0] if errors else f"g++ ended with {res.returncode}"
    except OSError as error:  # no g++
        why = str(error)
    for path in (tmp, tmp + ".for", CALLS_FOR, CALLS):
        if os.path.exists(path):
            os.remove(path)
    print(f"_calls.so is left out, calls go through Python: {why}")
    return False


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compile the CUDA library if it is missing or older than its sources, and the binding's
    short way into it likewise."""
    tag = f".tmp{os.getpid()}"
    calls = force or calls_stale()
    if not force and not stale() and not extra:
        if calls:
            build_calls(tag, verbose)
        return LIB
    objs = [os.path.join(CSRC, os.path.basename(s) + tag + ".o") for s in SRCS]
    try:
        with ThreadPoolExecutor(len(SRCS) + 1) as ex:
            if calls:
                ex.submit(build_calls, tag, verbose)
            rcs = list(ex.map(lambda so: _run(compile_command(so[0], so[1], extra), verbose),
                              zip(SRCS, objs)))
            if any(rcs):
                raise RuntimeError("nvcc failed compiling the CUDA sources")
            tmp = LIB + tag
            if _run(link_command(objs, tmp), verbose):
                raise RuntimeError("nvcc failed linking libspecverify.so")
            os.replace(tmp, LIB)
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose=True, extra=("-Xptxas", "-v"))
