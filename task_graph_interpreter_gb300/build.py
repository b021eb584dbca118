"""Build libmk.so in-tree with nvcc for sm_103a, and the CPython module of its
tensor-level calls (_calls.*.so) with the host compiler.

Each translation unit compiles in parallel into ``_build/``; the shared
libraries land next to this file.  No CMake, one -gencode.
"""
from __future__ import annotations

import os
import re
import shutil
import subprocess
import sys
import sysconfig
import types
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")          # graph, lowering, interpreter
OPS = os.path.join(HERE, "csrc_ops")       # operators that are called one by one
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libmk.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = [os.path.join(CSRC, f) for f in ("graph.cpp", "runtime.cu", "megakernel.cu", "noalloc.cu")] + \
          [os.path.join(OPS, f) for f in ("paged.cu", "paged_rows.cu", "paged_chunk.cu", "paged_attention.cu",
                                          "verify.cu")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def check_launch_registers(source: str, log: str) -> None:
    """The chunk kernel's warpgroups trade registers at run time, and their shares add up to exactly what it is
    launched with (kLaunchRegs of its source).  Another count by the compiler is an error of the build; the launch
    refuses it too."""
    want = int(re.search(r"kLaunchRegs = (\d+)", source).group(1))
    used = re.findall(r"Compiling entry function '\w*chunk_kernel\w*'(?:(?!Compiling entry).)*?Used (\d+) registers", log,
                      re.S)
    if not used or any(int(n) != want for n in used):
        raise RuntimeError(f"paged_chunk.cu: the chunk kernel has to be compiled to {want} registers, not to "
                           f"{', '.join(used) or 'an unknown number'}: set kLaunchRegs and the shares to this compiler's")


def _compile(src: str, verbose: bool) -> str:
    name = os.path.basename(src)
    obj = os.path.join(BUILD, os.path.splitext(name)[0] + ".o")
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O3",
           "-I", INCLUDE, "-I", CSRC, "-I", OPS, "-c", src, "-o", obj]
    if src.endswith(".cpp"):
        cmd[1:1] = ["-x", "cu"]
    if name == "paged_chunk.cu" or verbose and name == "megakernel.cu":
        cmd.append("-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {name}:\n{r.stdout}\n{r.stderr}")
    if name == "paged_chunk.cu":
        with open(src) as f:
            check_launch_registers(f.read(), r.stdout + r.stderr)
    if verbose and r.stderr:
        sys.stderr.write(r.stderr)
    return obj


def calls_path() -> str:
    """The CPython module of the tensor-level calls (csrc_ops/calls.cpp).  It is bound to the layouts of the Python and
    the PyTorch it was compiled against, so its name holds both: another environment on the same tree builds its own."""
    import torch
    tag = re.sub(r"[^0-9A-Za-z.]+", "_", f"torch{torch.__version__}")
    return os.path.join(HERE, f"_calls.{tag}{sysconfig.get_config_var('EXT_SUFFIX')}")


def _compile_calls() -> None:
    import torch
    base = os.path.dirname(torch.__file__)
    lib = os.path.join(base, "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    if not cxx:
        raise RuntimeError("no C++ compiler found")
    path = calls_path()
    tmp = path + ".tmp"
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           "-I", INCLUDE, "-isystem", os.path.join(base, "include"),
           "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"), "-isystem", cuda,
           "-isystem", sysconfig.get_paths()["include"], os.path.join(OPS, "calls.cpp"), "-o", tmp, "-L", lib,
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10_cuda", "-lc10", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the C++ compiler failed on calls.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)


def _link(objs: list[str]) -> None:
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def _stale(built: str, sources: list[str]) -> bool:
    return not os.path.exists(built) or any(os.path.getmtime(s) > os.path.getmtime(built) for s in sources)


def build(force: bool = False, verbose: bool = False) -> str:
    """Bring libmk.so and the module of the tensor-level calls up to date.  The library is linked whatever becomes of
    the module, which only PyTorch's users need: without PyTorch it is left out, and a failure to compile it is
    raised behind the link."""
    header, calls = os.path.join(INCLUDE, "mk.h"), os.path.join(OPS, "calls.cpp")
    sources = [os.path.join(d, f) for d in (CSRC, OPS) for f in os.listdir(d)]
    sources.remove(calls)
    lib_stale = force or _stale(LIB, [*sources, header])
    try:
        calls_stale = _stale(calls_path(), [calls, header]) or force
    except ImportError:
        calls_stale = False
    if not lib_stale and not calls_stale:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        compiled = ex.submit(_compile_calls) if calls_stale else None
        if lib_stale:
            _link(list(ex.map(lambda s: _compile(s, verbose), SOURCES)))
        if compiled:
            compiled.result()
    return LIB


class _Callable(types.ModuleType):
    """The package's attribute ``build`` is this module; calling it builds."""

    def __call__(self, force: bool = False, verbose: bool = False) -> str:
        return build(force=force, verbose=verbose)


sys.modules[__name__].__class__ = _Callable

if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
