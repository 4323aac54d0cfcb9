"""Build the C-ABI shared library for sm_103a with nvcc (no cmake, no torch extension).

Each translation unit under ``csrc/`` compiles in parallel to an object in
``<repo>/_build/``; the objects link into ``_lib/librank_adapter_gb300.so``
inside this package, next to the binding that loads it. The native marshalling
of the mixture-of-experts calls (``binding/moe_binding.cpp``) compiles beside
them with g++ against the headers of Python and of the installed torch, and
links to the library as ``_lib/_moe_binding.so``. A rebuild happens only when a
source or header is newer than what was built.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "librank_adapter_gb300.so")
BINDING_SRC = os.path.join(PKG, "binding", "moe_binding.cpp")
BINDING = os.path.join(LIBDIR, "_moe_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I" + INCLUDE, "-I" + CSRC]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build the library")
    return cand


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _inputs():
    files = sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return files


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(BINDING)):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(f) <= t for f in _inputs() + [BINDING_SRC, os.path.abspath(__file__)])


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")  # not imported: its headers and libraries are enough
    if spec is None or not spec.submodule_search_locations:
        raise RuntimeError("torch not found: the binding of the mixture-of-experts calls is built against it")
    return list(spec.submodule_search_locations)[0]


def _compile_binding():
    """Compile the marshalling to an object; returns (source, object, status, output, command)."""
    nvcc_root = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    inc = os.path.join(_torch_dir(), "include")
    obj = os.path.join(BUILD, "moe_binding.o")
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-I" + INCLUDE, "-I" + sysconfig.get_paths()["include"],
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(nvcc_root, "include"), "-c", BINDING_SRC, "-o", obj]
    p = subprocess.run(cmd, capture_output=True, text=True)
    return BINDING_SRC, obj, p.returncode, p.stdout + p.stderr, cmd


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile and link the library; returns its path. Raises on any compiler error."""
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc] + ARCH + NVCC_FLAGS + extra + ["-c", src, "-o", obj]
        p = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, p.returncode, p.stdout + p.stderr, cmd

    objs = []
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_compile_binding)
        for src, obj, rc, out, cmd in ex.map(compile_one, sources()):
            if verbose or rc != 0:
                sys.stderr.write(" ".join(cmd) + "\n" + out)
            if rc != 0:
                raise RuntimeError(f"nvcc failed on {os.path.basename(src)}")
            objs.append(obj)
        src, binding_obj, rc, out, cmd = binding.result()
        if verbose or rc != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + out)
        if rc != 0:
            raise RuntimeError(f"g++ failed on {os.path.basename(src)}")
    tmp = LIB + ".tmp"
    cmd = [nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs + ["-lpthread", "-ldl", "-lrt"]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or p.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + p.stdout + p.stderr)
    if p.returncode != 0:
        raise RuntimeError("linking librank_adapter_gb300.so failed")
    os.replace(tmp, LIB)
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, binding_obj, "-L" + LIBDIR, "-l:" + os.path.basename(LIB),
           "-L" + os.path.join(_torch_dir(), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10",
           "-Wl,-rpath,$ORIGIN"]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or p.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + p.stdout + p.stderr)
    if p.returncode != 0:
        raise RuntimeError("linking _moe_binding.so failed")
    os.replace(tmp, BINDING)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_verbose="--ptxas" in sys.argv))
