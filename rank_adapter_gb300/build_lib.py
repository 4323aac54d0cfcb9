"""Build the C-ABI shared library for sm_103a with nvcc (no cmake, no torch extension).

Each translation unit under ``csrc/`` compiles in parallel to an object in
``<repo>/_build/``; the objects link into ``_lib/librank_adapter_gb300.so``
inside this package, next to the binding that loads it. The native marshalling
of the mixture-of-experts calls (``binding/moe_binding.cpp``) compiles beside
them with g++ against the headers of Python and of the installed torch, and
links to the library as ``_lib/_moe_binding.so``. A rebuild happens only when a
source or header is newer than what was built, or, for the binding, when torch or
the interpreter is another than it was built for. Without a CUDA build of torch
only the library is built (users of the C ABI need no more).
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
BINDING_FOR = os.path.join(BUILD, "moe_binding.txt")  # the torch and interpreter it was built for

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


def _newer_than_all(built, files) -> bool:
    return os.path.exists(built) and all(os.path.getmtime(f) <= os.path.getmtime(built) for f in files)


def _library_current() -> bool:
    return _newer_than_all(LIB, _inputs() + [os.path.abspath(__file__)])


def _binding_current(target: str) -> bool:
    headers = [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    if not _newer_than_all(BINDING, [BINDING_SRC, os.path.abspath(__file__)] + headers) or not os.path.exists(BINDING_FOR):
        return False
    with open(BINDING_FOR) as f:
        return f.read() == target


def up_to_date() -> bool:
    torch_dir = _torch_dir()
    return _library_current() and (torch_dir is None or _binding_current(_binding_target(torch_dir)))


def _torch_dir():
    """The installed torch's folder (not imported: its headers and libraries are enough), None without CUDA support."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    path = list(spec.submodule_search_locations)[0]
    return path if os.path.exists(os.path.join(path, "lib", "libc10_cuda.so")) else None


def _binding_target(torch_dir: str) -> str:
    """What a built binding works with: this interpreter and the torch at torch_dir, with its version file's contents."""
    version = os.path.join(torch_dir, "version.py")
    text = ""
    if os.path.exists(version):
        with open(version) as f:
            text = f.read()
    return f"{sys.implementation.cache_tag}\n{torch_dir}\n{text}"


def _compile_binding(torch_dir):
    """Compile the marshalling to an object; returns (source, object, status, output, command)."""
    nvcc_root = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    inc = os.path.join(torch_dir, "include")
    obj = os.path.join(BUILD, "moe_binding.o")
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-I" + INCLUDE, "-I" + sysconfig.get_paths()["include"],
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(nvcc_root, "include"), "-c", BINDING_SRC, "-o", obj]
    p = subprocess.run(cmd, capture_output=True, text=True)
    return BINDING_SRC, obj, p.returncode, p.stdout + p.stderr, cmd


def _run(cmd, verbose, what):
    p = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or p.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + p.stdout + p.stderr)
    if p.returncode != 0:
        raise RuntimeError(what + " failed")


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile and link the library and the binding; returns the library's path. Raises on any compiler error."""
    torch_dir = _torch_dir()
    target = _binding_target(torch_dir) if torch_dir is not None else ""
    make_lib = force or not _library_current()
    make_binding = torch_dir is not None and (force or not _binding_current(target))
    if not make_lib and not make_binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc] + ARCH + NVCC_FLAGS + extra + ["-c", src, "-o", obj]
        p = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, p.returncode, p.stdout + p.stderr, cmd

    def checked(result, compiler):
        src, obj, rc, out, cmd = result
        if verbose or rc != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + out)
        if rc != 0:
            raise RuntimeError(f"{compiler} failed on {os.path.basename(src)}")
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_compile_binding, torch_dir) if make_binding else None
        objs = [checked(r, "nvcc") for r in ex.map(compile_one, sources())] if make_lib else []
        binding_obj = checked(binding.result(), "g++") if make_binding else None
    if make_lib:
        tmp = LIB + ".tmp"
        _run([nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs + ["-lpthread", "-ldl", "-lrt"], verbose,
             "linking librank_adapter_gb300.so")
        os.replace(tmp, LIB)
    if make_binding:
        tmp = BINDING + ".tmp"
        _run(["g++", "-shared", "-o", tmp, binding_obj, "-L" + LIBDIR, "-l:" + os.path.basename(LIB),
              "-L" + os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10",
              "-Wl,-rpath,$ORIGIN"], verbose, "linking _moe_binding.so")
        os.replace(tmp, BINDING)
        with open(BINDING_FOR, "w") as f:
            f.write(target)
    elif torch_dir is None:
        sys.stderr.write("no CUDA build of torch: the binding of the mixture-of-experts calls (_moe_binding.so) is not built\n")
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_verbose="--ptxas" in sys.argv))
