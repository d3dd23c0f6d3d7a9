"""Builds libpagedattn.so for sm_103a with nvcc.

Each translation unit in ``csrc/`` is compiled in parallel to an object file
under ``_build/`` and the objects are linked into ``_lib/libpagedattn.so``
(in-tree, so the test and benchmark processes load this exact file).  The
compiled part of the Python binding (``binding/``, a plain extension module that
takes torch tensors) is built beside it with g++ against the installed torch.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from importlib import metadata
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIBDIR = os.path.join(HERE, "_lib")
LIB = os.path.join(LIBDIR, "libpagedattn.so")
BINDING = os.path.join(HERE, "binding", "pa_ops_binding.cpp")
OPS = os.path.join(LIBDIR, "_pa_ops.so")
OPS_FOR = os.path.join(LIBDIR, "_pa_ops.for")  # the torch and the Python that OPS was built for

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-DNDEBUG"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp")))


def _lib_deps():
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "pagedattn.h")]


def _newer(path: str, deps) -> bool:
    return os.path.exists(path) and os.path.getmtime(path) >= max(os.path.getmtime(f) for f in deps)


def binding_target() -> str:
    """The torch and the Python the compiled binding is for: it calls both by their C++ and C interfaces, which differ
    between versions."""
    return "torch %s, %s" % (metadata.version("torch"), sysconfig.get_config_var("EXT_SUFFIX"))


def binding_built_for() -> str:
    try:
        with open(OPS_FOR) as f:
            return f.read()
    except OSError:
        return ""


def binding_fresh() -> bool:
    return _newer(OPS, [BINDING, os.path.join(INCLUDE, "pagedattn.h")]) and binding_built_for() == binding_target()


def _compile_binding() -> str:
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    obj = os.path.join(BUILD, "pa_ops_binding.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-DNDEBUG",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
           "-I", INCLUDE, "-I", sysconfig.get_paths()["include"]]
    for inc in (os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                os.path.join(cuda, "include")):
        cmd += ["-isystem", inc]
    r = subprocess.run(cmd + ["-c", BINDING, "-o", obj], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for %s:\n%s\n%s" % (BINDING, r.stdout, r.stderr))
    return obj


def _link_binding(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = OPS + ".%d.tmp" % os.getpid()
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", LIBDIR, "-l:libpagedattn.so", "-L", libs, "-ltorch_python",
           "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-Wl,-rpath,$ORIGIN:" + libs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link of the binding failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, OPS)
    tmp = OPS_FOR + ".%d.tmp" % os.getpid()
    with open(tmp, "w") as f:
        f.write(binding_target())
    os.replace(tmp, OPS_FOR)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compiles what is out of date (the library if a source of it is newer, the binding too if it was built for another
    torch or Python) and returns the library path."""
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    if not force and not ptxas_info and _newer(LIB, _lib_deps()):
        if not binding_fresh():
            _link_binding(_compile_binding())
        return LIB
    exe = nvcc()
    srcs = _sources()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.splitext(os.path.basename(src))[0] + ".o")
        cmd = [exe, *ARCH, *NVCC_FLAGS, "-I", INCLUDE, "-c", src, "-o", obj]
        if ptxas_info:
            cmd += ["-Xptxas", "-v"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        if verbose or ptxas_info:
            sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(compile_one, srcs))
        binding = binding.result()
    tmp = LIB + ".%d.tmp" % os.getpid()
    cmd = [exe, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    _link_binding(binding)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="-v" in sys.argv))
