"""Build the library ``libmoe_dispatch.so`` in-tree for sm_103a.

Each ``csrc/*.cu`` file is compiled to an object in parallel, then linked
into one shared library with the CUDA runtime linked statically (so the
library does not depend on which libcudart the process already loaded).
``csrc/torch_binding.cpp`` becomes ``_torch_binding.so``, a Python module that
calls the library on tensors of the installed torch; where there is no torch
with CUDA the library is all that is built.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_NAME = "libmoe_dispatch.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
BINDING_SRC = os.path.join(CSRC, "torch_binding.cpp")
BINDING_PATH = os.path.join(HERE, "_torch_binding.so")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
              "-Xptxas", "-warn-spills", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return cand


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return hs


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src, extra, verbose):
    obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
    if not _stale(obj, [src] + _headers() + [__file__]) and not extra:
        return obj
    cmd = [nvcc(), *ARCH_FLAGS, *NVCC_FLAGS, *extra, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj + ".tmp"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), res.stderr))
    if verbose and res.stderr.strip():
        sys.stderr.write(res.stderr)
    os.replace(obj + ".tmp", obj)
    return obj


def _torch_root():
    """The installed torch's folder; None without one that has CUDA."""
    try:
        import torch
    except ImportError:
        return None
    root = os.path.dirname(torch.__file__)
    return root if os.path.exists(os.path.join(root, "lib", "libtorch_cuda.so")) else None


def _compile_binding(root):
    """The object of the torch binding (compiled against the torch in `root`)."""
    import sysconfig
    obj = os.path.join(BUILD_DIR, "torch_binding.o")
    if not _stale(obj, [BINDING_SRC, __file__, os.path.join(root, "version.py")] + _headers()):
        return obj
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    includes = [INCLUDE, os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *["-I" + d for d in includes], "-c", BINDING_SRC,
           "-o", obj + ".tmp"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed for %s:\n%s\n%s" % (BINDING_SRC, " ".join(cmd), res.stderr))
    os.replace(obj + ".tmp", obj)
    return obj


def _link_binding(obj, root):
    if not _stale(BINDING_PATH, [obj, LIB_PATH]):
        return
    libs = os.path.join(root, "lib")
    tmp = BINDING_PATH + ".tmp%d" % os.getpid()
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", HERE, "-l:" + LIB_NAME, "-L", libs, "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + libs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), res.stderr))
    os.replace(tmp, BINDING_PATH)


def build(verbose: bool = False, extra_flags=None, force: bool = False) -> str:
    """Compile and link; returns the path of the shared library."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    extra = list(extra_flags or [])
    srcs = sources()
    if force:
        for f in os.listdir(BUILD_DIR):
            os.remove(os.path.join(BUILD_DIR, f))
    root = _torch_root()
    with cf.ThreadPoolExecutor(max_workers=min(10, len(srcs) + 1)) as ex:
        binding = ex.submit(_compile_binding, root) if root else None
        objs = list(ex.map(lambda s: _compile(s, extra, verbose), srcs))
    if _stale(LIB_PATH, objs) or extra or force:
        tmp = LIB_PATH + ".tmp%d" % os.getpid()
        cmd = [nvcc(), *ARCH_FLAGS, "-shared", "-cudart", "static", "-o", tmp, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), res.stderr))
        os.replace(tmp, LIB_PATH)
    if binding is not None:  # after the library, which does not need it
        _link_binding(binding.result(), root)
    return LIB_PATH


if __name__ == "__main__":
    v = "-v" in sys.argv
    flags = ["-Xptxas", "-v"] if v else []
    print(build(verbose=v, extra_flags=flags, force="--force" in sys.argv))
