"""Build libmsa.so in-tree with nvcc for sm_103a (GB300).

Each .cu file is compiled to an object in parallel, then linked into
``block_sparse_attention_prefill_gb300/_build/libmsa.so`` with the CUDA
runtime linked statically (the library needs only the driver at run time).
The driver entry point for TMA descriptors is looked up at run time, so the
library also loads on a machine without a GPU.

``csrc/binding.cpp``, the tree calls' way from Python to the library, is
compiled beside it with the C++ compiler against the installed PyTorch, into a
module of its own: the library itself does not know PyTorch.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import subprocess
import sys
import sysconfig
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_build")
LIB = os.path.join(OUT, "libmsa.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
         "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
         "-I", INCLUDE]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC)
                  if f.endswith(".cu"))


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC)
          if f.endswith((".cuh", ".h"))]
    hs.append(os.path.join(INCLUDE, "msa.h"))
    return hs


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _cuda_include() -> str:
    nvcc = _nvcc()
    home = os.path.dirname(os.path.dirname(nvcc)) if os.path.isabs(nvcc) else "/usr/local/cuda"
    return os.path.join(home, "include")


def binding_path() -> str:
    """The binding's module for this interpreter and PyTorch."""
    return os.path.join(OUT, "msa_binding-torch%s%s" % (importlib.metadata.version("torch"),
                                                        sysconfig.get_config_var("EXT_SUFFIX")))


_binding_lock = threading.Lock()


def build_binding(force: bool = False) -> str:
    """Compile the Python module if its source or the header is newer (threads
    that ask at once: one compiles, the others wait for it)."""
    with _binding_lock:
        return _build_binding(force)


def _build_binding(force: bool) -> str:
    os.makedirs(OUT, exist_ok=True)
    path, src = binding_path(), os.path.join(CSRC, "binding.cpp")
    if not force and not _stale(path, [src, os.path.join(INCLUDE, "msa.h"), __file__]):
        return path
    root = importlib.util.find_spec("torch").submodule_search_locations[0]
    torch, libs = os.path.join(root, "include"), os.path.join(root, "lib")
    tmp = path + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           "-fvisibility=hidden", "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-I", torch,
           "-I", os.path.join(torch, "torch", "csrc", "api", "include"), "-I", _cuda_include(), src,
           "-o", tmp, "-L", libs, "-Wl,-rpath," + libs, "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("the C++ compiler failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose: bool = False, ptxas_info=False) -> str:
    """Compile and link libmsa.so if any source or header is newer."""
    os.makedirs(OUT, exist_ok=True)
    srcs = sources()
    hdrs = _headers()
    if not force and not _stale(LIB, srcs + hdrs + [__file__]):
        return LIB
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(OUT, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s"
                               % (src, r.stdout, r.stderr))
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        results = list(ex.map(compile_one, srcs))
    if verbose or ptxas_info:
        for _, err in results:
            if err:
                sys.stderr.write(err)
    objs = [o for o, _ in results]
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                ptxas_info="--ptxas" in sys.argv))
