"""Build libpkv.so (the C-ABI CUDA library) in-tree with nvcc for sm_103a, and _pkv_torch.so (the
part of the Python binding that works on torch tensors) with the host compiler.

Each .cu file (and each host-only .cpp file) is compiled in parallel to an object file, then linked into a shared library
next to this file. cudart is linked statically; the driver API is reached at run time
through cudaGetDriverEntryPointByVersion, so no libcuda is needed at link time. The library needs
nvcc alone and is there also where the binding does not compile (an error all the same); without
torch there is no binding to build.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpkv.so")
BINDING_SRC = os.path.join(HERE, "binding", "pkv_torch.cpp")
BINDING = os.path.join(HERE, "_pkv_torch.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = os.path.join(cuda, "bin", "nvcc")
    return path if os.path.exists(path) else (shutil.which("nvcc") or "nvcc")


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(OBJ_DIR, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd[1:1] = ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and r.stderr:
        sys.stderr.write(r.stderr)
    return obj


def _compile_binding() -> str:
    import torch
    root = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    obj = os.path.join(OBJ_DIR, os.path.basename(BINDING_SRC) + ".o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-c", BINDING_SRC, "-o", obj, "-I", INCLUDE,
           "-isystem", sysconfig.get_paths()["include"], "-isystem", root, "-isystem",
           os.path.join(root, "torch", "csrc", "api", "include"), "-isystem",
           os.path.join(cuda, "include")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", libs, "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python", "-L", HERE, "-l:libpkv.so", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def _have_torch() -> bool:
    try:
        return importlib.util.find_spec("torch") is not None
    except ValueError:  # (sys.modules["torch"] is None)
        return False


def _torch_version() -> str:
    """What a binding is built for: another torch or Python needs another one."""
    return (f"torch {importlib.metadata.version('torch')} at "
            f"{importlib.util.find_spec('torch').origin}, python {sys.version}")


def _noted() -> str:
    return os.path.join(OBJ_DIR, os.path.basename(BINDING) + ".for")


def _note_binding() -> None:
    with open(_noted(), "w") as f:
        f.write(_torch_version())


def _older(path: str, deps: list[str]) -> bool:
    return not os.path.exists(path) or any(os.path.getmtime(d) > os.path.getmtime(path)
                                           for d in deps)


def _stale_lib() -> bool:
    return _older(LIB, glob.glob(os.path.join(CSRC, "*")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale_binding() -> bool:
    if not _have_torch():
        return False
    if _older(BINDING, glob.glob(os.path.join(INCLUDE, "*.h")) + [BINDING_SRC]):
        return True
    if not os.path.exists(_noted()):
        return True
    with open(_noted()) as f:
        return f.read() != _torch_version()


def _stale() -> bool:
    return _stale_lib() or _stale_binding()


def build(force: bool = False, verbose: bool = False) -> str:
    lib, binding = force or _stale_lib(), _have_torch() and (force or _stale_binding())
    if not lib and not binding:
        return LIB
    os.makedirs(OBJ_DIR, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))
    with cf.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        obj = ex.submit(_compile_binding) if binding else None
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs)) if lib else []
    if lib:
        tmp = LIB + f".tmp{os.getpid()}"
        r = subprocess.run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs], capture_output=True,
                           text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if obj:
        _link_binding(obj.result())
        _note_binding()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
