"""Compile libmsgl_attn.so in-tree with nvcc for sm_103a, and its native Python binding.

One translation unit per .cu file, compiled in parallel, then linked into
``paged_kv_attention_24_gb300/_build/libmsgl_attn.so``, which needs nothing but
the CUDA toolkit.  The binding (``csrc/python/binding.cpp``) is compiled against the
installed torch's headers and becomes ``_build/_msgl_binding-*.so`` beside it,
named after the torch and the Python it was built for; without torch it is left
out.  Each is built again when it is older than a source or header of its own.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import re
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libmsgl_attn.so")
BINDING_SRC = os.path.join(CSRC, "python", "binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
                     "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmsgl_attn")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _deps() -> list[str]:
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)])


def _torch():
    """torch, or None where it is not installed."""
    try:
        import torch
        return torch
    except ImportError:
        return None


def binding_path() -> str | None:
    """Where the binding for the installed torch and the running Python is; None without torch.

    It uses torch's C++ headers, so that one built for another version or ABI must not be loaded.
    """
    torch = _torch()
    if torch is None:
        return None
    abi = "cxx11" if torch._C._GLIBCXX_USE_CXX11_ABI else "cxx98"
    name = f"torch{torch.__version__}-{abi}-{sysconfig.get_config_var('SOABI')}"
    return os.path.join(BUILD, f"_msgl_binding-{re.sub('[^A-Za-z0-9_.+-]', '_', name)}.so")


def _newer(path: str, deps: list[str]) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path) for p in deps)


def _binding_up_to_date() -> bool:
    path = binding_path()
    return path is None or _newer(path, [BINDING_SRC, os.path.join(ROOT, "include", "msgl_attn.h"),
                                         os.path.abspath(__file__)])


def up_to_date() -> bool:
    return _newer(LIB, _deps()) and _binding_up_to_date()


def _run(cmd: list[str], what: str) -> subprocess.CompletedProcess:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")
    return r


def _compile_binding(cc: str) -> str:
    torch = _torch()
    t = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(cc)))
    obj = os.path.join(BUILD, "binding.o")
    _run(["g++", "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden", "-c", BINDING_SRC, "-o", obj,
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(t, "include"),
          "-isystem", os.path.join(t, "include", "torch", "csrc", "api", "include"),
          "-isystem", os.path.join(cuda, "include")], f"g++ failed on {BINDING_SRC}")
    return obj


def _link_binding(obj: str) -> None:
    torch_lib = os.path.join(os.path.dirname(os.path.abspath(_torch().__file__)), "lib")
    path = binding_path()
    tmp = path + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, LIB, "-L", torch_lib, "-ltorch_python", "-ltorch", "-ltorch_cpu",
          "-ltorch_cuda", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{torch_lib}"],
         f"link of {os.path.basename(path)} failed")
    os.replace(tmp, path)


def build(verbose: bool = False, force: bool = False, extra_flags: list[str] | None = None) -> str:
    """Builds what is missing or old.  The library stands before a failure of the binding is raised."""
    make_lib = force or not _newer(LIB, _deps())
    make_binding = binding_path() is not None and (force or not _binding_up_to_date())
    if not make_lib and not make_binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    flags = NVCC_FLAGS + list(extra_flags or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.splitext(os.path.basename(src))[0] + ".o")
        r = _run([cc] + flags + ["-c", src, "-o", obj], f"nvcc failed on {src}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=max(2, min(len(sources()) + 1, os.cpu_count() or 1))) as ex:
        binding = ex.submit(_compile_binding, cc) if make_binding else None
        if make_lib:
            objs = list(ex.map(compile_one, sources()))
            tmp = LIB + f".tmp{os.getpid()}"
            _run([cc] + ARCH + ["-shared", "-Xlinker", "-soname=libmsgl_attn.so", "-o", tmp] + objs + ["-lcuda"],
                 "link failed")
            os.replace(tmp, LIB)
    if binding is not None:
        _link_binding(binding.result())
    return LIB


if __name__ == "__main__":
    import sys
    print(build(verbose=True, force="--force" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None))
