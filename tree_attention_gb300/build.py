"""Build step for the sm_103a shared library ``libtreeattn.so`` and the extension
module ``_binding.so``.

Compiles the CUDA translation units under ``csrc/`` in parallel with nvcc
for ``sm_103a`` only and links them (with the static CUDA runtime) into
``tree_attention_gb300/libtreeattn.so``.  The driver API is reached at run
time through ``cudaGetDriverEntryPointByVersion``, so the library loads on a
machine without a GPU driver.  The extension module (the compiled argument
checks of ``PagedCache``) is one C++ file against torch's and Python's headers,
linked to that library.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libtreeattn.so")
BINDING_PATH = os.path.join(PKG, "_binding.so")
BINDING_STAMP = os.path.join(BUILD_DIR, "binding.txt")
SOURCES = ["ta_api.cu", "ta_plan.cu", "ta_attn.cu", "ta_merge.cu", "ta_cache.cu", "ta_decode.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))
    return files


def _newer_than_inputs(path: str) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path)
                                        for f in _inputs())


def _binding_for() -> str:
    """What the extension module is compiled against, beside its sources."""
    import torch
    return f"torch {torch.__version__} {torch.__file__}\npython {sysconfig.get_config_var('EXT_SUFFIX')}\n"


def binding_up_to_date() -> bool:
    if not _newer_than_inputs(BINDING_PATH) or not os.path.exists(BINDING_STAMP):
        return False
    try:
        want = _binding_for()
    except ImportError:   # no torch: building the module will say so
        return False
    with open(BINDING_STAMP) as f:
        return f.read() == want


def up_to_date() -> bool:
    return _newer_than_inputs(LIB_PATH) and binding_up_to_date()


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _torch_dir(name: str) -> str:
    import torch
    return os.path.join(os.path.dirname(torch.__file__), name)


def _compile_binding() -> str:
    import torch
    inc = _torch_dir("include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    obj = os.path.join(BUILD_DIR, "ta_binding.o")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-Wall",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-isystem", inc,
          "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda,
          "-c", os.path.join(CSRC, "ta_binding.cpp"), "-o", obj], "g++ for ta_binding.cpp")
    return obj


def _link_binding(obj: str) -> None:
    tmp = BINDING_PATH + ".tmp"
    _run(["g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:libtreeattn.so", "-Wl,-rpath,$ORIGIN",
          "-L", _torch_dir("lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"],
         "linking _binding.so")
    os.replace(tmp, BINDING_PATH)
    with open(BINDING_STAMP, "w") as f:
        f.write(_binding_for())


def _link_library(nvcc: str, objs) -> None:
    tmp = LIB_PATH + ".tmp"
    _run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"], "link")
    os.replace(tmp, LIB_PATH)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link the library and the extension module; returns the
    library's path.  The library is in place before a failure of the module,
    which alone needs torch's headers, is raised."""
    all_of_it = force or bool(extra_flags)
    library = all_of_it or not _newer_than_inputs(LIB_PATH)
    module = all_of_it or not binding_up_to_date()
    if not library and not module:
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding) if module else None
        if library:
            _link_library(nvcc, list(ex.map(compile_one, SOURCES)))
    if module:
        _link_binding(binding.result())
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose=True, extra_flags=tuple(sys.argv[1:])))
