"""Build libmea_attn.so in-tree with nvcc for sm_100a.

    python -m exact_memory_efficient_b200.build [--force] [--verbose]

The library is a plain C-ABI shared object (see include/mea_attn.h); nothing
in it depends on torch.  Objects are compiled in parallel and linked with nvcc
(relocatable device code, so the per-device error word is shared by all
kernels).  The CUDA runtime is linked statically.

_binding.so beside it is the CPython binding of the rotary and paged-cache
entry points for torch tensors (csrc/binding.cpp), compiled against the torch
and Python of the running interpreter and linked to the library.  It needs g++
and their headers; without them the library is built alone.
"""

from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG_DIR, "_build")
LIB_NAME = "libmea_attn.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)

SOURCES = ["api.cu", "fwd_f32.cu", "bwd_f32.cu", "fwd_bf16.cu", "fwd_persist.cu", "bwd_bf16.cu", "combine.cu", "decode.cu",
           "api_paged.cu", "rope.cu", "paged_attn.cu", "paged_tc.cu", "paged_weights.cu", "paged_weights_tc.cu", "paged_evict.cu"]
HEADERS = ["ptx.cuh", "kernels.h", "simt_f32.cuh", "rows.cuh", "paged.cuh", "api_internal.h"]

BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING_PATH = os.path.join(PKG_DIR, "_binding.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-rdc=true", "-Xcompiler", "-fPIC",
              "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _newest_input_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(INCLUDE, "mea_attn.h"),
                                                                  os.path.abspath(__file__)]
    return max(os.path.getmtime(f) for f in files)


def needs_build() -> bool:
    return not os.path.exists(LIB_PATH) or os.path.getmtime(LIB_PATH) < _newest_input_mtime()


def _compile(nvcc: str, src: str, verbose: bool, extra: list[str]) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0 or verbose:
        sys.stderr.write(r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}")
    return obj


def binding_tag() -> str:
    """The Python and torch of this interpreter, as text that a binding built for them holds."""
    import torch
    return (f"_binding for {sysconfig.get_config_var('SOABI')}, torch {torch.__version__} {torch.version.git_version}, "
            f"cxx11 abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)}")


def binding_fits() -> bool:
    """Whether _binding.so was built for this interpreter (found in the file: one of another ABI cannot be asked)."""
    try:
        with open(BINDING_PATH, "rb") as f:
            return binding_tag().encode() + b"\0" in f.read()
    except FileNotFoundError:
        return False


def needs_binding() -> bool:
    src = max(os.path.getmtime(f) for f in (BINDING_SRC, os.path.join(INCLUDE, "mea_attn.h"), os.path.abspath(__file__)))
    return not binding_fits() or os.path.getmtime(BINDING_PATH) < src


def binding_lacks() -> list[str]:
    """What is not installed of what _binding.so needs beside the library."""
    try:
        import torch
    except ImportError:
        return ["torch"]
    headers = {"Python.h": sysconfig.get_paths()["include"],
               "ATen/ATen.h": os.path.join(os.path.dirname(torch.__file__), "include")}
    return [h for h, at in headers.items() if not os.path.exists(os.path.join(at, h))] + \
        ([] if shutil.which("g++") else ["g++"])


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Compile _binding.so (needs the library)."""
    if not force and not needs_binding():
        return BINDING_PATH
    lacks = binding_lacks()
    if lacks:
        raise RuntimeError(f"_binding.so needs {', '.join(lacks)}")
    import torch
    torch_dir = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    includes = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
    tmp = BINDING_PATH + ".tmp"
    cmd = [shutil.which("g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DMEA_BINDING_FOR="{binding_tag()}"',
           *[x for p in includes for x in ("-isystem" if p != INCLUDE else "-I", p)], BINDING_SRC, "-o", tmp,
           "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           "-L", PKG_DIR, f"-l:{LIB_NAME}", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0 or verbose:
        sys.stderr.write(r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError("g++ failed on binding.cpp")
    os.replace(tmp, BINDING_PATH)
    return BINDING_PATH


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    """The library, and the binding where what it needs is installed (the library needs nvcc alone)."""
    _build_library(force, verbose, extra)
    lacks = binding_lacks()
    if lacks and ("torch" in lacks or force or needs_binding()):
        sys.stderr.write(f"_binding.so is not built without {', '.join(lacks)}: the rotary and paged-cache functions of "
                         "the Python package need it\n")
    elif not lacks:
        build_binding(force, verbose)
    return LIB_PATH


def _build_library(force: bool, verbose: bool, extra: list[str] | None) -> str:
    if not force and not needs_build():
        return LIB_PATH
    nvcc = nvcc_path()
    os.makedirs(BUILD_DIR, exist_ok=True)
    extra = list(extra or [])
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(nvcc, s, verbose, extra), SOURCES))
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-rdc=true", "-Xcompiler", "-fPIC", *objs, "-o", tmp, "-lcudart_static",
           "-lrt", "-ldl", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("nvcc link failed")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, verbose=args.verbose))


if __name__ == "__main__":
    main()
