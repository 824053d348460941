"""Build the CUDA library ``libgdn_decode.so`` in-tree with nvcc (sm_103a).

Each translation unit compiles in its own process (in parallel), then nvcc
links them into one shared library against the shared CUDA runtime.  Beside it
g++ compiles the attention layers' binding for the installed PyTorch; without
it the package makes the same calls through ctypes.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libgdn_decode.so")
SOURCES = ["gdn_api.cu", "gdn_stream.cu", "gdn_conv.cu", "gdn_prefill.cu", "gdn_chunked.cu", "gdn_chunked_tc.cu",
           "kv_api.cu", "kv_pages.cu", "attn_prologue.cu", "attn_tc.cu", "attn_f32.cu",
           "linear_api.cu", "linear_attn.cu", "linear_attn_tc.cu", "linear_attn_f32.cu"]
HEADERS = [os.path.join(CSRC, "gdn_device.cuh"), os.path.join(CSRC, "gdn_ptx.cuh"),
           os.path.join(CSRC, "gdn_chunk_common.cuh"), os.path.join(CSRC, "attn_plan.cuh"),
           os.path.join(CSRC, "tc_ops.cuh"), os.path.join(CSRC, "linear_plan.cuh"),
           os.path.join(CSRC, "tf32_ops.cuh"),
           os.path.join(CSRC, "gdn_internal.h"),
           os.path.join(ROOT, "include", "gdn_decode.h")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC"]


def _find_nvcc():
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    return None


def _nvcc() -> str:
    nvcc = _find_nvcc()
    if nvcc is None:
        raise RuntimeError("nvcc not found: the GDN decode library needs the CUDA toolkit to build")
    return nvcc


def _stale() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    deps = [os.path.join(CSRC, s) for s in SOURCES] + HEADERS
    return any(os.path.getmtime(d) > t for d in deps)


def _newer(path: str, t: float) -> bool:
    return os.path.exists(path) and os.path.getmtime(path) >= t


BINDING_SOURCE = os.path.join(CSRC, "fast_binding.cpp")


def binding_path() -> str:
    """Where the binding for this interpreter and this PyTorch lies: it fits no other."""
    import sysconfig

    import torch
    return os.path.join(PKG, f"_fast_binding-torch{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")


def binding_fresh() -> bool:
    """Whether the binding is there and as new as its sources, whose calls it makes by address."""
    return _newer(binding_path(), _binding_sources_time())


def _binding_failed() -> str:
    """What the compiler said when the binding did not compile: it is asked again once the sources are newer."""
    return os.path.join(BUILD_DIR, os.path.basename(binding_path()) + ".failed")


def _binding_sources_time() -> float:
    return max(os.path.getmtime(f) for f in (BINDING_SOURCE, os.path.join(ROOT, "include", "gdn_decode.h")))


def _start_binding(force: bool):
    """The compiler's process for the binding, and where its output goes; None if it is up to date or cannot be made."""
    import sysconfig

    import torch
    path = binding_path()
    if not force and (binding_fresh() or _newer(_binding_failed(), _binding_sources_time())):
        return None
    gxx, nvcc = shutil.which("g++"), _find_nvcc()  # the toolkit's headers lie beside nvcc
    if not gxx or not nvcc or not os.access(PKG, os.W_OK):
        return None
    base = os.path.dirname(torch.__file__)
    inc = [sysconfig.get_paths()["include"], os.path.join(base, "include"),
           os.path.join(base, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")]
    tmp = path + f".tmp{os.getpid()}"
    cmd = [gxx, "-O2", "-std=c++17", "-fPIC", "-shared", *(f"-I{i}" for i in inc), BINDING_SOURCE, "-o", tmp,
           f"-L{os.path.join(base, 'lib')}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT), tmp, path


def _end_binding(started) -> None:
    if started is None:
        return
    proc, tmp, path = started
    out, _ = proc.communicate()
    if proc.returncode == 0:
        os.replace(tmp, path)
    else:
        os.makedirs(BUILD_DIR, exist_ok=True)
        with open(_binding_failed(), "wb") as f:
            f.write(out)
        print("the C++ binding did not build; the package calls through ctypes\n" + out.decode(errors="replace")[-2000:],
              file=sys.stderr)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link what is not up to date. Returns the library's path."""
    binding = _start_binding(force)
    try:
        return _build_library(force, verbose)
    finally:
        _end_binding(binding)


def _build_library(force: bool, verbose: bool) -> str:
    if not force and not _stale():
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        objs.append(obj)
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-c",
               os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append((src, out.decode(errors="replace")))
        elif verbose and out:
            print(out.decode(errors="replace"), file=sys.stderr)
    if failed:
        raise RuntimeError("nvcc failed:\n" + "\n".join(f"--- {s}\n{o}" for s, o in failed))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        raise RuntimeError("nvcc link failed:\n" + r.stdout.decode(errors="replace"))
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
