"""Builds librope_gb300.so in-tree with nvcc for sm_103a.

The translation units compile in parallel (``nvcc -c``) and link into
one shared library with the CUDA runtime linked statically, so the library
loads on a machine without a GPU driver (every entry point then fails with
ROPE_ERR_CUDA once it reaches a CUDA call; argument checks still run).
"""

import glob
import hashlib
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_lib")
LIB_PATH = os.path.join(OUT_DIR, "librope_gb300.so")
SOURCES = ["rope_api.cu", "k_rope.cu", "k_mrope.cu", "k_fused.cu", "k_tma.cu", "k_qkv.cu", "k_mrope_qkv.cu", "k_qkv_tma.cu", "k_mrope_qkv_tma.cu",
           "k_mrope_heads.cu", "k_qkv_heads.cu", "no_alloc.cu", "kv_api.cu", "k_kv_append.cu", "k_kv_simple.cu", "k_kv_token.cu", "k_kv_tile_f16.cu",
           "k_kv_tile_f16_fp8.cu", "k_kv_tile_bf16.cu", "k_kv_tile_bf16_fp8.cu", "paged_api.cu",
           "k_paged_append.cu", "k_paged_simple.cu", "k_paged_token.cu", "k_paged_tile_f16.cu", "k_paged_tile_bf16.cu",
           "k_paged_keep.cu"]
HEADERS = ["rope_kernels.cuh", "rope_internal.h", "rope_tma.cuh", "rope_qkv.cuh", "rope_qkv_tma.cuh", "rope_packed.cuh", "rope_fused.cuh",
           "rope_mrope_heads.cuh", "rope_qkv_heads.cuh", "kv_internal.h", "kv_common.cuh", "kv_append.cuh", "kv_simple.cuh", "kv_careful.cuh", "kv_token.cuh", "kv_tile.cuh", "kv_maps.h", "kv_host.h",
           "paged_internal.h", "paged_common.cuh", "paged_append.cuh", "paged_append_heads.cuh", "paged_simple.cuh", "paged_careful.cuh", "paged_token.cuh",
           "paged_tile.cuh", "paged_maps.h", "paged_keep.cuh"]
BINDING = os.path.join(CSRC, "binding.cpp")


def _torch_version():
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return "none"


_SUFFIX = sysconfig.get_config_var("EXT_SUFFIX") or ".so"


def binding_path(sources, out_dir=OUT_DIR):
    """Where the short way made of these sources lies. What was compiled of others is not found, and not loaded: of
    another PyTorch its classes may be laid out differently, of another header the library's calls."""
    h = hashlib.sha256()
    for f in sources:
        if os.path.exists(f):  # (a package without its sources has no short way)
            with open(f, "rb") as s:
                h.update(s.read())
    return os.path.join(out_dir, f"_binding-torch{_torch_version()}-{h.hexdigest()[:16]}{_SUFFIX}")


BINDING_SOURCES = (BINDING, os.path.join(INCLUDE, "rope.h"))
BINDING_PATH = binding_path(BINDING_SOURCES)
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path():
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build librope_gb300.so")


def _inputs():
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    files.append(os.path.join(INCLUDE, "rope.h"))
    files.append(os.path.abspath(__file__))
    return files


def build_binding(force=False):
    """Compile (if needed) the short way into the library for calls with PyTorch tensors, csrc/binding.cpp, and
    return its path; None where it cannot be compiled (calls then go through ctypes)."""
    path = binding_path(BINDING_SOURCES, OUT_DIR)
    if not force and os.path.exists(path):
        return path
    try:
        torch = list(importlib.util.find_spec("torch").submodule_search_locations)[0]
        os.makedirs(OUT_DIR, exist_ok=True)
        tmp = path + f".tmp{os.getpid()}"
        cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include")
        cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-D_GLIBCXX_USE_CXX11_ABI=1",
               "-I", os.path.join(torch, "include"), "-I", os.path.join(torch, "include/torch/csrc/api/include"),
               "-I", sysconfig.get_paths()["include"], "-I", INCLUDE, "-I", cuda, BINDING, "-o", tmp,
               "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(r.stderr)
        os.replace(tmp, path)
        for old in glob.glob(os.path.join(OUT_DIR, f"_binding-torch{_torch_version()}*{_SUFFIX}")):
            if old != path:  # of sources that are gone
                os.remove(old)
        return path
    except Exception as e:  # no PyTorch, no Python.h, no g++: the library works without it
        sys.stderr.write(f"binding.cpp was not compiled, calls go through ctypes: {e}\n")
        return None


def up_to_date(path=LIB_PATH):
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build_library(force=False, extra_flags=(), out_path=None, verbose=False):
    """Compile (if needed) and return the path of the shared library."""
    out_path = out_path or LIB_PATH
    binding = out_path == LIB_PATH
    if not force and not extra_flags and up_to_date(out_path):
        if binding:
            build_binding()
        return out_path
    nvcc = nvcc_path()
    obj_dir = os.path.join(os.path.dirname(out_path), f"_obj{os.getpid()}")
    os.makedirs(obj_dir, exist_ok=True)
    common = [nvcc, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
              "-I", INCLUDE, "-I", CSRC, *extra_flags]
    if verbose:
        common += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(obj_dir, os.path.splitext(src)[0] + ".o")
        cmd = common + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        if binding:
            ex.submit(build_binding)
        results = list(ex.map(compile_one, SOURCES))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = out_path + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out_path)
    shutil.rmtree(obj_dir, ignore_errors=True)
    return out_path


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose="-v" in sys.argv))
