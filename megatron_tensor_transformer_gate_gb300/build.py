"""Build ``libtp.so`` in-tree with nvcc for sm_103a.

Each translation unit is compiled in parallel; an object is rebuilt when its
source or any header under ``csrc/`` or ``include/`` is newer.  The CUDA
runtime is linked statically and the driver is reached through the runtime's
entry-point query, so the library loads (and reports its symbols) on a
machine without a GPU driver.
"""

import concurrent.futures
import glob
import importlib.metadata
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
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libtp.so")

SOURCES = ["api.cu", "gemm_tc.cu", "gemm_simt.cu", "elementwise.cu",
           "attn_fwd_tc.cu", "attn_bwd_tc.cu", "fp8.cu", "fp8_block.cu",
           "gemm_fp8_block.cu", "gemm_fp8_block_thin.cu", "account.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                "-Xcompiler", "-O3", "-I", INCLUDE]


def nvcc():
    exe = shutil.which("nvcc")
    if exe is None:
        cand = "/usr/local/cuda/bin/nvcc"
        if os.path.exists(cand):
            return cand
        raise RuntimeError("nvcc not found")
    return exe


def _headers_mtime():
    hs = glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(
        os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return max((os.path.getmtime(h) for h in hs), default=0.0)


def _compile(src, verbose=False):
    path = os.path.join(CSRC, src)
    obj = os.path.join(BUILD, src + ".o")
    newest = max(os.path.getmtime(path), _headers_mtime())
    if os.path.exists(obj) and os.path.getmtime(obj) >= newest:
        return obj, None
    cmd = [nvcc()] + FLAGS + ["-c", path, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, (r.stdout + r.stderr).strip() or None


def pycall_path():
    """The CPython module beside the binding.  It reads torch's own objects, so
    its name says which Python and which torch it was built against."""
    return os.path.join(PKG, "_tpcall-torch" +
                        importlib.metadata.version("torch") +
                        sysconfig.get_config_var("EXT_SUFFIX"))


def _build_pycall():
    """Compile that module (host code).  Returns None, or why there is none:
    everything works without it, the block-scaled calls some 4 µs slower."""
    try:
        path = pycall_path()
    except importlib.metadata.PackageNotFoundError:
        return "torch not found"
    src = os.path.join(CSRC, "pycall.cpp")
    if os.path.exists(path) and os.path.getmtime(path) >= max(
            os.path.getmtime(src), os.path.getmtime(__file__)):
        return None
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        return "g++ not found"
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = path + ".tmp"
    r = subprocess.run(
        [cxx, "-O2", "-std=c++17", "-shared", "-fPIC", src, "-o", tmp,
         "-I", sysconfig.get_paths()["include"],
         "-I", os.path.join(torch, "include"),
         "-I", os.path.join(torch, "include", "torch", "csrc", "api",
                            "include"),
         "-I", os.path.join(cuda, "include"),
         "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu",
         "-lc10", "-lc10_cuda"], capture_output=True, text=True)
    if r.returncode != 0:
        return f"{cxx} failed for pycall.cpp:\n{r.stdout}\n{r.stderr}"
    os.replace(tmp, path)
    return None


def build(verbose=False, jobs=None):
    """Compile every source and link ``libtp.so``; returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    jobs = jobs or min(len(SOURCES) + 1, os.cpu_count() or 4)
    with concurrent.futures.ThreadPoolExecutor(jobs) as ex:
        pycall = ex.submit(_build_pycall)
        results = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
        missing = pycall.result()
    if missing:
        print(f"the module of the block-scaled calls is not built: {missing}",
              file=sys.stderr)
    objs = [o for o, _ in results]
    if verbose:
        for o, log in results:
            if log:
                print(f"== {os.path.basename(o)}\n{log}", file=sys.stderr)
    newest = max(os.path.getmtime(o) for o in objs)
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < newest:
        tmp = LIB + ".tmp"
        cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
