"""Build libnvfp4kv.so in-tree with nvcc for sm_103a (GB300), and the Python module beside it
that carries the decode-step calls from torch tensors to the library (calls.cpp, with g++).

Each translation unit under csrc/ is compiled in parallel, then linked into one shared
library next to this file. A stamp of the sources and flags skips rebuilds when nothing
changed.
"""

from __future__ import annotations

import concurrent.futures as cf
import hashlib
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libnvfp4kv.so")
CALLS_PATH = os.path.join(HERE, "nvfp4kv_calls.so")
CALLS_SOURCE = "calls.cpp"
SOURCES = ["abi.cu", "append.cu", "dequant.cu", "materialize.cu", "global_scale.cu",
           "norm_rope.cu", "attention.cu", "pages.cu"]
HEADERS = ["device.cuh", "internal.h", "scan.cuh", "pipeline.cuh", "quantize.cuh",
           "attention.h"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", *ARCH, "-lineinfo", "-fmad=false", "--extended-lambda",
              "-Xcompiler", "-fPIC,-fvisibility=hidden,-O2", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    cand = [shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"]
    for c in cand:
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libnvfp4kv")


def _calls_command() -> list:
    """g++ on calls.cpp against this interpreter's and this torch's headers."""
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    includes = [sysconfig.get_paths()["include"], os.path.join(base, "include"),
                os.path.join(base, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-w",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *(f"-isystem{i}" for i in includes), "-c", os.path.join(CSRC, CALLS_SOURCE)]


def _calls_link(obj: str, out: str) -> list:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    return ["g++", "-shared", obj, "-o", out, f"-L{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
            f"-L{HERE}", "-l:" + os.path.basename(LIB_PATH), "-Wl,-rpath,$ORIGIN"]


def _stamp() -> str:
    import torch
    h = hashlib.sha256()
    h.update(f"{torch.__version__} {sysconfig.get_python_version()}".encode())
    for name in SOURCES + HEADERS + [CALLS_SOURCE]:
        with open(os.path.join(CSRC, name), "rb") as f:
            h.update(name.encode() + f.read())
    with open(os.path.join(ROOT, "include", "nvfp4kv.h"), "rb") as f:
        h.update(f.read())
    h.update(" ".join(NVCC_FLAGS).encode())
    return h.hexdigest()


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if stale) and return the path of libnvfp4kv.so."""
    stamp = _stamp()
    stamp_file = os.path.join(BUILD_DIR, "stamp")
    if not force and os.path.exists(LIB_PATH) and os.path.exists(CALLS_PATH) and os.path.exists(stamp_file):
        with open(stamp_file) as f:
            if f.read() == stamp:
                return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    exe = nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        if src == CALLS_SOURCE:
            cmd = [*_calls_command(), "-o", obj]
        else:
            cmd = [exe, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
            if verbose:
                cmd += ["-Xptxas", "-v"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{cmd[0]} failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        *objs, calls = ex.map(compile_one, SOURCES + [CALLS_SOURCE])
    tmp = LIB_PATH + ".tmp"
    r = subprocess.run([exe, "-shared", *ARCH, "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    tmp = CALLS_PATH + ".tmp"
    r = subprocess.run(_calls_link(calls, tmp), capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS_PATH)
    with open(stamp_file, "w") as f:
        f.write(stamp)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
