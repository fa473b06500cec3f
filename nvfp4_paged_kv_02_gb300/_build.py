"""Build libnvfp4kv.so in-tree with nvcc for sm_103a (GB300), and the Python module beside it
that carries the decode-step calls from torch tensors to the library (calls.cpp, with g++).

Each translation unit under csrc/ is compiled in parallel, then linked into one shared
library next to this file. A stamp of the sources and flags skips rebuilds when nothing
changed. The library needs nvcc alone (`python _build.py library`); the module has its own
stamp, and its failure leaves the library in place.
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
           "norm_rope.cu", "attention.cu", "pages.cu", "prefill.cu",
           "attention_sinks.cu", "attention_tokens.cu"]
HEADERS = ["device.cuh", "internal.h", "scan.cuh", "pipeline.cuh", "quantize.cuh",
           "attention.h", "attention.cuh", "softmax.cuh", "tcgen05.cuh", "prefill_tiles.h",
           "attention_sizes.h"]
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


def _digest(names: list, *more: str) -> str:
    h = hashlib.sha256()
    for name in names:
        with open(os.path.join(CSRC, name), "rb") as f:
            h.update(name.encode() + f.read())
    with open(os.path.join(ROOT, "include", "nvfp4kv.h"), "rb") as f:
        h.update(f.read())
    h.update(" ".join(more).encode())
    return h.hexdigest()


def _library_stamp() -> str:
    return _digest(SOURCES + HEADERS, *NVCC_FLAGS)


def _calls_stamp() -> str:
    import torch
    return _digest([CALLS_SOURCE], torch.__version__, sysconfig.get_python_version(), *_calls_command())


def _is_current(path: str, stamp_file: str, stamp: str) -> bool:
    if not (os.path.exists(path) and os.path.exists(stamp_file)):
        return False
    with open(stamp_file) as f:
        return f.read() == stamp


def _run(cmd: list, what: str, verbose: bool = False) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed on {what}:\n{r.stdout}\n{r.stderr}")
    if verbose and r.stderr:
        print(r.stderr)


def _obj(src: str) -> str:
    return os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")


def _put(path: str, tmp: str, stamp_file: str, stamp: str) -> None:
    os.replace(tmp, path)
    with open(stamp_file, "w") as f:
        f.write(stamp)


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile the C-ABI library (if stale) and return its path. It needs nvcc alone."""
    stamp, stamp_file = _library_stamp(), os.path.join(BUILD_DIR, "stamp")
    if not force and _is_current(LIB_PATH, stamp_file, stamp):
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    exe = nvcc()

    def compile_one(src: str) -> str:
        _run([exe, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", _obj(src),
              *(["-Xptxas", "-v"] if verbose else [])], src, verbose)
        return _obj(src)

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB_PATH + ".tmp"
    _run([exe, "-shared", *ARCH, "-o", tmp, *objs], "the library's link")
    _put(LIB_PATH, tmp, stamp_file, stamp)
    return LIB_PATH


def _compile_calls() -> None:
    os.makedirs(BUILD_DIR, exist_ok=True)
    _run([*_calls_command(), "-o", _obj(CALLS_SOURCE)], CALLS_SOURCE)


def build_calls(force: bool = False, compiled: bool = False) -> str:
    """Compile the decode-step calls' module (if stale) against this interpreter's and this torch's headers,
    and return its path; the library comes first. `compiled`: its object file is up to date."""
    stamp, stamp_file = _calls_stamp(), os.path.join(BUILD_DIR, "stamp_calls")
    if not force and _is_current(CALLS_PATH, stamp_file, stamp):
        return CALLS_PATH
    build_library()
    if not compiled:
        _compile_calls()
    tmp = CALLS_PATH + ".tmp"
    _run(_calls_link(_obj(CALLS_SOURCE), tmp), "the calls' link")
    _put(CALLS_PATH, tmp, stamp_file, stamp)
    return CALLS_PATH


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile what is stale of the library and the calls' module, side by side, and return the library's path.
    The library is there even where the module cannot be compiled (which raises)."""
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        stale = force or not _is_current(CALLS_PATH, os.path.join(BUILD_DIR, "stamp_calls"), _calls_stamp())
        calls = ex.submit(_compile_calls) if stale else None
        build_library(force, verbose)
        if calls:
            calls.result()
            build_calls(force=True, compiled=True)
    return LIB_PATH


if __name__ == "__main__":  # "library": the C ABI alone, without torch
    import sys
    print((build_library if sys.argv[1:] == ["library"] else build)(force=True, verbose=True))
