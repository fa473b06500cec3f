"""Which prompts' rows go to the kernel of single tokens (csrc/attention_sizes.h), on the CPU: never more than its 32-bit
counts hold."""
import ctypes
import os
import shutil
import subprocess

import pytest

import nvfp4_paged_kv_02_gb300 as nv

CSRC = os.path.join(os.path.dirname(nv.__file__), "csrc")
PROGRAM = r"""
#include "attention_sizes.h"
extern "C" int32_t few(int64_t rows, int32_t head_dim, int32_t batch, int32_t kv_heads, int64_t reach) {
  return nvfp4::few_rows_of(rows, head_dim, batch, kv_heads, reach);
}
extern "C" int countable(int64_t lists, int64_t reach) { return nvfp4::places_countable(lists, reach); }
"""


@pytest.fixture(scope="module")
def sizes(tmp_path_factory):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("needs g++")
    d = tmp_path_factory.mktemp("sizes")
    (d / "sizes.cpp").write_text(PROGRAM)
    r = subprocess.run([gxx, "-O1", "-std=c++17", "-Wall", "-shared", "-fPIC", "-I", CSRC, str(d / "sizes.cpp"), "-o", str(d / "sizes.so")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(str(d / "sizes.so"))
    i32, i64 = ctypes.c_int32, ctypes.c_int64
    lib.few.argtypes, lib.countable.argtypes = [i64, i32, i32, i32, i64], [i64, i64]
    return lib


MOST = 2 ** 31 - 512  # positions of a request


@pytest.mark.parametrize("batch,heads,reach", [
    (16384, 1, MOST), (16384, 1, 2 ** 29), (16384, 8, 2 ** 26), (16384, 128, 2 ** 22), (4096, 8, MOST), (512, 128, MOST), (1, 2 ** 17, MOST),
])
def test_what_it_cannot_count_stays(sizes, batch, heads, reach):
    # places of all lists of the largest lengths, and of the longest run of 152 CTAs
    assert batch * heads * ((reach - 1) // 32 + 1 + 9) > 2 ** 38
    for D in (64, 256):
        assert sizes.few(batch, D, batch, heads, reach) == 0


@pytest.mark.parametrize("batch,heads,reach", [(16384, 1, 2 ** 28), (16384, 8, 2 ** 25), (1, 8, MOST), (64, 8, MOST), (128, 128, 2 ** 28)])
def test_what_it_counts_goes(sizes, batch, heads, reach):
    assert batch * heads * ((reach - 1) // 32 + 1 + 9) // 152 < 2 ** 31
    assert sizes.countable(batch * heads, reach) and sizes.few(batch, 128, batch, heads, reach) == 8


def test_few_rows_on_average(sizes):
    few = lambda rows, D=128, B=4, H=8, reach=4096: sizes.few(rows, D, B, H, reach)  # noqa: E731
    assert few(32) == 8 and few(33) == 16 and few(64) == 16 and few(65) == 0
    assert few(32, D=144) == 8 and few(33, D=144) == 0
    assert few(32, reach=1024) == 0 and few(32, reach=1025) == 8
    assert few(1, B=1) == 8


def test_nothing_to_count(sizes):
    assert sizes.countable(0, MOST) and sizes.countable(1, 0)
