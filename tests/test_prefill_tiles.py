"""Which tiles the rows of a prompt see (csrc/prefill_tiles.h), on the CPU: the rule that the kernel's warps share,
compiled by the host's compiler, against the positions that every row sees by the definition of the masks."""
import ctypes
import os
import shutil
import subprocess

import pytest

import nvfp4_paged_kv_02_gb300 as nv

CSRC = os.path.join(os.path.dirname(nv.__file__), "csrc")
PROGRAM = r"""
#include "prefill_tiles.h"
#include <random>
#include <vector>
using namespace nvfp4;

// Tiles that rows [r0, r1) see, row by row: t < L; causal: t <= p; with a window: t >= p - window or t < sink.
static std::vector<char> seen(int64_t L, int64_t n, int64_t G, bool causal, int64_t window, int64_t sink, int64_t r0, int64_t r1, int BN) {
  std::vector<char> tiles(L / BN + 2, 0);
  auto mark = [&](int64_t a, int64_t b) {  // positions [a, b)
    if (a < 0) a = 0;
    if (a < b) for (int64_t j = a / BN; j <= (b - 1) / BN; ++j) tiles[j] = 1;
  };
  for (int64_t token = r0 / G; token <= (r1 - 1) / G; ++token) {
    const int64_t p = L - n + token, hi = causal ? (p + 1 < L ? p + 1 : L) : L;
    mark(window < 0 ? 0 : p - window, hi);
    mark(0, sink < hi ? sink : hi);
  }
  return tiles;
}

// 0, or which of the checks fails for a request of n tokens at L positions.
template <int BN>
static int check(int32_t L, int32_t n, int32_t G, bool causal, int32_t window, int32_t sink, std::mt19937& rng) {
  const int32_t rows = n * G, kRows = 256;
  for (int32_t s0 = 0; s0 < rows; s0 += kRows) {
    const int32_t s1 = s0 + kRows < rows ? s0 + kRows : rows;
    const Sight all = sight_of_tokens(L - n + s0 / G, L - n + (s1 - 1) / G, L, causal, window, sink);
    const Units u = units_of_sight<BN>(all);
    const std::vector<char> want = seen(L, n, G, causal, window, sink, s0, s1, BN);
    std::vector<char> got(want.size(), 0);
    for (int32_t k = 0; k < u.units; ++k) {
      const int32_t t0 = tile_of_unit<BN>(k, u.first_units, u.gap);
      if (t0 % BN || t0 < 0 || t0 >= L || got[t0 / BN]) return 1;
      got[t0 / BN] = 1;
    }
    if (got != want) return 2;
    for (int tries = 0; tries < 4 && u.units > 0; ++tries) {  // the whole segment, and portions of it
      const int32_t from = tries ? rng() % u.units : 0, end = tries ? from + 1 + rng() % (u.units - from) : u.units;
      for (int half = 0; half < 2 && s0 + 128 * half < s1; ++half) {
        const int32_t r0 = s0 + 128 * half, r1 = r0 + 128 < s1 ? r0 + 128 : s1;
        const Sight see = sight_of_tokens(L - n + r0 / G, L - n + (r1 - 1) / G, L, causal, window, sink);
        const Reach reach = reach_of<BN>(see, u.first_units, u.gap, from, end - from);
        const std::vector<char> mine = seen(L, n, G, causal, window, sink, r0, r1, BN);
        int32_t first = -1, last = -1;
        for (int32_t k = 0; k < end - from; ++k) {
          const bool in = mine[tile_of_unit<BN>(from + k, u.first_units, u.gap) / BN];
          if (in != reach.has(k)) return 3;
          if (in && first < 0) first = k;
          if (in) last = k;
        }
        if (reach.any() != (first >= 0)) return 4;
        if (first >= 0 && (reach.first() != first || reach.last() != last)) return 5;
      }
    }
  }
  return 0;
}

extern "C" int one(int32_t BN, int32_t L, int32_t n, int32_t G, int32_t causal, int32_t window, int32_t sink) {
  std::mt19937 rng(7);
  return BN == 64 ? check<64>(L, n, G, causal, window, sink, rng) : check<128>(L, n, G, causal, window, sink, rng);
}

// The first of `count` random requests that fails a check, as its five sizes and the check in `failed`; 0: none.
extern "C" int many(uint32_t seed, int32_t count, int32_t* failed) {
  std::mt19937 rng(seed);
  for (int i = 0; i < count; ++i) {
    const int32_t G = rng() % 2 ? 1 : 1 + rng() % 9, n = 1 + rng() % 1300, L = rng() % 2500, causal = rng() % 2;
    int32_t window = static_cast<int32_t>(rng() % 1400) - 1, sink = rng() % 500;
    if (rng() % 2) window = 64 * (rng() % 20);
    if (rng() % 2 && L > n && L - n > window) window = L - n - 128 * ((L - n - window) / 128);  // a window that begins with a tile
    if (rng() % 8 == 0) sink = 0x7FFFFFFF;
    if (rng() % 16 == 0) window = 0x7FFFFFFF;
    const int bad = rng() % 2 ? check<64>(L, n, G, causal, window, sink, rng) : check<128>(L, n, G, causal, window, sink, rng);
    if (bad) {
      const int32_t what[] = {L, n, G, causal, window, sink, bad};
      for (int k = 0; k < 7; ++k) failed[k] = what[k];
      return 1;
    }
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("needs g++")
    d = tmp_path_factory.mktemp("tiles")
    (d / "rule.cpp").write_text(PROGRAM)
    out = str(d / "rule.so")
    r = subprocess.run([gxx, "-O2", "-std=c++17", "-Wall", "-shared", "-fPIC", "-fwrapv", "-I", CSRC, str(d / "rule.cpp"), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return ctypes.CDLL(out)


@pytest.mark.parametrize("window", [256, 512, 768, 1024])
@pytest.mark.parametrize("sink", [1, 4, 129, 300])
@pytest.mark.parametrize("L,n", [(600, 600), (1024, 1024), (1100, 716), (2048, 2048), (1500, 1100)])
@pytest.mark.parametrize("causal", [0, 1])
def test_windows_that_begin_with_a_tile(rule, causal, L, n, sink, window):
    """One query head to a KV head: the second 128 rows' window begins a tile later than the first's, and what is a tile
    of the first's window is one of the second's first tokens."""
    for BN in (64, 128):
        assert rule.one(BN, L, n, 1, causal, window, sink) == 0


@pytest.mark.parametrize("seed", range(8))
def test_every_row_sees_its_tiles(rule, seed):
    failed = (ctypes.c_int32 * 7)()
    assert rule.many(seed, 2500, failed) == 0, dict(zip(("L", "n", "G", "causal", "window", "sink", "check"), failed))
