// prefill_tiles.h -- which tiles of BN positions rows of a prompt see. Plain arithmetic, the one place that says so: the
// warps of the kernel that look up pages and those that weigh scores both go by it, and a host compiler takes it.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define NVFP4_ANYWHERE __host__ __device__ __forceinline__
#else
#define NVFP4_ANYWHERE inline
#endif

namespace nvfp4 {

NVFP4_ANYWHERE int32_t least(int32_t a, int32_t b) { return a < b ? a : b; }
NVFP4_ANYWHERE int32_t most(int32_t a, int32_t b) { return a > b ? a : b; }

// Positions that rows of a request see: t < hi and (t >= lo or t < sink); sink <= lo <= hi.
struct Sight {
  int32_t hi, lo, sink;
};
// Of query tokens at positions first to last of a request of L positions.
NVFP4_ANYWHERE Sight sight_of_tokens(int32_t first, int32_t last, int32_t L, bool causal, int32_t window_left, int32_t sink) {
  Sight s;
  s.hi = causal ? most(last + 1, 0) : L;
  s.lo = window_left >= 0 && first > window_left ? least(first - window_left, s.hi) : 0;
  s.sink = least(sink, s.lo);
  return s;
}

// The tiles that hold what a segment's rows see, counted as units: the first `first_units`, which hold its first
// tokens, and those from the one that holds lo on (`gap` tiles are passed over).
struct Units {
  int32_t first_units, gap, units;
};
template <int BN>
NVFP4_ANYWHERE Units units_of_sight(const Sight& s) {
  Units u;
  u.first_units = (s.sink + BN - 1) / BN;
  u.gap = most(s.lo / BN - u.first_units, 0);
  u.units = s.hi > 0 ? (s.hi - 1) / BN + 1 - u.gap : 0;
  return u;
}
template <int BN>
NVFP4_ANYWHERE int32_t tile_of_unit(int32_t u, int32_t first_units, int32_t gap) {  // its first position
  return (u < first_units ? u : u + gap) * BN;
}

// The units u + k, 0 <= k < n, of a portion that hold a position that some of the segment's rows see: k < sinks, and
// [k0, k1). `s` is the sight of those rows. Where the segment passes tiles over, its first tokens end before its
// window's, so they are all rows' alike; where it passes none over, later rows may see more first tokens than it
// counts as its own (their windows begin later), and the bound is their own `sink`.
struct Reach {
  int32_t sinks, k0, k1;
  NVFP4_ANYWHERE bool any() const { return sinks > 0 || k0 < k1; }
  NVFP4_ANYWHERE bool has(int32_t k) const { return k < sinks || (k >= k0 && k < k1); }
  NVFP4_ANYWHERE int32_t first() const { return sinks > 0 ? 0 : k0; }
  NVFP4_ANYWHERE int32_t last() const { return k0 < k1 ? k1 - 1 : sinks - 1; }
};
template <int BN>
NVFP4_ANYWHERE Reach reach_of(const Sight& s, int32_t first_units, int32_t gap, int32_t u, int32_t n) {
  // of the portion, the unit that holds position t or, if it is passed over, the next one
  auto unit_at = [&](int32_t t) {
    const int32_t j = t / BN;
    return (j < first_units ? j : most(j - gap, first_units)) - u;
  };
  if (s.hi <= 0) return {0, 0, 0};
  Reach r;
  r.k1 = least(most(unit_at(s.hi - 1) + 1, 0), n);
  r.k0 = least(most(unit_at(s.lo), 0), n);
  r.sinks = s.sink > 0 ? least(most(unit_at(s.sink - 1) + 1, 0), r.k0) : 0;
  return r;
}

}  // namespace nvfp4
