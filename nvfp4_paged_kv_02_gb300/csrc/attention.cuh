// attention.cuh -- attention of one new token per request over a paged NVFP4 cache.
//
// For request b, query head i of KV head h = i / G (G = Hq / H), over the live tokens t:
//   x_t = sm_scale * gs_k * sum_d q[d] (e2m1 * S)_K[t, d]      (soft cap c: c tanh(x_t / c))
//   out = gs_v * sum_t exp(x_t - m) (e2m1 * S)_V[t, :] / l,    m = max x_t, l = sum exp(x_t - m)
//   lse = m + log(l)
// (live: t < len; with a window w also t >= len - 1 - w, or t < sink, the first tokens that stay)
// in one pass with a running maximum and sum. No live token: out = 0, lse = -inf.
//
// What bounds it is reading the cache: 9/8 byte for an element of K and of V together, against
// 4 G operations, so at the measured copy bandwidth an SM has to take in about 42 elements a
// clock. A tile that goes through shared memory as binary16 for tcgen05.mma would have to be
// decoded to registers and written back first; mma.sync takes the decoded registers as they
// are, and its 1024 multiply-adds a clock and SM (measured) are three times what G <= 8 needs.
// It takes some 690 instructions of a warp for 32 tokens of 128 elements, 2.7 a lane and element, of
// which decoding, scaling and multiplying are 1.7. On large calls nothing is full: 59 % of the issue
// slots, 51 % of the ALU pipe, 22 % of the tensor pipe, 4.4 of 6.8 TB/s; 165 registers admit twelve
// warps to an SM, and each of them looks up pages, copies and computes in turn. On small calls it is
// the start (lengths, their scan, the first pages: 4 us), one unit's latency and the joins. At 8 KV heads
// of 128, in calls back to back: 430 K tokens of 128 requests, G = 4: 111 us (4.4 TB/s); 110 K tokens of
// 64 requests, G = 8: 42 us (3.1); one request of 131 K tokens, G = 4: 47.5 us (3.2); 16 requests of 30
// tokens 8.4 us (7.7 in a graph).
//
// Work. A unit is 32 tokens of one (request, KV head, chunk of up to 8 NT query heads). All
// units of a launch, in that order, are cut into equal runs, one for each CTA, so that ragged
// lengths balance and one long request fills the GPU; the lengths are read on the device. In a
// run, the four warps take the units of a segment (request, head, chunk) in turn and are joined
// in shared memory at its end. A segment that several CTAs share is joined by the last of them
// to finish (a counter), always in the order of the runs: results do not depend on timing. Short
// segments are not cut.
//
// A warp's units come through its own ring of stages (cp.async, no barrier with other warps).
// Rows that are not live are zero-filled, never read, and masked.
//
// Scores. S^T = K Q^T by m16n8k16: A is K (16 tokens), B is Q^T (8 heads). Lane (r, c) = (lane
// / 4, lane % 4) holds elements 16 NW c .. 16 NW (c + 1) of its two rows; Q is laid out to
// match (any order of d serves, as long as both have it). e2m1 * S is exact in binary16. A
// query row is scaled by a power of two, so that its largest element is in [2^14, 2^15), and
// is then exact in binary16 down to 2^-38 of that element.
// Weights. p = 2^(x log2 e - m + 8) <= 2^15 (m may lag behind the maximum by 7), rounded to
// binary16 for the second product: 2^-11 relative, and below 2^-14, that is 2^-22 of the weight
// at m, an absolute 2^-25. The sum that they are divided by, and that the log-sum-exp comes from, is
// binary32 and of the weights before that rounding. What the rounding saves: a second product
// with the weights' low parts (binary32 in effect) takes 124 us instead of 111 (430 K tokens), 50 instead of
// 47.5 (one request of 131 K); a sum of the rounded weights beside the other one 113.6 and 48.7. What
// it costs: outputs in binary16 are 2.8e-4 (root of the mean square, relative) from 64 bits on that request,
// where weights in binary32 leave 2.1e-4, the output's own rounding; in bf16 it does not show.
// Sums. The matrix instructions accumulate in binary32 registers, in an order of their own and without
// rounding every step to nearest: a few 2^-24 of the sum of the magnitudes for 16 products.
// Output. O^T = V^T P^T: A is V^T (16 of d), B is P^T, which movmatrix makes of S^T. A
// fragment pairs tokens, codes pair elements of d, so nibbles of two tokens are interleaved
// before they are decoded.
#pragma once

#include "attention.h"
#include "softmax.cuh"

#include <cfloat>
#include <type_traits>

namespace nvfp4 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = 32;     // tokens
constexpr int kTiles = kUnit / 16;  // of 16 tokens
constexpr int kMinUnits = 4;  // of a CTA's run: one for each warp
constexpr int kMaxCtasPerSm = 4;
constexpr int kPlain = 0, kSinks = 1, kTokens = 2;  // kinds of the kernel
constexpr int kSegmentCost = 9;
constexpr size_t kMostSmem = 224 * 1024;  // dynamic; the CTA's limit less its static arrays
// A segment of so few units is the run's that it begins in: cutting it costs a join (3 us) and saves
// less. 512 lists of 20 to 400 tokens: 15 us (with 8 here: 17), of 384: 19.3 (20.7); one request of 500
// tokens (16 units): 9.1 us in a graph, cut (with 16 here 0.5 more), 32 lists of 512: 11.2 (12.7).
constexpr int kWholeUnits = 12;

// ---- instructions ------------------------------------------------------------------------

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// ---- which units ---------------------------------------------------------------------------

// The live range of request b: tokens [lo, len), and with a window the first `sink` ones. Its units are the
// `first_units` that hold those, and from the unit that holds lo on (`gap` units are passed over).
struct Span {
  int32_t lo, len, sink, first_units, gap;
};
template <int KIND>
__device__ __forceinline__ Span span_of(const AttentionArgs& a, int32_t b, int32_t tokens = 1) {
  const int64_t reach = a.max_pages * a.ps;
  const int32_t n = max(__ldg(a.seq_lens + b), 0);
  Span s;
  s.len = n > reach ? static_cast<int32_t>(reach) : n;
  const int32_t first = s.len - tokens;  // the first query token's position
  s.lo = a.window_left >= 0 ? max(0, first - min(a.window_left, s.len)) : 0;
  if constexpr (KIND == kPlain) {
    s.sink = s.first_units = 0;
    s.gap = s.lo / kUnit;
    return s;
  }
  s.sink = min(a.sink, s.lo);
  s.first_units = static_cast<int32_t>((static_cast<uint32_t>(s.sink) + kUnit - 1) / kUnit);
  s.gap = max(s.lo / kUnit - s.first_units, 0);  // (0: the last of the first units may hold lo too)
  return s;
}

// kTokens: the query tokens [q0, q0 + n) of request b, if their rows are for this kernel (n = 0: they are not).
struct Tokens {
  int64_t q0;
  int32_t n;
};
__device__ __forceinline__ Tokens tokens_of(const AttentionArgs& a, int32_t b) {
  const int64_t p0 = min(max(static_cast<int64_t>(__ldg(a.qo_indptr + b)), int64_t(0)), a.nnz);
  const int64_t p1 = min(max(static_cast<int64_t>(__ldg(a.qo_indptr + b + 1)), p0), a.nnz);
  return {p0, (p1 - p0) * a.G <= a.most_rows ? static_cast<int32_t>(p1 - p0) : 0};
}

// Units of one (request, head): of its tokens, or of the slots of its selected pages.
template <int KIND>
__device__ __forceinline__ int32_t units_of(const AttentionArgs& a, int32_t b, int32_t h) {
  if constexpr (KIND == kTokens) {
    const Tokens q = tokens_of(a, b);
    if (q.n == 0) return 0;
    const Span s = span_of<KIND>(a, b, q.n);
    return s.len > 0 ? (s.len - 1) / kUnit + 1 - s.gap : 0;
  }
  if (a.selected) {
    const int32_t n = min(max(__ldg(a.num_selected + static_cast<int64_t>(b) * a.H + h), 0), a.max_selected);
    return (n * a.ps + kUnit - 1) / kUnit;
  }
  const Span s = span_of<KIND>(a, b);
  return s.len > 0 ? (s.len - 1) / kUnit + 1 - s.gap : 0;
}

// What a segment counts for when the runs are cut: its units, and kSegmentCost for its queries,
// its join and its output. Those trailing places of a segment hold no work.
__device__ __forceinline__ int32_t places_of(int32_t units) { return units > 0 ? units + kSegmentCost : 0; }

template <int KIND>
__device__ __forceinline__ int64_t places_of_request(const AttentionArgs& a, int32_t b) {
  int64_t n = 0;
  if (a.selected) {
    for (int32_t h = 0; h < a.H; ++h) n += places_of(units_of<KIND>(a, b, h));
  } else {
    n = static_cast<int64_t>(places_of(units_of<KIND>(a, b, 0))) * a.H;
  }
  return n * a.chunks;
}

// cum[e] = places of the requests up to the end of group e (of 1 << a.log2_group in order, a.groups of
// them); every thread calls it, ends with a barrier.
template <int KIND>
__device__ __forceinline__ void scan_places(const AttentionArgs& a, int64_t* cum, int64_t* s_warp) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.groups + kThreads - 1) / kThreads;
  const int lo = tid * per, hi = min(a.groups, lo + per);
  int64_t local = 0;
  for (int e = lo; e < hi; ++e) {
    local += places_of_request<KIND>(a, e << a.log2_group);
    for (int b = (e << a.log2_group) + 1; b < min(a.B, (e + 1) << a.log2_group); ++b) local += places_of_request<KIND>(a, b);
    cum[e] = local;
  }
  int64_t v = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  int64_t before = v - local;
  for (int w = 0; w < warp; ++w) before += s_warp[w];
  for (int e = lo; e < hi; ++e) cum[e] += before;
  __syncthreads();
}

// One (request, head, chunk of query heads), and the place of its first unit relative to the
// run's first.
struct Segment {
  int32_t b, h, chunk, units, start;
};

template <int KIND>
__device__ __forceinline__ Segment find_segment(const AttentionArgs& a, const int64_t* cum, int64_t place) {
  int32_t lo = 0, hi = a.groups - 1;
  while (lo < hi) {
    const int32_t mid = (lo + hi) >> 1;
    if (cum[mid] > place) hi = mid;
    else lo = mid + 1;
  }
  Segment s{lo << a.log2_group, 0, 0, 0, 0};
  int64_t start = lo > 0 ? cum[lo - 1] : 0;
  if (a.log2_group > 0) {  // the request in its group
    for (int64_t n; place >= start + (n = places_of_request<KIND>(a, s.b)); ++s.b) start += n;
  }
  s.units = units_of<KIND>(a, s.b, 0);
  if (a.selected) {
    for (;;) {
      const int64_t head = static_cast<int64_t>(places_of(s.units)) * a.chunks;
      if (place < start + head || s.h + 1 == a.H) break;
      start += head;
      s.units = units_of<KIND>(a, s.b, ++s.h);
    }
  } else {
    const int64_t head = static_cast<int64_t>(places_of(s.units)) * a.chunks;
    s.h = static_cast<int32_t>(quotient64(place - start, head));
    start += s.h * head;
  }
  if (a.chunks > 1) s.chunk = static_cast<int32_t>(quotient64(place - start, places_of(s.units)));
  s.start = static_cast<int32_t>(start + static_cast<int64_t>(s.chunk) * places_of(s.units) - place);
  return s;
}

// The next segment that has units (the caller knows that there is one).
template <int KIND>
__device__ __forceinline__ void next_segment(const AttentionArgs& a, Segment& s) {
  s.start += places_of(s.units);
  if (++s.chunk < a.chunks) return;
  s.chunk = 0;
  do {
    if (++s.h == a.H) {
      s.h = 0;
      ++s.b;
    }
    s.units = s.b < a.B ? units_of<KIND>(a, s.b, s.h) : 1;
  } while (s.units == 0);
}

// ---- one warp's stages ---------------------------------------------------------------------

// Physical order of eight tokens in a fragment. With it and the swizzle below, the reads of K
// (rows by lane / 4) and of V (rows by 2 (lane % 4)) both touch every bank once.
__device__ __forceinline__ int token_of(int k) { return k < 4 ? k : k ^ 1; }

template <int NW>
struct Tile {
  static constexpr int kRow = 32 * NW;       // bytes of a row of codes, D rounded up to 64 NW
  static constexpr int kScales = 4 * NW;     // bytes of its scales
  static constexpr int kV = kUnit * kRow;    // V's codes
  static constexpr int kKs = 2 * kUnit * kRow;
  static constexpr int kVs = kKs + kUnit * kScales;
  static constexpr int kMask = kVs + kUnit * kScales;
  static constexpr int kBytes = kMask + 16;
  // 16-byte chunks of row t are exchanged so that a fragment's rows spread over the banks
  __host__ __device__ static constexpr int swizzle(int t) { return NW == 2 ? t & 2 : (NW == 4 ? t & 7 : 0); }
};

constexpr int kStages = 3;

// ---- the kernel ------------------------------------------------------------------------------

// NW: words of codes that a lane holds of a V row (D <= 64 NW). NT: eights of query heads.
// KIND: kPlain; kSinks, with first tokens that stay beside a window (111.1 us of attend-large's calls without them
// would be 112.5 with their arithmetic); kTokens, of several query tokens of each request, which see different positions: a row in place of a query head is
// a (token, head) pair, row r of KV head h is token r / G and head h G + r % G. Requests of up to most_rows rows.
// FULL: D = 64 NW and scale rows that cp.async can copy; otherwise any D, and scales of any
// alignment, which go through registers.
template <int NW, int NT, bool FULL, int KIND>
__global__ void __launch_bounds__(kThreads, NW <= 2 && NT == 1 ? 3 : 1) attention_kernel(const AttentionArgs a) {
  using T = Tile<NW>;
  constexpr int NS = kStages;
  constexpr int kHeads = 8 * NT;
  constexpr int kPitch = 64 * NW + 4;  // floats of a row of O in shared memory
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t s_scan[kWarps];
  __shared__ float s_m[kWarps][kHeads], s_l[kWarps][kHeads], s_f[kWarps][kHeads], s_top[kHeads], s_sum[kHeads];
  __shared__ struct { int32_t b, h, chunk, first, last, join; } s_shared[2];  // segments shared with other runs
  float* s_o = reinterpret_cast<float*>(smem + kWarps * NS * T::kBytes);  // [kWarps][kHeads][kPitch]
  int64_t* cum = reinterpret_cast<int64_t*>(s_o + kWarps * kHeads * kPitch);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, c = lane & 3;
  const int D = FULL ? 64 * NW : a.D;
  const float gk = __ldg(a.k_scale), gv = __ldg(a.v_scale);
  scan_places<KIND>(a, cum, s_scan);

  // heads without live tokens get zeros
  auto write_zeros = [&] {
    for (int32_t b = blockIdx.x; b < a.B; b += gridDim.x) {
      const int64_t reach = a.max_pages * a.ps;
      if (tid == 0 && __ldg(a.seq_lens + b) > reach) flag(a.status, NVFP4_DEV_LEN_CLAMPED);
      if (!a.selected && units_of<KIND>(a, b, 0) > 0) continue;
      if constexpr (KIND == kTokens) {
        const Tokens q = tokens_of(a, b);
        const int64_t row = q.q0 * a.Hq, rows = static_cast<int64_t>(q.n) * a.Hq;
        uint2* o = reinterpret_cast<uint2*>(a.out + row * D * 2);
        for (int64_t i = tid; i < rows * D / 4; i += kThreads) o[i] = make_uint2(0, 0);
        for (int64_t i = tid; i < rows && a.lse; i += kThreads) a.lse[row + i] = -INFINITY;
      } else {
      for (int32_t h = 0; h < a.H; ++h) {
        if (units_of<KIND>(a, b, h) > 0) continue;
        const int64_t row = static_cast<int64_t>(b) * a.Hq + static_cast<int64_t>(h) * a.G;
        uint2* o = reinterpret_cast<uint2*>(a.out + row * D * 2);
        for (int i = tid; i < a.G * D / 4; i += kThreads) o[i] = make_uint2(0, 0);
        for (int i = tid; i < a.G && a.lse; i += kThreads) a.lse[row + i] = -INFINITY;
      }
      }
    }
  };
  const int64_t total = cum[a.groups - 1];
  const int64_t want = (total + kMinUnits - 1) / kMinUnits;
  const int64_t ncta = want < gridDim.x ? want : gridDim.x;
  if (blockIdx.x >= ncta) {
    write_zeros();
    return;
  }
  Cut cut;
  cut.per = quotient64(total, ncta);
  cut.more = total - cut.per * ncta;
  const int64_t c0 = cut.begin(blockIdx.x);
  const int32_t run = static_cast<int32_t>(cut.per + (blockIdx.x < cut.more ? 1 : 0));  // places

  const uint32_t ring = smem_addr(smem) + warp * NS * T::kBytes;
  uint8_t* const ring_p = smem + warp * NS * T::kBytes;
  if (!FULL) {
    // what lies between D and 64 NW stays zero: no copy writes there
    for (int i = lane; i < NS * T::kBytes / 16; i += 32) reinterpret_cast<uint4*>(ring_p)[i] = uint4{};
    __syncwarp();
  }

  auto more = [&](const Segment& s) { return s.start + places_of(s.units) < run; };
  Segment cs = find_segment<KIND>(a, cum, c0);  // the consumer's segment
  // the run begins in the segment's empty places, or in a segment that is not cut
  if (cs.start + cs.units <= 0 || (cs.start < 0 && cs.units <= kWholeUnits)) {
    if (!more(cs)) {
      write_zeros();
      return;
    }
    next_segment<KIND>(a, cs);
  }
  uint32_t raw[NT][8 * NW];  // the coming segment's query rows, as they are
  auto load_queries = [&](const Segment& s) {
    if constexpr (KIND == kTokens) {
      const Tokens tk = tokens_of(a, s.b);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int row = 8 * nt + r, token = row / a.G;
        const uint8_t* q = a.q + (tk.q0 + token) * a.q_row_bytes + ((static_cast<int64_t>(s.h) * a.G + row - token * a.G) * D + 16 * NW * c) * 2;
#pragma unroll
        for (int i = 0; i < 2 * NW; ++i) {
          const bool in = token < tk.n && 16 * NW * c + 8 * i < D;
          const uint4 x = in ? __ldg(reinterpret_cast<const uint4*>(q) + i) : uint4{};
          raw[nt][4 * i] = x.x; raw[nt][4 * i + 1] = x.y; raw[nt][4 * i + 2] = x.z; raw[nt][4 * i + 3] = x.w;
        }
      }
      return;
    }
    const int head0 = s.chunk * a.chunk_heads, heads = min(a.chunk_heads, a.G - head0);
    const uint8_t* q = a.q + s.b * a.q_row_bytes +
                       ((static_cast<int64_t>(s.h) * a.G + head0 + r) * D + 16 * NW * c) * 2;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2 * NW; ++i) {
        const bool in = 8 * nt + r < heads && 16 * NW * c + 8 * i < D;
        const uint4 x = in ? __ldg(reinterpret_cast<const uint4*>(q + 16 * nt * D) + i) : uint4{};
        raw[nt][4 * i] = x.x; raw[nt][4 * i + 1] = x.y; raw[nt][4 * i + 2] = x.z; raw[nt][4 * i + 3] = x.w;
      }
  };
  load_queries(cs);

  Segment ps = cs;  // the producer's segment
  // -- the producer: this warp's units, one looked up ahead of its copies --
  // the units [u, end) of a segment that lie in this run
  auto portion = [&](const Segment& s, int32_t& u, int32_t& end) {
    u = max(-s.start, 0);
    end = s.units <= kWholeUnits ? s.units : min(run - s.start, s.units);
  };
  int32_t pu, pend;
  Span span;            // the producer's request
  int32_t slots = 0;    // slots of its selected pages
  const uint8_t* list;  // its row of the page table
  auto enter = [&] {
    portion(ps, pu, pend);
    pu += warp;
    span = span_of<KIND>(a, ps.b, KIND == kTokens ? tokens_of(a, ps.b).n : 1);
    list = static_cast<const uint8_t*>(a.block_tables) + (ps.b * a.max_pages << (a.table64 ? 3 : 2));
    if (a.selected)
      slots = min(max(__ldg(a.num_selected + static_cast<int64_t>(ps.b) * a.H + ps.h), 0), a.max_selected) * a.ps;
  };
  enter();
  auto settle = [&] {  // to a unit of this warp, or past the run's end (pu >= pend)
    while (pu >= pend && more(ps)) {
      next_segment<KIND>(a, ps);
      enter();
    }
  };
  settle();
  // What this lane has looked up of the next unit: its row `lane`. The table's entry stays as it
  // was loaded until the copies are issued, so that nothing waits for it here.
  int32_t lk_lo = 0, lk_hi = 0;
  uint32_t lk_row = 0;
  bool lk_unit = false, lk_live = false;
  auto look_up = [&] {
    lk_unit = pu < pend;
    lk_live = false;
    if (!lk_unit) return;
    // a token, or a slot of the selected pages
    const int32_t p = static_cast<int32_t>(static_cast<uint32_t>((a.selected || (KIND != kPlain && pu < span.first_units) ? 0 : span.gap) + pu) * kUnit + lane);
    int32_t col = div_q32(p, a.div_ps);
    const int32_t slot = p - col * a.ps;
    if (a.selected) {
      if (p >= slots) return;
      col = __ldg(a.selected + (static_cast<int64_t>(ps.b) * a.H + ps.h) * a.max_selected + col);
      if (col < 0 || col >= a.max_pages) {
        flag(a.status, NVFP4_DEV_BAD_PAGE);
        return;
      }
      if (static_cast<int64_t>(col) * a.ps + slot >= span.len) return;
    } else if ((p < span.lo && (KIND == kPlain || p >= span.sink)) || p >= span.len) {
      return;
    }
    const int32_t* entry = reinterpret_cast<const int32_t*>(list + (static_cast<int64_t>(col) << (a.table64 ? 3 : 2)));
    lk_lo = __ldg(entry);
    if (a.table64) lk_hi = __ldg(entry + 1);
    lk_row = a.layout == NVFP4_NHD ? slot * a.H + ps.h : ps.h * a.ps + slot;
    lk_live = true;
  };
  look_up();

  // !FULL: scale bytes on their way to the stage of the unit issued last
  uint32_t pk[NW], pv[NW];
  int carried_stage = -1;
  const int nb = D / 16;
  auto put_scales = [&] {
    if (carried_stage < 0) return;
    uint8_t* st = ring_p + carried_stage * T::kBytes + lane * T::kScales;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      *reinterpret_cast<uint32_t*>(st + T::kKs + 4 * w) = pk[w];
      *reinterpret_cast<uint32_t*>(st + T::kVs + 4 * w) = pv[w];
    }
  };
  // Lanes copy 16 bytes each of consecutive rows (FULL; kRows rows at a time).
  constexpr int kChunks = 2 * NW;
  constexpr bool kEven = FULL && NW != 3;  // a row's chunks divide the warp
  constexpr int kRows = 32 / kChunks;
  const int my_row = lane / kChunks, my_chunk = lane % kChunks;
  const uint32_t my_dst = my_row * T::kRow + ((my_chunk ^ T::swizzle(my_row)) << 4);
  const uint8_t* const k_base = a.kc.data + 16 * my_chunk;
  const uint8_t* const v_base = a.vc.data + 16 * my_chunk;
  // Copies of the unit looked up into stage s, then the look-up of the next one.
  auto issue = [&](int s) {
    if (!FULL) put_scales();
    if (lk_unit) {
      const uint32_t st = ring + s * T::kBytes;
      uint32_t page = static_cast<uint32_t>(lk_lo);
      bool live = lk_live;
      if (live && (page >= a.pool_pages || (a.table64 && lk_hi != 0))) {
        flag(a.status, NVFP4_DEV_BAD_PAGE);
        live = false;
      }
      const uint32_t mask = __ballot_sync(0xFFFFFFFFu, live);
      if (lane == 0) *reinterpret_cast<uint32_t*>(ring_p + s * T::kBytes + T::kMask) = mask;
      const uint32_t ksd = st + T::kKs + lane * T::kScales, vsd = st + T::kVs + lane * T::kScales;
      constexpr int kPart = NW == 3 ? 4 : 4 * NW;
      if (kEven && a.compact && mask == 0xFFFFFFFFu) {
        // the common unit: every row live, one 32-bit offset for K and V, in 16 (scales: 4) bytes
        const uint32_t sf = page * (a.k_sf_stride / 4) + lk_row * (T::kScales / 4);
        cp_async<kPart>(ksd, a.kc.sf + sf * uint64_t(4), true);
        cp_async<kPart>(vsd, a.vc.sf + sf * uint64_t(4), true);
        const uint32_t off = page * (a.k_stride / 16) + lk_row * (T::kRow / 16);
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const uint64_t at = __shfl_sync(0xFFFFFFFFu, off, i * kRows + my_row) * uint64_t(16);
          const uint32_t dst = st + i * kRows * T::kRow + (NW == 4 && (i & 1) ? my_dst ^ 64u : my_dst);
          cp_async<16>(dst, k_base + at, true);
          cp_async<16>(dst + T::kV, v_base + at, true);
        }
      } else {
        if (!live) page = 0;  // (a row that is not live is copied as zeros)
        const uint32_t rw = live ? lk_row : 0;
        const uint8_t* ks = a.kc.sf + static_cast<uint64_t>(page) * a.k_sf_stride + static_cast<uint64_t>(rw) * nb;
        const uint8_t* vs = a.vc.sf + static_cast<uint64_t>(page) * a.v_sf_stride + static_cast<uint64_t>(rw) * nb;
        if (FULL) {
#pragma unroll
          for (int w = 0; w < T::kScales / kPart; ++w) {
            cp_async<kPart>(ksd + w * kPart, ks + w * kPart, live);
            cp_async<kPart>(vsd + w * kPart, vs + w * kPart, live);
          }
        } else {
#pragma unroll
          for (int w = 0; w < NW; ++w) pk[w] = pv[w] = 0;
#pragma unroll
          for (int w = 0; w < 4 * NW; ++w) {
            if (live && w < nb) {
              pk[w / 4] |= static_cast<uint32_t>(__ldg(ks + w)) << (8 * (w % 4));
              pv[w / 4] |= static_cast<uint32_t>(__ldg(vs + w)) << (8 * (w % 4));
            }
          }
        }
        auto copy = [&](int row, int off, auto bytes) {
          constexpr int B = decltype(bytes)::value;
          const uint32_t pg = __shfl_sync(0xFFFFFFFFu, page, row);
          const uint64_t in = static_cast<uint64_t>(__shfl_sync(0xFFFFFFFFu, rw, row)) * (D / 2) + off;
          const bool ok = mask >> row & 1u;
          const uint32_t at = st + row * T::kRow + (((off >> 4) ^ T::swizzle(row)) << 4) + (off & 15);
          cp_async<B>(at, a.kc.data + static_cast<uint64_t>(pg) * a.k_stride + in, ok);
          cp_async<B>(at + T::kV, a.vc.data + static_cast<uint64_t>(pg) * a.v_stride + in, ok);
        };
        if (FULL) {
#pragma unroll 1
          for (int i = 0; i < kChunks; ++i) {
            const int k = i * 32 + lane;
            copy(k / kChunks, k % kChunks * 16, std::integral_constant<int, 16>{});
          }
        } else {
          // eight rows at a time, four lanes to a row
#pragma unroll 1
          for (int i = 0; i < 4; ++i)
            for (int w = 0; w < nb; w += 4) {
              const int off = min(w + (lane & 3), nb - 1) * 8;  // (the last chunk again, rather than none)
              copy(8 * i + (lane >> 2), off, std::integral_constant<int, 8>{});
            }
        }
      }
      carried_stage = s;
      pu += kWarps;
      settle();
      look_up();
    } else {
      carried_stage = -1;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < NS - 1; ++s) issue(s);

  // -- the consumer --
  const int t0 = token_of(r);                    // this lane's K rows: t0 and t0 + 8
  const int v0 = token_of(2 * c), v1 = token_of(2 * c + 1);  // its V rows, and 8 more
  // factors of the `parts` parts and the joined maximum and sum, by the first threads (what lies past the
  // parts is of another segment: a NaN there must not get into the sum, not even with a factor of 0)
  auto join_stats = [&](int parts) {
    if (tid < kHeads) {
      float M = -INFINITY, L = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        if (w < parts) M = fmaxf(M, s_m[w][tid]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w >= parts) break;
        const float f = s_m[w][tid] == -INFINITY ? 0.0f : ex2(s_m[w][tid] - M);
        s_f[w][tid] = f;
        L += f * s_l[w][tid];
      }
      s_top[tid] = M;
      s_sum[tid] = L;
    }
    __syncthreads();
  };
  auto joined = [&](int head, int d, int parts) {
    float4 v{0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w >= parts) break;
      const float f = s_f[w][head];
      const float4 x = *reinterpret_cast<const float4*>(s_o + (w * kHeads + head) * kPitch + d);
      v.x += f * x.x; v.y += f * x.y; v.z += f * x.z; v.w += f * x.w;
    }
    return v;
  };
  // (kTokens: `row` is the request's first token, `h` the KV head)
  auto write_out = [&](int64_t row, int heads, int parts, int32_t h) {
    auto at = [&](int head) -> int64_t {
      if constexpr (KIND == kTokens) {
        const int token = head / a.G;
        return (row + token) * a.Hq + static_cast<int64_t>(h) * a.G + head - token * a.G;
      }
      return row + head;
    };
    for (int i = tid; i < heads * D / 4; i += kThreads) {
      const int head = i / (D / 4), d = i % (D / 4) * 4;
      const float4 v = joined(head, d, parts);
      const float f = s_sum[head] == 0.0f ? 0.0f : gv / s_sum[head];
      uint2 w;
      w.x = a.bf16 ? bf16x2_from_f32(v.x * f, v.y * f) : f16x2_from_f32(v.x * f, v.y * f);
      w.y = a.bf16 ? bf16x2_from_f32(v.z * f, v.w * f) : f16x2_from_f32(v.z * f, v.w * f);
      *reinterpret_cast<uint2*>(a.out + (at(head) * D + d) * 2) = w;
    }
    if (a.lse && tid < heads)
      a.lse[at(tid)] = s_sum[tid] == 0.0f ? -INFINITY
                                            : (s_top[tid] - kWeightBias) * (1.0f / kLog2e) + logf(s_sum[tid]);
  };
  // Parts of shared segments: run i's slot 0 if the segment began before the run, else its slot 1.
  constexpr int kStats = kHeads * 64 * NW, kSlot = kStats + 2 * kHeads;
  float* const parts = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + NVFP4_COUNTER_BYTES);
  auto part_of = [&](int32_t i, int32_t first) {
    return parts + (2 * static_cast<int64_t>(i) + (i == first ? 1 : 0)) * kSlot;
  };
  uint32_t arrived0 = 0, arrived1 = 0;
  int shared = 0;
  int stage = 0, refill = NS - 1;
  for (;;) {
    // the segment's query heads
    const int head0 = cs.chunk * a.chunk_heads;
    int heads = min(a.chunk_heads, a.G - head0);
    const int64_t q_row = static_cast<int64_t>(cs.h) * a.G + head0;
    // kTokens: what this lane's rows see (t < row_hi, and t >= row_lo or t < sink); units below `plain` and at or past
    // `open` (or of first tokens) are all rows' alike
    Span seen{};
    int64_t q_first = 0;
    int32_t row_hi[NT][2], row_lo[NT][2], plain = 0, open = 0;
    if constexpr (KIND == kTokens) {
      const Tokens tk = tokens_of(a, cs.b);
      heads = tk.n * a.G;
      q_first = tk.q0;
      seen = span_of<KIND>(a, cs.b, tk.n);
      const int32_t first = seen.len - tk.n;
      auto lo_of = [&](int32_t p) { return a.window_left >= 0 && p > a.window_left ? p - a.window_left : 0; };
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int32_t p = first + min((8 * nt + 2 * c + k) / a.G, tk.n - 1);
          row_hi[nt][k] = a.causal ? p + 1 : seen.len;
          row_lo[nt][k] = lo_of(p);
        }
      plain = a.causal ? first + 1 : seen.len;
      open = lo_of(seen.len - 1);
    }
    uint32_t qf[NT][4 * NW][2];
    float factor[NT][2];  // base-2 logarithm units of a score (before the cap: natural ones)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < 8 * NW; ++i) {
        const uint32_t w = raw[nt][i];
        const float lo = a.bf16 ? __uint_as_float(w << 16) : f32_from_f16_lo(w);
        const float hi = a.bf16 ? f32_from_bf16_hi(w) : f32_from_f16_hi(w);
        top = fmaxf(top, fmaxf(fabsf(lo), fabsf(hi)));
      }
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      const int e = top > 0.0f && top <= FLT_MAX ? ilogbf(top) - 14 : 0;
      float f = ldexpf(a.sm_scale, e) * gk;
      // 2^-e as two factors (it may be out of range by itself), with f's sign: f is not negative
      // from here on, and a maximum of scores is one of logits; f = 0 is a query of zeros
      float f1 = __int_as_float((127 - e / 2) << 23);
      const float f2 = __int_as_float((127 - (e - e / 2)) << 23);
      if (f < 0.0f) f1 = -f1;
      if (f == 0.0f) f1 = 0.0f;
      f = f == 0.0f ? 1.0f : fabsf(f);
#pragma unroll
      for (int i = 0; i < 8 * NW; ++i) {
        const uint32_t w = raw[nt][i];
        const float lo = a.bf16 ? __uint_as_float(w << 16) : f32_from_f16_lo(w);
        const float hi = a.bf16 ? f32_from_bf16_hi(w) : f32_from_f16_hi(w);
        qf[nt][i >> 1][i & 1] = f16x2_from_f32(lo * f1 * f2, hi * f1 * f2);
      }
      if (a.soft_cap == 0.0f) f *= kLog2e;
      factor[nt][0] = __shfl_sync(0xFFFFFFFFu, f, 8 * c);
      factor[nt][1] = __shfl_sync(0xFFFFFFFFu, f, 8 * c + 4);
    }
    float o[NT][NW][4][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[nt][w][i][k] = 0.0f;
    }

    float unit[NT][2];  // what turns x into base-2 logarithms
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) unit[nt][k] = a.soft_cap > 0.0f ? kLog2e : factor[nt][k];

    int32_t cu, cend;
    portion(cs, cu, cend);
    const bool whole = cu == 0 && cend == cs.units;
    for (cu += warp; cu < cend; cu += kWarps) {
      cp_async_wait<NS - 2>();
      __syncwarp();
      issue(refill);
      const uint8_t* st = ring_p + stage * T::kBytes;
      refill = stage;
      stage = stage + 1 == NS ? 0 : stage + 1;
      const uint32_t mask = *reinterpret_cast<const uint32_t*>(st + T::kMask);

      float x[kTiles][NT][4];
#pragma unroll
      for (int mt = 0; mt < kTiles; ++mt) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) x[mt][nt][k] = 0.0f;
        // rows t0 + 16 mt and + 8: 8 NW bytes each, NW scales each
        uint32_t kw[2][2 * NW], S2[2][NW];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int t = 16 * mt + 8 * p + t0;
          const uint8_t* row = st + t * T::kRow;
          const uint8_t* sr = st + T::kKs + t * T::kScales + NW * c;
          if (NW == 1) {
            const uint2 v = *reinterpret_cast<const uint2*>(row + 8 * c);
            kw[p][0] = v.x; kw[p][1] = v.y;
            const uint32_t s = *sr;
            S2[p][0] = f16x2_from_e4m3x2(s * 0x0101u);
          } else if (NW == 3) {
#pragma unroll
            for (int i = 0; i < NW; ++i) {
              const uint2 v = *reinterpret_cast<const uint2*>(row + 8 * NW * c + 8 * i);
              kw[p][2 * i] = v.x; kw[p][2 * i + 1] = v.y;
              S2[p][i] = f16x2_from_e4m3x2(static_cast<uint32_t>(sr[i]) * 0x0101u);
            }
          } else {
            const uint32_t s = NW == 2 ? static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(sr))
                                       : *reinterpret_cast<const uint32_t*>(sr);
#pragma unroll
            for (int i = 0; i < NW / 2; ++i) {
              const uint4 v = *reinterpret_cast<const uint4*>(row + (((NW / 2 * c + i) ^ T::swizzle(t)) << 4));
              kw[p][4 * i] = v.x; kw[p][4 * i + 1] = v.y; kw[p][4 * i + 2] = v.z; kw[p][4 * i + 3] = v.w;
              const uint32_t s2 = f16x2_from_e4m3x2(i == 0 ? s : s >> 16);
              S2[p][2 * i] = low_twice(s2);
              S2[p][2 * i + 1] = high_twice(s2);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < NW; ++i) {
          uint32_t k0[8], k1[8];
          decode16(kw[0][2 * i], kw[0][2 * i + 1], S2[0][i], k0);
          decode16(kw[1][2 * i], kw[1][2 * i + 1], S2[1][i], k1);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t f[4] = {k0[2 * j], k1[2 * j], k0[2 * j + 1], k1[2 * j + 1]};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(x[mt][nt], f, qf[nt][4 * i + j][0], qf[nt][4 * i + j][1]);
          }
        }
      }
      // x[mt][nt][2 p + k]: token 16 mt + 8 p + t0, head 8 nt + 2 c + k
      if (a.soft_cap > 0.0f) {
#pragma unroll
        for (int mt = 0; mt < kTiles; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              x[mt][nt][k] = soft_capped(x[mt][nt][k] * factor[nt][k & 1], a.soft_cap);
      }
      if (mask != 0xFFFFFFFFu) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (!(mask >> (8 * k + t0) & 1u)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) x[k / 2][nt][k % 2 * 2] = x[k / 2][nt][k % 2 * 2 + 1] = -INFINITY;
          }
      }
      uint32_t nan_rows[NT][2];  // blocks of V that are NaN where a row sees them
      bool nan_seen = false;
      if constexpr (KIND == kTokens) {
        const int32_t base = (cu < seen.first_units ? cu : cu + seen.gap) * kUnit;
        if (base + kUnit > plain || (base < open && base + kUnit > seen.sink)) {
          auto sees = [&](int32_t t, int nt, int k) {
            return t < row_hi[nt][k] && (t >= row_lo[nt][k] || t < a.sink);
          };
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (!sees(base + 8 * k + t0, nt, e)) x[k / 2][nt][k % 2 * 2 + e] = -INFINITY;
          // A weight of 0 does not keep a NaN of V from a row that does not see it: NaN scales are taken out of the
          // stage here, and put into the sums of the rows that do.
          uint8_t* const sr = const_cast<uint8_t*>(st) + T::kVs + lane * T::kScales;
          uint32_t blocks = 0;
#pragma unroll
          for (int e = 0; e < 4 * NW; ++e)
            if ((sr[e] & 0x7Fu) == 0x7Fu && (mask >> lane & 1u)) blocks |= 1u << e;
          nan_seen = __any_sync(0xFFFFFFFFu, blocks != 0);
          if (nan_seen) {
#pragma unroll
            for (int e = 0; e < 4 * NW; ++e)
              if (blocks >> e & 1u) sr[e] = 0;
            __syncwarp();
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) nan_rows[nt][e] = 0;
            for (int from = 0; from < kUnit; ++from) {
              const uint32_t theirs = __shfl_sync(0xFFFFFFFFu, blocks, from);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (sees(base + from, nt, e)) nan_rows[nt][e] |= theirs;
            }
          }
        }
      }
      // The maximum follows the scores only when one is more than kSlack above it: until then a
      // weight is at most 2^(kWeightBias + kSlack), which binary16 holds.
      float top[NT][2];
      bool grew = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float v = fmaxf(x[0][nt][k], x[0][nt][k + 2]);
#pragma unroll
          for (int mt = 1; mt < kTiles; ++mt) v = max3(v, x[mt][nt][k], x[mt][nt][k + 2]);
          top[nt][k] = v * unit[nt][k];
          grew = grew || top[nt][k] > m[nt][k] + kSlack;
        }
      if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float m2 = top[nt][k];
            m2 = fmaxf(m2, __shfl_xor_sync(0xFFFFFFFFu, m2, 4));
            m2 = fmaxf(m2, __shfl_xor_sync(0xFFFFFFFFu, m2, 8));
            m2 = fmaxf(m2, __shfl_xor_sync(0xFFFFFFFFu, m2, 16));
            const bool rises = m2 > m[nt][k] + kSlack;  // (by head: a result does not depend on other heads)
            const float f = rises ? ex2(m[nt][k] - m2) : 1.0f;
            m[nt][k] = rises ? m2 : m[nt][k];
            l[nt][k] *= f;
#pragma unroll
            for (int w = 0; w < NW; ++w)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                o[nt][w][i][k] *= f;
                o[nt][w][i][k + 2] *= f;
              }
          }
      }
      uint32_t pb[kTiles][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float off0 = m[nt][0] == -INFINITY ? 0.0f : kWeightBias - m[nt][0];
        const float off1 = m[nt][1] == -INFINITY ? 0.0f : kWeightBias - m[nt][1];
#pragma unroll
        for (int mt = 0; mt < kTiles; ++mt)
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const float p0 = ex2(__fmaf_rn(x[mt][nt][2 * p], unit[nt][0], off0));
            const float p1 = ex2(__fmaf_rn(x[mt][nt][2 * p + 1], unit[nt][1], off1));
            l[nt][0] += p0;
            l[nt][1] += p1;
            pb[mt][nt][p] = transpose8x8(f16x2_from_f32(p0, p1));
          }
      }
      // V: tokens v0, v1 (k = 2c, 2c + 1) and 8 more, words NW r .. of each row
#pragma unroll
      for (int mt = 0; mt < kTiles; ++mt) {
        uint32_t vw[4][NW], S01[NW], S23[NW];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const int t = 16 * mt + (p >= 2 ? 8 : 0) + ((p & 1) ? v1 : v0);
          const uint8_t* row = st + T::kV + t * T::kRow;
          if (NW == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(row + (((r >> 1) ^ T::swizzle(t)) << 4) + 8 * (r & 1));
            vw[p][0] = v.x; vw[p][1 % NW] = v.y;
          } else if (NW == 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(row + ((r ^ T::swizzle(t)) << 4));
            vw[p][0] = v.x; vw[p][1 % NW] = v.y; vw[p][2 % NW] = v.z; vw[p][3 % NW] = v.w;
          } else {
#pragma unroll
            for (int w = 0; w < NW; ++w) vw[p][w] = *reinterpret_cast<const uint32_t*>(row + 4 * (NW * r + w));
          }
        }
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          if ((NW == 2 || NW == 4) && (w & 1)) {  // two words to a block
            S01[w] = S01[w - 1 < 0 ? 0 : w - 1];
            S23[w] = S23[w - 1 < 0 ? 0 : w - 1];
            continue;
          }
          const uint8_t* sr = st + T::kVs + 16 * mt * T::kScales + ((NW * r + w) >> 1);
          const uint32_t s0 = sr[v0 * T::kScales], s1 = sr[v1 * T::kScales];
          const uint32_t s2 = sr[(v0 + 8) * T::kScales], s3 = sr[(v1 + 8) * T::kScales];
          S01[w] = f16x2_from_e4m3x2(s1 * 256u + s0);
          S23[w] = f16x2_from_e4m3x2(s3 * 256u + s2);
        }
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          constexpr uint32_t kLow = 0x0F0F0F0Fu;
          uint32_t x01[4], y01[4], x23[4], y23[4];
          const uint32_t e01 = (vw[0][w] & kLow) | ((vw[1][w] << 4) & ~kLow);
          const uint32_t o01 = ((vw[0][w] >> 4) & kLow) | (vw[1][w] & ~kLow);
          const uint32_t e23 = (vw[2][w] & kLow) | ((vw[3][w] << 4) & ~kLow);
          const uint32_t o23 = ((vw[2][w] >> 4) & kLow) | (vw[3][w] & ~kLow);
          f16x2x4_from_e2m1x8(e01, x01[0], x01[1], x01[2], x01[3]);
          f16x2x4_from_e2m1x8(o01, y01[0], y01[1], y01[2], y01[3]);
          f16x2x4_from_e2m1x8(e23, x23[0], x23[1], x23[2], x23[3]);
          f16x2x4_from_e2m1x8(o23, y23[0], y23[1], y23[2], y23[3]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t f[4] = {hmul2_rn(x01[i], S01[w]), hmul2_rn(y01[i], S01[w]),
                                   hmul2_rn(x23[i], S23[w]), hmul2_rn(y23[i], S23[w])};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt][w][i], f, pb[mt][nt][0], pb[mt][nt][1]);
          }
        }
      }
      if (KIND == kTokens && nan_seen) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int w = 0; w < NW; ++w)
              if (nan_rows[nt][k] >> ((NW * r + w) >> 1) & 1u) {
#pragma unroll
                for (int i = 0; i < 4; ++i) o[nt][w][i][k] = o[nt][w][i][k + 2] = NAN;
              }
      }
    }

    // the next segment's queries arrive while this one is joined
    const Segment done = cs;
    const bool last_segment = !more(cs);
    if (!last_segment) {
      next_segment<KIND>(a, cs);
      load_queries(cs);
    }

    // -- the four warps' parts, joined --
    // o[nt][w][i][k], [k + 2]: head 8 nt + 2 c + k, d = 8 (NW r + w) + 2 i, + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float s = l[nt][k];
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 4);
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 8);
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 16);
        const int head = 8 * nt + 2 * c + k;
        if (r == 0) {
          s_m[warp][head] = m[nt][k];
          s_l[warp][head] = s;
        }
        float4* dst = reinterpret_cast<float4*>(s_o + (warp * kHeads + head) * kPitch + 8 * NW * r);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          dst[2 * w] = make_float4(o[nt][w][0][k], o[nt][w][0][k + 2], o[nt][w][1][k], o[nt][w][1][k + 2]);
          dst[2 * w + 1] = make_float4(o[nt][w][2][k], o[nt][w][2][k + 2], o[nt][w][3][k], o[nt][w][3][k + 2]);
        }
      }
    __syncthreads();
    join_stats(kWarps);
    if (whole) {
      write_out(KIND == kTokens ? q_first : static_cast<int64_t>(done.b) * a.Hq + q_row, heads, kWarps, done.h);
    } else {
      // this run's part of a segment that others share: the last of them will join the parts, at its
      // end, so that nobody waits here for the count (a run shares at most its first and its last)
      const int64_t start = c0 + done.start;
      const int32_t first = static_cast<int32_t>(cut.run_of(start));
      const int32_t last = static_cast<int32_t>(cut.run_of(start + done.units - 1));
      float* part = part_of(blockIdx.x, first);
      for (int i = tid; i < heads * D / 4; i += kThreads) {
        const int head = i / (D / 4), d = i % (D / 4) * 4;
        __stcg(reinterpret_cast<float4*>(part + head * (64 * NW) + d), joined(head, d, kWarps));
      }
      if (tid < heads) {
        __stcg(part + kStats + tid, s_top[tid]);
        __stcg(part + kStats + kHeads + tid, s_sum[tid]);
      }
      __syncthreads();
      if (tid == 0) {
        // releases what the CTA wrote (the barrier puts it before) and acquires what others released
        uint32_t before;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;"
                     : "=r"(before) : "l"(static_cast<uint32_t*>(a.workspace) + first) : "memory");
        if (shared == 0) arrived0 = before;
        else arrived1 = before;
        s_shared[shared] = {done.b, done.h, done.chunk, first, last, 0};
      }
      ++shared;
    }
    if (last_segment) break;
    __syncthreads();  // the buffers of the join are free again
  }
  cp_async_wait<0>();

  // -- shared segments whose last part was this run's --
  if (shared > 0) {
    if (tid == 0) {
      for (int n = 0; n < shared; ++n)
        if ((n == 0 ? arrived0 : arrived1) == static_cast<uint32_t>(s_shared[n].last - s_shared[n].first)) {
          s_shared[n].join = 1;
          static_cast<uint32_t*>(a.workspace)[s_shared[n].first] = 0;
        }
    }
    __syncthreads();
    for (int n = 0; n < shared; ++n) {
      if (!s_shared[n].join) continue;
      const int32_t first = s_shared[n].first, last = s_shared[n].last, head0 = s_shared[n].chunk * a.chunk_heads;
      const Tokens tk = KIND == kTokens ? tokens_of(a, s_shared[n].b) : Tokens{0, 0};
      const int heads = KIND == kTokens ? tk.n * a.G : min(a.chunk_heads, a.G - head0);
      // The last of them adds all up, in the runs' order, with kBatch parts' loads under way at once:
      // this is a chain of trips to L2, at the kernel's end. Few parts: all threads go over all of
      // them; many: every warp over a fourth.
      constexpr int kBatch = 8;
      const int teams = last - first >= kBatch ? kWarps : 1;
      const int team = teams > 1 ? warp : 0, size = kThreads / teams;
      for (int k0 = teams > 1 ? lane : tid; k0 < heads * D / 4; k0 += size) {
        const int head = k0 / (D / 4), d = k0 % (D / 4) * 4;
        float M = -INFINITY, L = 0.0f;
        float4 v{0, 0, 0, 0};
        for (int32_t i0 = first + team; i0 <= last; i0 += kBatch * teams) {
          float mi[kBatch], li[kBatch], top = M;
          float4 x[kBatch];
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const int32_t i = i0 + k * teams;
            const float* p = part_of(i, first);
            mi[k] = i <= last ? __ldcg(p + kStats + head) : -INFINITY;
            li[k] = i <= last && d == 0 ? __ldcg(p + kStats + kHeads + head) : 0.0f;
            x[k] = i <= last ? __ldcg(reinterpret_cast<const float4*>(p + head * (64 * NW) + d)) : float4{};
          }
#pragma unroll
          for (int k = 0; k < kBatch; ++k) top = fmaxf(top, mi[k]);
          // Nothing above -inf so far: the parts hold zeros, or NaN where every score was NaN, which has to
          // stay in the sums; a later maximum multiplies them by 0.
          const bool none = top == -INFINITY;
          const float f = none ? 1.0f : ex2(M - top);
          M = top;
          L *= f;
          v.x *= f; v.y *= f; v.z *= f; v.w *= f;
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const float g = none ? 1.0f : ex2(mi[k] - top);
            L += g * li[k];
            v.x += g * x[k].x; v.y += g * x[k].y; v.z += g * x[k].z; v.w += g * x[k].w;
          }
        }
        *reinterpret_cast<float4*>(s_o + (team * kHeads + head) * kPitch + d) = v;
        if (d == 0) {
          s_m[team][head] = M;
          s_l[team][head] = L;
        }
      }
      __syncthreads();
      join_stats(teams);
      write_out(KIND == kTokens ? tk.q0 : static_cast<int64_t>(s_shared[n].b) * a.Hq + static_cast<int64_t>(s_shared[n].h) * a.G + head0,
                heads, teams, s_shared[n].h);
      __syncthreads();
    }
  }
  write_zeros();
}

template <int NW, int NT, bool FULL, int KIND>
nvfp4_status launch_t(AttentionArgs a, cudaStream_t stream) {
  const auto kern = attention_kernel<NW, NT, FULL, KIND>;
  const size_t fixed = kWarps * kStages * Tile<NW>::kBytes + kWarps * 8 * NT * (64 * NW + 4) * 4;
  // an entry of the scan for each request; where they do not fit (above some 10,600 requests with head_dim
  // above 192, 15,100 above 128), for two
  a.groups = a.B;
  while (fixed + static_cast<size_t>(a.groups) * 8 > kMostSmem) a.groups = (a.B + (1 << ++a.log2_group) - 1) >> a.log2_group;
  const size_t smem = fixed + static_cast<size_t>(a.groups) * 8;
  int64_t cap;
  if (nvfp4_status st = resident_ctas(reinterpret_cast<const void*>(kern), kThreads, smem, kMaxCtasPerSm,
                                      "nvfp4_paged_attention_decode", &cap))
    return st;
  const int64_t reach = a.selected ? static_cast<int64_t>(a.max_selected) * a.ps : a.max_pages * a.ps;
  const int64_t most = static_cast<int64_t>(a.B) * a.H * a.chunks * ((reach + kUnit - 1) / kUnit + kSegmentCost);  // places
  const int64_t need = (most + kMinUnits - 1) / kMinUnits;
  const int grid = static_cast<int>(need < cap ? (need < 1 ? 1 : need) : cap);
  kern<<<grid, kThreads, smem, stream>>>(a);
  return check_launch("nvfp4_paged_attention_decode");
}

template <int NW, int NT, int KIND>
nvfp4_status launch_f(const AttentionArgs& a, bool full, cudaStream_t s) {
  return full ? launch_t<NW, NT, true, KIND>(a, s) : launch_t<NW, NT, false, KIND>(a, s);
}

// nw: head_dim / 64, rounded up; nt: eights of rows.
template <int KIND>
nvfp4_status launch_kind(const AttentionArgs& a, int nw, int nt, bool full, cudaStream_t stream) {
  switch (nw * 2 + nt) {
    case 3: return launch_f<1, 1, KIND>(a, full, stream);
    case 4: return launch_f<1, 2, KIND>(a, full, stream);
    case 5: return launch_f<2, 1, KIND>(a, full, stream);
    case 6: return launch_f<2, 2, KIND>(a, full, stream);
    case 7: return launch_f<3, 1, KIND>(a, full, stream);
    default: return launch_f<4, 1, KIND>(a, full, stream);
  }
}

}  // namespace
}  // namespace nvfp4
