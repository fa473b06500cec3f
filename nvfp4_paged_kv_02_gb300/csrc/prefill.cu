// prefill.cu -- attention of the last tokens of each request (a prompt, a chunk of one, drafts) over a paged
// NVFP4 cache.
//
// Query token i of the n of request b is at position p = L - n + i (L = its length). Over the live positions t:
//   x_t = sm_scale * gs_k * sum_d q[d] (e2m1 * S)_K[t, d]      (soft cap c: c tanh(x_t / c))
//   out = gs_v * sum_t exp(x_t - m) (e2m1 * S)_V[t, :] / l,    m = max x_t, l = sum exp(x_t - m)
//   lse = m + log(l)
// live: t < L; causal: t <= p; with a window w: t >= p - w, or t < sink. No live position: out = 0, lse = -inf.
//
// Rows. The G query heads of a KV head share its cache, so the rows of one matrix product are (token, head) pairs:
// row r of request b and KV head h is token r / G and head h G + r % G. A segment is 128 or 256 such rows of one
// (request, KV head) and the tiles of BN positions that any of them sees.
//
// Work. All segments' tiles, in order, are cut into equal runs, one for each CTA, by the lengths on the device, so
// that ragged batches balance and few rows over a long cache fill the GPU. A segment of few tiles is not cut. The
// parts of one that is go to the workspace, and a second kernel adds them in the runs' order: results do not
// depend on timing.
//
// A CTA (one to an SM) has four kinds of warps, which wait for one another on mbarriers only:
//   page     (3 warps, in turn) walk the run's tiles, look up the pages and leave in a ring what the others need to
//            know of a tile;
//   decode   (8 warps, some rows of a tile to each) copy codes and scales to shared memory a tile or two ahead, and
//            turn them into e2m1 * S, exact in binary16, in the tensor cores' order;
//   product  (one warp) S = Q K^T and O += P V by tcgen05.mma, sums in tensor memory;
//   softmax  (8 warps, a row to a thread) S from tensor memory, its running maximum and sum, P in binary16 back to
//            tensor memory over S; at a segment's end O to the output. They also bring the next queries.
// Two streams keep the tensor cores busy while the other one is at its weights: the two halves of 256 rows over the
// same tiles, or the same 128 rows over every second tile, joined at the end. head_dim above 128 leaves tensor
// memory for one stream: there S of the next tile is computed meanwhile.
//
// What bounds it. 256 rows of 128 elements take the tensor cores 2048 cycles for a tile of 128 positions, and the CTA
// some 4400: the chain of a stream (S from tensor memory, its maximum, 128 exponentials to a row, P back; O of it; the
// next S: 2900 cycles of a softmax warp, 1000 of the tensor cores, the rest hand-overs), half of which the other
// stream's products fill. One prompt of 12,345 tokens, 32 query heads and 8 KV heads of 128: 1158 us (1078 TFLOP/s; at
// the measured 1947 it would be 641), the tensor pipe busy for 46 %, 57 % of the issue slots, 40 % of the ALU pipe. Eight
// chunks of up to 2048 tokens over up to 10 K positions: 207 us (750 TFLOP/s); four prompts of up to 7879 tokens with
// a window of 1023 and 64 first tokens, 32 query heads on 4: 714 (648); 16 requests of up to 1024 tokens of images with
// heads of 256 and capped logits: 178 (343). A segment's beginning and end cost 15 to 20 K cycles, which the short ones
// of a window feel. What mattered most was that the loops over tiles stay in the instruction cache (they were 3225 us
// for the first prompt when unrolled wide: 28 % of the requests missed) and that little is spilled (36 to 48 bytes a
// thread, reloaded at 84 to 152): 227 KB of shared memory leave the other cache too little to hold more.
// Two warps for the products, one to a stream, are slower (1403 us against 1203 then: the streams fall into step, and
// want the tensor cores and the exponentials at the same times); so are copies by the page warps (1870), rows of S
// held whole in registers (2230, with spills), and decoding warps with K or V to themselves (images 203 against 184).
//
// Queries are scaled row by row by a power of two into binary16 (what is below 2^-38 of a row's largest element is
// lost). Weights are rounded to binary16 for the second product, as in attention.cuh: 2^-11 relative, and below 2^-22 of
// the weight at the running maximum an absolute 2^-33 of that one. The maximum and the sum, of the weights before that
// rounding, stay in binary32. What it costs: outputs in binary16 are 2.7e-4 (root of the mean square, relative) from 64
// bits on the first prompt, where weights in binary32 leave 2.1e-4; in bf16 it does not show. A NaN block scale of V is
// taken as 0 in the product and the outputs that see it are set to NaN: a weight of 0 would not keep it from rows that do
// not.
#include "attention.h"
#include "prefill_tiles.h"
#include "softmax.cuh"
#include "tcgen05.cuh"

#include <algorithm>
#include <cfloat>

namespace nvfp4 {
namespace {

constexpr int kSoftmaxWarps = 8;
constexpr int kDecodeWarps = 8;
constexpr int kProductWarp = kSoftmaxWarps + kDecodeWarps;
constexpr int kPageWarps = 3;
constexpr int kWarps = kProductWarp + 1 + kPageWarps;
constexpr int kThreads = kWarps * 32;
// Registers of a thread of each warpgroup: the launch's 96 for 640 threads, dealt out again.
constexpr int kLaunchRegisters = 96, kSoftmaxRegisters = 136, kDecodeRegisters = 64, kOtherRegisters = 80;
static_assert(2 * kSoftmaxRegisters + 2 * kDecodeRegisters + kOtherRegisters <= 5 * kLaunchRegisters, "more than the launch has");
constexpr int kRing = 8;          // tiles whose places are kept
constexpr int kSegmentCost = 5;   // what a segment's queries and outputs count for, in tiles (2: 1543 us for the long prompt, 4: 1203)
constexpr int kWholeUnits = 8;    // a segment of so few tiles is not cut (12: drafts 127 us against 116, a window 694 against 723)

// DP: head_dim rounded up to 64, 128 or 256. MT: 128 rows of a segment, or twice as many.
template <int DP, int MT>
struct Shape {
  static constexpr int BN = DP > 128 ? 64 : 128;     // positions of a tile
  static constexpr int kRows = 128 * MT;
  static constexpr int kQBytes = 128 * DP * 2;       // of 128 rows
  static constexpr int kTileBytes = BN * DP * 2;
  // codes and scales as they are: of kRaw tiles (and one more of scales), K and V
  static constexpr int kRaw = MT * DP == 256 ? 1 : 2;
  static constexpr int kCodeBytes = BN * DP / 2, kScaleBytes = BN * DP / 16;
  static constexpr int kK = MT * kQBytes, kCodes = kK + 4 * kTileBytes, kScales = kCodes + kRaw * 2 * kCodeBytes;
  static constexpr int kBytes = kScales + (kRaw + 1) * 2 * kScaleBytes;
  static constexpr int kWarpTokens = BN / kDecodeWarps;
  static constexpr uint32_t kO = 2 * BN;             // columns of tensor memory: two of S, then O
};

struct Request {
  int64_t q0;     // first row of query
  int32_t n, L;   // query tokens, positions
};
__device__ __forceinline__ Request request_of(const PrefillArgs& a, int32_t b) {
  const int64_t p0 = min(max(static_cast<int64_t>(__ldg(a.qo_indptr + b)), int64_t(0)), a.nnz);
  const int64_t p1 = min(max(static_cast<int64_t>(__ldg(a.qo_indptr + b + 1)), p0), a.nnz);
  const int64_t reach = a.max_pages * a.ps;
  const int32_t n = max(__ldg(a.seq_lens + b), 0);
  const int32_t tokens = (p1 - p0) * a.G <= a.few_rows ? 0 : static_cast<int32_t>(p1 - p0);
  return {p0, tokens, n > reach ? static_cast<int32_t>(reach) : n};
}

// What rows [r0, r1) of a request see.
__device__ __forceinline__ Sight sight_of(const PrefillArgs& a, const Request& q, int32_t r0, int32_t r1) {
  const int32_t first = q.L - q.n + div_q32(r0, a.div_g), last = q.L - q.n + div_q32(r1 - 1, a.div_g);
  return sight_of_tokens(first, last, q.L, a.causal, a.window_left, a.sink);
}

// A segment, and the place of its first tile relative to the run's first.
struct Segment {
  int32_t b, t, h, units;
  int64_t start;
  Request q;
  Sight see;
  int32_t first_units, gap;
};

// The units [u, end) of a segment that are this run's of `run` places; `mine`: it is, wholly, if it is not cut.
struct Portion {
  int32_t u, end;
  bool mine;
};

template <class S>
__device__ __forceinline__ void fill(const PrefillArgs& a, Segment& s) {
  const int32_t rows = s.q.n * a.G, r0 = s.t * S::kRows;
  s.see = sight_of(a, s.q, r0, min(rows - r0, S::kRows) + r0);
  const Units u = units_of_sight<S::BN>(s.see);
  s.first_units = u.first_units;
  s.gap = u.gap;
  s.units = u.units;
}
// The units of a portion that the 128 rows of half i of a segment see.
template <class S>
__device__ __forceinline__ Reach reach_of_half(const PrefillArgs& a, const Segment& s, const Portion& part, int i) {
  const int32_t r0 = s.t * S::kRows, rows = min(s.q.n * a.G - r0, S::kRows);
  const Sight see = 128 * i < rows ? sight_of(a, s.q, r0 + 128 * i, r0 + min(rows, 128 * i + 128)) : Sight{0, 0, 0};
  return reach_of<S::BN>(see, s.first_units, s.gap, part.u, part.end - part.u);
}
template <class S>
__device__ __forceinline__ int32_t tiles_of(const PrefillArgs& a, const Request& q) {
  return static_cast<int32_t>((static_cast<uint32_t>(q.n * a.G) + S::kRows - 1) / S::kRows);
}
__device__ __forceinline__ int32_t places_of(int32_t units) { return units + kSegmentCost; }
// The next segment (the caller knows that there is one).
template <class S>
__device__ __forceinline__ void next_segment(const PrefillArgs& a, Segment& s) {
  s.start += places_of(s.units);
  if (++s.h < a.H) return;
  s.h = 0;
  if (++s.t >= tiles_of<S>(a, s.q)) {
    s.t = 0;
    do s.q = request_of(a, ++s.b);
    while (s.q.n == 0);
  }
  fill<S>(a, s);
}
__device__ __forceinline__ Portion portion_of(const Segment& s, int64_t run) {
  if (s.units <= kWholeUnits) {
    const bool mine = s.start >= 0 && s.start < run;
    return {0, mine ? s.units : 0, mine};
  }
  const int64_t u = s.start < 0 ? -s.start : 0, left = run - s.start;
  const int32_t end = left < s.units ? static_cast<int32_t>(left) : s.units;
  return {u < end ? static_cast<int32_t>(u) : end, end, false};
}

struct Barriers {
  uint64_t full[4], empty[4];          // K's two stages, then V's
  uint64_t s_full[2], p_full[2], o_full[2], q_full[2], o_step, merge, done;
  uint64_t ring_full[kRing], ring_empty[kRing];
};
// One tile of the run, as the page warps leave it to the others. `stream`: bits 0 and 1, the streams whose rows see
// it; 2 and 3, it is their first of the portion; 4 and 5, their last; 6 and 7, they have one; 8, set; 9, all of its
// positions are on pages of the pool. `rest`: tiles of the portion after it.
struct __align__(16) Tile {
  uint2 where[128];              // page (kNoPage: none) and row in it of each position
  uint32_t live[4];              // positions that are on a page of the pool, 32 to a word
  uint8_t nan[kDecodeWarps];     // a decode warp's V scales hold NaN (eight, read with the next two at once)
  uint32_t stream;
  int32_t rest;
  uint16_t nan_blocks[128];      // which blocks of a position (where its warp's nan is set)
  int32_t first;                 // of its portion
};
constexpr uint32_t kNoPage = 0xFFFFFFFFu;
constexpr int32_t kEnd = -1;          // `rest` after the last tile
struct Shared {
  Barriers bar;
  Tile ring[kRing];
  Segment first;                      // the run's
  Segment next[kSoftmaxWarps];        // a softmax warp's
  uint32_t tmem;
  int32_t dead;                       // a wait has run out
  int32_t last;                       // request that counts
  float factor[256];                  // of the query rows
  float m[128], l[128];               // of the second stream
  uint32_t poison[128];
  int64_t scan[kWarps];
};

// The part of a cut segment that run i holds: [rows][DP] sums, then their maxima and weights. Slot 0: the segment
// began before the run.
__device__ __forceinline__ float* part_of(const PrefillArgs& a, int64_t run, int slot, int rows, int dp) {
  return reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + a.parts_offset) +
         (2 * run + slot) * static_cast<int64_t>(rows) * (dp + 2);
}

// Inclusive sum over the CTA's threads; the total in s_scan[kWarps - 1] on return.
__device__ __forceinline__ int64_t scan_cta(int64_t v, int64_t* s_scan) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == 31) s_scan[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int64_t w = lane < kWarps ? s_scan[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xFFFFFFFFu, w, o);
      if (lane >= o) w += u;
    }
    if (lane < kWarps) s_scan[lane] = w;
  }
  __syncthreads();
  return v + (warp > 0 ? s_scan[warp - 1] : 0);
}

__device__ __forceinline__ uint32_t low_bits(int32_t n) { return n >= 32 ? ~0u : (n <= 0 ? 0u : (1u << n) - 1); }

// E: elements of a row that a lane decodes, 32 (two blocks; 16-byte copies of codes and 4-byte ones of scales) or 16.
template <int DP, int MT, int E>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const PrefillArgs a) {
  using S = Shape<DP, MT>;
  constexpr int BN = S::BN;
  constexpr bool kTwo = MT == 2;                  // streams are halves of the rows
  constexpr bool kTurns = MT == 1 && DP <= 128;   // streams take turns at the tiles
  constexpr bool kOne = DP > 128;                 // one stream
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  uint8_t* const smem = smem_raw + (1024 - smem_addr(smem_raw) % 1024) % 1024;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t limit = a.pipe.wait_limit;  // (of naps)

  // -- the run: tiles of all requests, then places of all tiles --
  int64_t c0, run, ncta;
  Cut cut;
  {
    int32_t* cum = reinterpret_cast<int32_t*>(smem);
    const int per = (a.B + kThreads - 1) / kThreads;
    const int lo = min(a.B, tid * per), hi = min(a.B, lo + per);
    // Requests after an entry of qo_indptr that is below the one before it may share rows with others: they get
    // none, and the tiles stay within 2^24 and one more for each request.
    if (tid == 0) sh.last = a.B - 1;
    int32_t local = 0, last = a.B - 1;
    for (int b = lo; b < hi; ++b) {
      const Request q = request_of(a, b);
      if (__ldg(a.qo_indptr + b + 1) < __ldg(a.qo_indptr + b)) last = min(last, b);
      local += tiles_of<S>(a, q);
      cum[b] = local;
      if (blockIdx.x == 0) {
        if (__ldg(a.seq_lens + b) > a.max_pages * a.ps) flag(a.status, NVFP4_DEV_LEN_CLAMPED);
        const int32_t p0 = __ldg(a.qo_indptr + b), p1 = __ldg(a.qo_indptr + b + 1);
        if (p0 < 0 || p1 < p0 || p1 > a.nnz) flag(a.status, NVFP4_DEV_BAD_BATCH);
      }
    }
    const int32_t before = static_cast<int32_t>(scan_cta(local, sh.scan)) - local;
    for (int b = lo; b < hi; ++b) cum[b] += before;
    if (last < a.B - 1) atomicMin(&sh.last, last);
    __syncthreads();
    const int32_t tiles = cum[sh.last];
    const int32_t per2 = (tiles + kThreads - 1) / kThreads;
    const int32_t f0 = static_cast<int32_t>(min(static_cast<int64_t>(tiles), static_cast<int64_t>(tid) * per2));
    const int32_t f1 = static_cast<int32_t>(min(static_cast<int64_t>(tiles), static_cast<int64_t>(f0) + per2));
    Segment s;
    s.h = 0;
    // every tile of this thread's slice, until `stop` says so
    auto walk = [&](auto stop) {
      int32_t x = 0, y = sh.last;
      while (x < y) {
        const int32_t mid = (x + y) >> 1;
        if (cum[mid] > f0) y = mid;
        else x = mid + 1;
      }
      s.b = x;
      s.t = f0 - (x > 0 ? cum[x - 1] : 0);
      s.q = request_of(a, s.b);
      for (int32_t f = f0;;) {
        fill<S>(a, s);
        if (stop() || ++f == f1) break;
        if (++s.t >= tiles_of<S>(a, s.q)) {
          s.t = 0;
          do s.q = request_of(a, ++s.b);
          while (s.q.n == 0);
        }
      }
    };
    int64_t mine = 0;
    if (f0 < f1)
      walk([&] {
        mine += static_cast<int64_t>(places_of(s.units)) * a.H;
        return false;
      });
    int64_t at = scan_cta(mine, sh.scan) - mine;
    const int64_t total = sh.scan[kWarps - 1];
    const int64_t want = (total + kSegmentCost) / (kSegmentCost + 1);
    ncta = want < gridDim.x ? want : gridDim.x;
    PrefillCut* const cuts = reinterpret_cast<PrefillCut*>(static_cast<uint8_t*>(a.workspace) + NVFP4_COUNTER_BYTES);
    if (tid == 0) cuts[blockIdx.x].last = -1;
    if (blockIdx.x >= ncta) return;
    cut.per = quotient64(total, ncta);
    cut.more = total - cut.per * ncta;
    c0 = cut.begin(blockIdx.x);
    run = cut.per + (blockIdx.x < cut.more ? 1 : 0);
    if (f0 < f1 && c0 >= at && c0 < at + mine) {
      walk([&] {
        const int64_t all = static_cast<int64_t>(places_of(s.units)) * a.H;
        if (c0 >= at + all) {
          at += all;
          return false;
        }
        s.h = static_cast<int32_t>(quotient64(c0 - at, places_of(s.units)));
        s.start = at + static_cast<int64_t>(s.h) * places_of(s.units) - c0;
        sh.first = s;
        return true;
      });
    }
  }
  Barriers& bar = sh.bar;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar.full + i, kDecodeWarps);
      mbar_init(bar.full + 2 + i, kDecodeWarps);
      mbar_init(bar.empty + i, 1);
      mbar_init(bar.empty + 2 + i, 1);
      mbar_init(bar.s_full + i, 1);
      mbar_init(bar.p_full + i, 4);
      mbar_init(bar.o_full + i, 1);
    }
    mbar_init(bar.q_full, kTurns ? kSoftmaxWarps : 4);
    mbar_init(bar.q_full + 1, 4);  // (of the second half)
    mbar_init(&bar.o_step, 1);
    mbar_init(&bar.merge, kSoftmaxWarps);
    mbar_init(&bar.done, 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(bar.ring_full + i, 1);
      mbar_init(bar.ring_empty + i, 1);
    }
    sh.dead = 0;
    fence_mbar_init();
  }
  if (warp == kProductWarp) tmem_alloc(&sh.tmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;

  // A warp's bounded wait; when it runs out, or another's has, all of the CTA's warps return.
  volatile int32_t* const dead = &sh.dead;
  auto wait_warp = [&](uint64_t* b, uint32_t parity) -> bool {
    for (uint32_t i = 0; !__all_sync(0xFFFFFFFFu, mbar_wait_nap(b, parity)); ++i)
      if (__any_sync(0xFFFFFFFFu, i == limit || *dead != 0)) {
        *dead = 1;
        return false;
      }
    return true;
  };
  auto more = [&](const Segment& s) { return s.start + places_of(s.units) < run; };
  const int D = E == 32 && DP <= 128 ? DP : a.D;
  const uint32_t base = smem_addr(smem);

  if (warp >= kProductWarp) set_registers<kOtherRegisters, false>();
  if (warp == kProductWarp) {
    // ---- product ----
    const uint32_t leader = elected();
    {
      const uint32_t shape_s = mma_shape(BN, false), shape_o = mma_shape(D, true);
      const uint32_t q_op = smem_operand(base, 16), k_op = smem_operand(base + S::kK, 16);
      const uint32_t v_op = smem_operand(base + S::kK + 2 * S::kTileBytes, BN * 128);
      uint32_t q_counts = 0, p_counts = 0;  // a bit for each: parities
      auto issue_s = [&](int half, int buf, uint32_t g) {
        const uint32_t q = q_op + half * (S::kQBytes / 16), k = k_op + (g & 1) * (S::kTileBytes / 16), d = tmem + buf * BN;
#pragma unroll
        for (int i = 0; i < DP / 16; ++i)
          if (16 * i < D) mma_ss(leader, d, q + (i >> 2) * 1024 + (i & 3) * 2, k + (i >> 2) * (BN * 8) + (i & 3) * 2, shape_s, i > 0);
        mma_commit(leader, bar.s_full + buf);
      };
      auto issue_o = [&](int stream, int buf, uint32_t g, bool sum) {
        const uint32_t v = v_op + (g & 1) * (S::kTileBytes / 16), d = tmem + S::kO + stream * DP, p = tmem + buf * BN;
#pragma unroll
        for (int i = 0; i < BN / 16; ++i) mma_ts(leader, d, p + 8 * i, v + i * 128, shape_o, sum || i > 0);
      };
      auto k_ready = [&](uint32_t g) {
        const bool ok = wait_warp(bar.full + (g & 1), (g >> 1) & 1);
        tc_fence_after();
        return ok;
      };
      auto v_ready = [&](uint32_t g) { return wait_warp(bar.full + 2 + (g & 1), (g >> 1) & 1); };
      auto q_ready = [&](int half) {
        const bool ok = wait_warp(bar.q_full + half, q_counts >> half & 1);
        q_counts ^= 1u << half;
        return ok;
      };
      auto p_ready = [&](int buf) {
        const bool ok = wait_warp(bar.p_full + buf, p_counts >> buf & 1);
        p_counts ^= 1u << buf;
        tc_fence_after();
        return ok;
      };
      auto tile_ready = [&](uint32_t g) { return wait_warp(bar.ring_full + g % kRing, g / kRing & 1); };
      auto tile = [&](uint32_t g) -> const Tile& { return sh.ring[g % kRing]; };
      auto pass_on = [&](uint32_t g) { if (leader) mbar_arrive(bar.ring_empty + g % kRing); };
      if constexpr (kTwo) {
        // Steps: O of tile g in both halves, and S of the next tile, each behind the O whose P it overwrites. A
        // portion's first step has no O, its last one no S.
        // (A stage of K that is full says that its tile is in the ring: only a portion's first tile, which may be the
        // run's end instead, is waited for there.)
        uint32_t g = 0, now = 0;  // now: the flags of g, 0 in a first step
        int32_t rest = 0;
        for (bool ok = true; ok;) {
          const uint32_t ahead = now ? g + 1 : g;
          const bool more_s = !now || rest > 0;
          uint32_t next = 0;
          auto look = [&] {  // the next tile's stage and flags
            ok = k_ready(ahead);
            if (!ok) return;
            rest = uniform(tile(ahead).rest);
            next = uniform(tile(ahead).stream);
          };
          if (!now) {
            if (!tile_ready(ahead) || static_cast<int32_t>(uniform(tile(ahead).rest)) == kEnd) break;
            look();
          } else {
            ok = v_ready(g);
          }
#pragma unroll 1
          for (int i = 0; ok && i < 2; ++i) {
            if (now >> i & 1) {
              ok = p_ready(i);
              if (!ok) break;
              issue_o(i, i, g, !(now >> (2 + i) & 1));
              if (now >> (4 + i) & 1) mma_commit(leader, bar.o_full + i);
            }
            if (now && more_s && i == 0) look();
            if (ok && !now && (next >> (6 + i) & 1)) ok = q_ready(i);
            if (ok && (next >> i & 1)) issue_s(i, i, ahead);
          }
          if (!ok) break;
          if (now) {
            mma_commit(leader, bar.empty + 2 + (g & 1));
            pass_on(g);
            ++g;
          }
          if (next) mma_commit(leader, bar.empty + (ahead & 1));
          now = next;
        }
      } else {
        // In one stream S of the next tile goes ahead of O of this one; in two, S of the one after the next follows
        // O of this one, whose P it overwrites.
        constexpr int kAhead = kOne ? 1 : 2;
        uint32_t started = 0;  // tiles whose S has been issued
        int turn = 0;          // of the tile's buffers, from a portion's first tile on
        for (uint32_t g = 0; tile_ready(g); ++g) {
          const int32_t rest = uniform(tile(g).rest);
          if (rest == kEnd) break;
          const uint32_t now = uniform(tile(g).stream);
          bool ok = true;
          const bool first = uniform(tile(g).first);
          if (first) {
            turn = 0;
            ok = q_ready(0);
          }
          // the tiles of this portion that are due
          const uint32_t due = kTurns && !first ? g + 1 : g + min(rest, 1) + 1;
#pragma unroll 1
          for (; ok && started < due; ++started) {
            ok = tile_ready(started) && k_ready(started);
            if (!ok) break;
            issue_s(0, (turn + (started - g)) & 1, started);
            mma_commit(leader, bar.empty + (started & 1));
          }
          if (!ok || !v_ready(g) || !p_ready(turn)) break;
          issue_o(kOne ? 0 : turn, turn, g, !(now >> (kOne ? 2 : 2 + turn) & 1));
          mma_commit(leader, bar.empty + 2 + (g & 1));
          if (kOne) mma_commit(leader, &bar.o_step);
          if (now >> 4 & 3) mma_commit(leader, bar.o_full + (kOne ? 0 : turn));
          if (kTurns && rest > 1) {
            if (!tile_ready(g + kAhead) || !k_ready(g + kAhead)) break;
            issue_s(0, turn, g + kAhead);
            mma_commit(leader, bar.empty + ((g + kAhead) & 1));
            started = g + kAhead + 1;
          }
          turn ^= 1;
          pass_on(g);
        }
      }
      // nothing of this CTA is under way any more when it ends
      mma_commit(leader, &bar.done);
      for (uint32_t i = 0; i < kNapLimit && !mbar_wait_nap(&bar.done, 0); ++i) {}
    }
    __syncwarp();
  } else if (warp > kProductWarp) {
    // ---- page ----
    const int turn = warp - kProductWarp - 1;
    Segment s = sh.first;
    Portion part{0, 0, false};
    int32_t k = turn, n = 0;       // this warp's tile of the portion's n
    uint32_t g = turn;
    Reach reach[2];
    auto enter = [&] {
      part = portion_of(s, run);
      n = part.end - part.u;
      if (!kTwo || n <= 0) return;
#pragma unroll
      for (int i = 0; i < 2; ++i) reach[i] = reach_of_half<S>(a, s, part, i);
    };
    enter();
    for (;; g += kPageWarps) {
      bool any = true;
      while (k >= n) {
        if (!more(s)) {
          any = false;
          break;
        }
        k -= n;
        next_segment<S>(a, s);
        enter();
      }
      Tile& out = sh.ring[g % kRing];
      if (!wait_warp(bar.ring_empty + g % kRing, (g / kRing & 1) ^ 1)) break;
      if (any) {
        const int32_t t0 = tile_of_unit<BN>(part.u + k, s.first_units, s.gap);
        bool whole = true;
#pragma unroll 1
        for (int j = 0; j < BN / 32; ++j) {
          const int32_t t = t0 + 32 * j + lane;
          uint2 where = make_uint2(kNoPage, 0);
          if (t < s.see.hi && t < s.q.L && (t >= s.see.lo || t < s.see.sink)) {
            const int32_t col = div_q32(t, a.div_ps), slot = t - col * a.ps;
            const int64_t at = s.b * a.max_pages + col;
            const int64_t p = a.table64 ? __ldg(static_cast<const int64_t*>(a.block_tables) + at)
                                        : static_cast<int64_t>(__ldg(static_cast<const int32_t*>(a.block_tables) + at));
            if (p >= 0 && p < a.pool_pages) where.x = static_cast<uint32_t>(p);
            else flag(a.status, NVFP4_DEV_BAD_PAGE);
            where.y = a.layout == NVFP4_NHD ? slot * a.H + s.h : s.h * a.ps + slot;
          }
          out.where[32 * j + lane] = where;
          const uint32_t word = __ballot_sync(0xFFFFFFFFu, where.x != kNoPage);
          whole = whole && word == ~0u;
          if (lane == 0) out.live[j] = word;
        }
        if (lane == 0) {
          uint32_t stream = whole ? 768 : 256;
          if constexpr (kTwo) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (reach[i].any()) stream |= 64u << i;
              if (reach[i].has(k)) stream |= 1u << i | (k == reach[i].first() ? 4u << i : 0u) | (k == reach[i].last() ? 16u << i : 0u);
            }
          } else if constexpr (kTurns) {
            stream |= 1u << (k & 1) | (k < 2 ? 4u << (k & 1) : 0u) | (k + 2 >= n ? 16u << (k & 1) : 0u);
          } else {
            stream |= 1u | (k == 0 ? 4u : 0u) | (k + 1 == n ? 16u : 0u);
          }
          out.stream = stream;
          out.rest = n - 1 - k;
          out.first = k == 0;
        }
      } else if (lane == 0) {
        out.rest = kEnd;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar.ring_full + g % kRing);
      if (!any) break;
      k += kPageWarps;
    }
  } else if (warp >= kSoftmaxWarps) {
    // ---- decode ----
    set_registers<kDecodeRegisters, false>();
    // A warp's positions are its own from the copies on: only the tiles that it writes are shared.
    constexpr int TW = S::kWarpTokens;
    constexpr int kLanes = DP / E;             // of a row
    constexpr int kStep = 32 / kLanes;         // rows at a time
    constexpr int kItems = TW / kStep;         // of a lane, in a tile
    constexpr int kRaw = S::kRaw;
    static_assert(kItems >= 1 && TW * DP / 64 <= 32, "a warp's scales are a word to a lane");
    const int w = warp - kSoftmaxWarps;
    const int my_row = w * TW + lane / kLanes, my_part = lane % kLanes;
    const bool in_row = my_part * E < D;
    const int nb = D / 16;
    // scales: 4 bytes to a lane (E = 32), copied; else one by one through registers, from issue to issue
    const int scale_row = w * TW + (E == 32 ? lane / (DP / 64) : 0), scale_word = lane % (DP / 64);
    const bool scale_lane = lane < TW * (DP / 64) && scale_word * 4 < nb;
    constexpr int kBytesEach = TW * (DP / 16) / 32;  // of a lane
    uint32_t carried[2] = {0, 0};
    auto code_slot = [&](uint32_t g, int kv) { return base + S::kCodes + ((g % kRaw) * 2 + kv) * S::kCodeBytes; };
    auto scale_slot = [&](uint32_t g, int kv) { return S::kScales + ((g % (kRaw + 1)) * 2 + kv) * S::kScaleBytes; };
    auto issue_scales = [&](uint32_t g) {
      const Tile& tile = sh.ring[g % kRing];
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint8_t* const sf = kv ? a.vc.sf : a.kc.sf;
        const uint32_t stride = kv ? a.v_sf_stride : a.k_sf_stride;
        if constexpr (E == 32) {
          if (scale_lane) {
            const uint2 at = tile.where[scale_row];
            const bool in = at.x != kNoPage;
            cp_async<4>(base + scale_slot(g, kv) + scale_row * (DP / 16) + 4 * scale_word,
                        in ? sf + static_cast<uint64_t>(at.x) * stride + static_cast<uint64_t>(at.y) * nb + 4 * scale_word : sf, in);
          }
        } else {
          carried[kv] = 0;
#pragma unroll
          for (int i = 0; i < kBytesEach; ++i) {
            const int n = lane * kBytesEach + i, row = w * TW + n / (DP / 16), block = n % (DP / 16);
            const uint2 at = tile.where[row];
            if (at.x != kNoPage && block < nb)
              carried[kv] |= static_cast<uint32_t>(__ldg(sf + static_cast<uint64_t>(at.x) * stride + static_cast<uint64_t>(at.y) * nb + block)) << (8 * i);
          }
        }
      }
    };
    // the carried scales of tile g to their slots
    auto put_scales = [&](uint32_t g) {
#pragma unroll
      for (int kv = 0; kv < 2; ++kv)
#pragma unroll
        for (int i = 0; i < kBytesEach; ++i)
          smem[scale_slot(g, kv) + w * TW * (DP / 16) + lane * kBytesEach + i] = static_cast<uint8_t>(carried[kv] >> (8 * i));
    };
    auto issue_codes = [&](uint32_t g, int kv) {
      const uint2* where = sh.ring[g % kRing].where + my_row;
      const uint8_t* const codes = (kv ? a.vc.data : a.kc.data) + my_part * (E / 2);
      const uint32_t stride = kv ? a.v_stride : a.k_stride, dst = code_slot(g, kv) + my_row * (DP / 2) + my_part * (E / 2);
      if (!in_row) return;
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const uint2 at = where[i * kStep];
        const bool in = at.x != kNoPage;
        cp_async<E / 2>(dst + i * kStep * (DP / 2),
                        in ? codes + static_cast<uint64_t>(at.x) * stride + static_cast<uint64_t>(at.y) * static_cast<uint32_t>(D / 2) : codes, in);
      }
    };
    // NaN scales of V, for the softmax (they are taken as 0 in the tile)
    auto find_nan = [&](uint32_t g) {
      Tile& tile = sh.ring[g % kRing];
      uint32_t bad = 0;
      const uint8_t* const sf = smem + scale_slot(g, 1) + my_row * (DP / 16) + my_part * (E / 16);
      auto scale_of = [&](int i) -> uint32_t {
        return !in_row ? 0u : (E == 32 ? *reinterpret_cast<const uint16_t*>(sf + i * kStep * (DP / 16)) : sf[i * kStep * (DP / 16)]);
      };
#pragma unroll
      for (int i = 0; i < kItems; ++i) bad |= ((scale_of(i) & 0x7F7Fu) + 0x0101u) & 0x8080u;
      const bool any = __any_sync(0xFFFFFFFFu, bad != 0);
      if (any) {
#pragma unroll 1
        for (int i = 0; i < kItems; ++i) {
          const uint32_t x = scale_of(i);
          uint32_t blocks = 0;
          for (int b = 0; b < E / 16; ++b)
            if ((x >> (8 * b) & 0x7Fu) == 0x7Fu) blocks |= 1u << (my_part * (E / 16) + b);
          for (int o = 1; o < kLanes; o <<= 1) blocks |= __shfl_xor_sync(0xFFFFFFFFu, blocks, o);
          if (my_part == 0) tile.nan_blocks[my_row + i * kStep] = static_cast<uint16_t>(blocks);
        }
      }
      if (lane == 0) tile.nan[w] = any;
    };
    // Decoded rows to a tile's atoms. Lanes of a row whose chunks would meet in the same banks store them in
    // another order (DP = 128: 8 lanes are two rows of two atoms; 256: one row of four).
    auto decode = [&](uint32_t g, int kv) {
      if (!in_row) return;
      const uint32_t tile = base + S::kK + (2 * kv + (g & 1)) * S::kTileBytes;
      const uint8_t* const codes = smem + (code_slot(g, kv) - base) + my_row * (DP / 2) + my_part * (E / 2);
      const uint8_t* const sf = smem + scale_slot(g, kv) + my_row * (DP / 16) + my_part * (E / 16);
#pragma unroll 2
      for (int i = 0; i < kItems; ++i) {
        const int row = my_row + i * kStep;
        uint32_t sc = E == 32 ? *reinterpret_cast<const uint16_t*>(sf + i * kStep * (DP / 16)) : sf[i * kStep * (DP / 16)] * 0x0101u;
        if (kv) sc &= ~((((sc & 0x7F7Fu) + 0x0101u) & 0x8080u) / 128 * 255);
        const uint32_t s2 = f16x2_from_e4m3x2(sc);
        auto put = [&](uint32_t word, uint32_t scale, uint32_t dst) {
          uint32_t x[4];
          f16x2x4_from_e2m1x8(word, x[0], x[1], x[2], x[3]);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(hmul2_rn(x[0], scale)), "r"(hmul2_rn(x[1], scale)),
                       "r"(hmul2_rn(x[2], scale)), "r"(hmul2_rn(x[3], scale)) : "memory");
        };
        if constexpr (E == 32) {
          const int atom = my_part >> 1;
          const uint32_t at = tile + atom * (BN * 128) + row * 128;
          const int turn = DP == 128 ? 2 * (atom & 1) : (DP == 256 ? atom : 0);
          const uint4 raw = *reinterpret_cast<const uint4*>(codes + i * kStep * (DP / 2));
          const bool two = turn & 2, one = turn & 1;
          uint32_t r[4] = {two ? raw.z : raw.x, two ? raw.w : raw.y, two ? raw.x : raw.z, two ? raw.y : raw.w};
          if (DP == 256) {
            const uint32_t q[4] = {r[0], r[1], r[2], r[3]};
#pragma unroll
            for (int j = 0; j < 4; ++j) r[j] = one ? q[j ^ 1] : q[j];
          }
          const uint32_t s_lo = two ? high_twice(s2) : low_twice(s2), s_hi = two ? low_twice(s2) : high_twice(s2);
#pragma unroll
          for (int j = 0; j < 4; ++j) put(r[j], j < 2 ? s_lo : s_hi, at + (((4 * (my_part & 1) + (j ^ turn)) ^ (row & 7)) << 4));
        } else {
          const uint32_t at = tile + (my_part >> 2) * (BN * 128) + row * 128;
          const uint2 raw = *reinterpret_cast<const uint2*>(codes + i * kStep * (DP / 2));
          put(raw.x, s2, at + (((2 * (my_part & 3)) ^ (row & 7)) << 4));
          put(raw.y, s2, at + (((2 * (my_part & 3) + 1) ^ (row & 7)) << 4));
        }
      }
    };
    bool live[kRaw + 1] = {};  // whether tiles g .. g + kRaw are there
    bool ok = !a.pipe.stall;   // (a test: nothing comes, and every wait runs out)
#pragma unroll 1
    for (int32_t g = -kRaw; ok; ++g) {
      const uint32_t ahead = g + kRaw;
      const bool due = g >= 0 && live[0];
      if (g >= 0 && !due) break;
      if (E != 32 && ahead > 0 && live[kRaw - 1]) put_scales(ahead - 1);
      live[kRaw] = (g < 0 ? ahead == 0 || live[kRaw - 1] : live[kRaw - 1]) &&
                   wait_warp(bar.ring_full + ahead % kRing, ahead / kRing & 1) && sh.ring[ahead % kRing].rest != kEnd;
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        if (due) {
          cp_async_wait<2 * kRaw - 1>();
          __syncwarp();
          if (kv == 0) find_nan(g);
          if (!wait_warp(bar.empty + 2 * kv + (g & 1), ((g >> 1) & 1) ^ 1)) {
            ok = false;
            break;
          }
          decode(g, kv);
          fence_async_proxy();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar.full + 2 * kv + (g & 1));
        }
        if (live[kRaw]) {
          if (kv == 0) issue_scales(ahead);
          issue_codes(ahead, kv);
        }
        cp_async_commit();
      }
#pragma unroll
      for (int i = 0; i < kRaw; ++i) live[i] = live[i + 1];
    }
    cp_async_wait<0>();
  } else {
    // ---- softmax ----
    set_registers<kSoftmaxRegisters, true>();
    if (!kOne || warp < 4) {
    const int stream = warp >> 2, quarter = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(quarter) << 21;  // this warp's lanes of tensor memory
    const float gk = __ldg(a.k_scale), gv = __ldg(a.v_scale);
    const float cap = a.soft_cap;
    uint32_t tiles = 0, q_count = 0, o_count = 0, merges = 0, steps = 0;
    uint32_t s_count[2] = {0, 0};
    // -- the queries --
    // A warp brings its own rows: as they are, by asynchronous copies to where the products will read them, and
    // then turns them in place into binary16, each row scaled by a power of two. kPer lanes share a row.
    constexpr int kPer = kTurns ? 2 : 1;
    const int q_row = kTurns ? warp * 16 : (kTwo ? warp * 32 : quarter * 32);  // this warp's first
    const int width = D / 8;                                                  // 16-byte chunks of a row
    auto chunk = [&](int row, int j) -> uint8_t* {
      const int r = row & 127;
      return smem + (row >> 7) * S::kQBytes + (j >> 3) * 16384 + r * 128 + (((j & 7) ^ (r & 7)) << 4);
    };
    auto fetch = [&](const Segment& s) {
      int log_t = 0;
      while ((1 << log_t) < width) ++log_t;
      const int j = lane & ((1 << log_t) - 1), step = 32 >> log_t;
      const int32_t first = s.t * S::kRows, rows = s.q.n * a.G - first;
      if (j < width) {
#pragma unroll 1
        for (int i = q_row + (lane >> log_t); i < q_row + 32 / kPer; i += step) {
          const bool in = i < rows;
          const int32_t row = in ? first + i : first, tk = div_q32(row, a.div_g);
          const int64_t hd = static_cast<int64_t>(s.h) * a.G + (row - tk * a.G);
          cp_async<16>(smem_addr(chunk(i, j)), a.q + (s.q.q0 + tk) * a.q_row_bytes + hd * D * 2 + 16 * j, in);
        }
      }
      cp_async_commit();
    };
    fetch(sh.first);
    for (bool begun = false;; begun = true) {
      const Segment s = begun ? sh.next[warp] : sh.first;
      const bool final = !more(s);
      const Portion part = portion_of(s, run);
      const int32_t n = part.end - part.u;
      const int32_t r0 = s.t * S::kRows, rows = min(s.q.n * a.G - r0, S::kRows);  // the segment's first, and their count
      const int local = (kTwo ? 128 * stream : 0) + quarter * 32 + lane;          // this thread's row of them
      const bool alive = local < rows;
      const int32_t token = div_q32(alive ? r0 + local : 0, a.div_g), head = (alive ? r0 + local : 0) - token * a.G;
      uint8_t* const out = a.out + ((s.q.q0 + token) * a.Hq + static_cast<int64_t>(s.h) * a.G + head) * D * 2;
      float* const lse = a.lse ? a.lse + (s.q.q0 + token) * a.Hq + static_cast<int64_t>(s.h) * a.G + head : nullptr;
      if (n == 0 && part.mine && stream == (kTwo ? stream : 0) && alive) {  // nothing that any row sees
        for (int i = 0; i < D / 8; ++i) reinterpret_cast<uint4*>(out)[i] = uint4{};
        if (lse) *lse = -INFINITY;
      }
      Reach reach{0, 0, n};  // this stream's tiles of the portion
      if constexpr (kTwo) reach = reach_of_half<S>(a, s, part, stream);
      const bool mine = reach.any();
      if (final) {
        // the run's last segment, if others continue it
        if (tid == 0 && s.units > kWholeUnits && s.start >= 0 && s.start < run && s.start + s.units > run) {
          PrefillCut* const cuts = reinterpret_cast<PrefillCut*>(static_cast<uint8_t*>(a.workspace) + NVFP4_COUNTER_BYTES);
          cuts[blockIdx.x] = {s.b, s.t, s.h, static_cast<int32_t>(cut.run_of(c0 + s.start + s.units - 1))};
        }
      } else {  // (kept in shared memory: the registers are for the scores)
        Segment next = s;
        next_segment<S>(a, next);
        __syncwarp();
        if (lane == 0) sh.next[warp] = next;
        __syncwarp();
      }
      if (n > 0) {
        if (mine) {
          cp_async_wait<0>();
          __syncwarp();
          const int row = q_row + lane / kPer;
          float top = 0.0f;
#pragma unroll 1
          for (int j = lane % kPer; j < width; j += kPer) {
            const uint4 raw = *reinterpret_cast<const uint4*>(chunk(row, j));
            const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float v0 = a.bf16 ? __uint_as_float(x[e] << 16) : f32_from_f16_lo(x[e]);
              const float v1 = a.bf16 ? f32_from_bf16_hi(x[e]) : f32_from_f16_hi(x[e]);
              top = max3(top, fabsf(v0), fabsf(v1));
            }
          }
          if (kPer == 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
          const int exponent = max(static_cast<int>(__float_as_uint(top) >> 23), 1) - 127;
          const int e2 = top > 0.0f && top <= FLT_MAX ? exponent - 14 : 0;
          // 2^e2 and 2^-e2 as two factors (they may be out of range by themselves), with f's sign: f is not
          // negative from here on, and a maximum of scores is one of logits; f = 0 is a query of zeros
          float f = (a.sm_scale * __int_as_float((127 + e2 / 2) << 23)) * (gk * __int_as_float((127 + (e2 - e2 / 2)) << 23));
          float f1 = __int_as_float((127 - e2 / 2) << 23);
          const float f2 = __int_as_float((127 - (e2 - e2 / 2)) << 23);
          if (f < 0.0f) f1 = -f1;
          if (f == 0.0f) f1 = 0.0f;
          f = f == 0.0f ? 1.0f : fabsf(f);
#pragma unroll 1
          for (int j = lane % kPer; j < width; j += kPer) {
            uint4* const at = reinterpret_cast<uint4*>(chunk(row, j));
            const uint4 raw = *at;
            uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float v0 = a.bf16 ? __uint_as_float(x[e] << 16) : f32_from_f16_lo(x[e]);
              const float v1 = a.bf16 ? f32_from_bf16_hi(x[e]) : f32_from_f16_hi(x[e]);
              x[e] = f16x2_from_f32(v0 * f1 * f2, v1 * f1 * f2);
            }
            *at = make_uint4(x[0], x[1], x[2], x[3]);
          }
          sh.factor[row] = f;
          fence_async_proxy();
          __syncwarp();
          uint64_t* const full = bar.q_full + (kTwo ? stream : 0);
          if (lane == 0) mbar_arrive(full);
          if (!wait_warp(full, q_count++ & 1)) break;
        }
        // -- this row --
        const float f = mine ? sh.factor[local] : 1.0f;
        const float unit2 = f * kLog2e;  // what turns a sum of products into base-2 logarithms
        // cap tanh(x / cap) of x = f v, by 1 - 2 / (e^(2x/cap) + 1): absolute error a few 2^-24 of the cap
        const float turn2 = cap > 0.0f ? f / cap * (2.0f * kLog2e) : 0.0f;
        auto capped = [&](float v) { return cap * __fmaf_rn(-2.0f, rcp(ex2(v * turn2) + 1.0f), 1.0f); };
        const int32_t p = s.q.L - s.q.n + token;
        const int32_t hi = !alive ? 0 : (a.causal ? min(max(p + 1, 0), s.q.L) : s.q.L);
        const int32_t lo = a.window_left >= 0 && p > a.window_left ? p - a.window_left : 0;
        const int32_t sink = a.window_left >= 0 ? a.sink : 0;
        const bool busy = __any_sync(0xFFFFFFFFu, alive);
        const int32_t all_hi = __reduce_min_sync(0xFFFFFFFFu, alive ? hi : INT32_MAX);
        const int32_t all_lo = __reduce_max_sync(0xFFFFFFFFu, alive ? lo : 0);
        float m = -INFINITY, l = 0.0f;
        uint32_t poison = 0;
        bool started = false, ok = true;
        for (int32_t k = kTurns ? stream : 0; k < n; k += kTurns ? 2 : 1) {
          const int32_t t0 = tile_of_unit<BN>(part.u + k, s.first_units, s.gap);
          if (kTwo && !reach.has(k)) continue;
          const int buf = kTwo ? stream : k & 1;
          ok = wait_warp(bar.s_full + buf, s_count[buf]++ & 1);
          if (!ok) break;
          tc_fence_after();
          const Tile& tile = sh.ring[(tiles + k) % kRing];
          const uint4 about = *reinterpret_cast<const uint4*>(tile.nan);  // nan, stream, rest
          const uint32_t s_at = tmem + lanes + buf * BN;
          if (busy) {
            const bool full = t0 + BN <= all_hi && (t0 >= all_lo || t0 + BN <= sink) && (about.z & 512);
            auto weigh = [&](auto masked_, auto capped_) {
              constexpr bool kMasked = decltype(masked_)::value, kCapped = decltype(capped_)::value;
              constexpr int NC = BN / 32;  // words of 32 positions
              float x[32], y[32], tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
              auto seen = [&](int c) -> uint32_t {  // which of a word's
                const int32_t t = t0 + 32 * c;
                return tile.live[c] & low_bits(hi - t) & (~low_bits(lo - t) | low_bits(sink - t));
              };
              auto take = [&](float (&v)[32], int c) {
                tmem_loaded(v);
                const uint32_t word = kMasked ? seen(c) : 0u;
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                  const float v0 = kMasked && !(word >> e & 1u) ? -INFINITY : v[e];
                  const float v1 = kMasked && !(word >> (e + 1) & 1u) ? -INFINITY : v[e + 1];
                  tops[e / 2 % 4] = max3(tops[e / 2 % 4], v0, v1);
                }
              };
              tmem_load(x, s_at);
              tmem_wait();
#pragma unroll 1
              for (int c = 0; c < NC; c += 2) {
                tmem_load(y, s_at + 32 * (c + 1));
                take(x, c);
                tmem_wait();
                tmem_load(x, c + 2 < NC ? s_at + 32 * (c + 2) : s_at);  // (at last the first again, for the weights)
                take(y, c + 1);
                tmem_wait();
              }
              float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
              top = kCapped ? capped(top) * kLog2e : top * unit2;
              const bool rises = top > m + kSlack;  // (by row: a result does not depend on other rows)
              if (__any_sync(0xFFFFFFFFu, rises)) {
                const float g = rises ? ex2(m - top) : 1.0f;
                m = rises ? top : m;
                l *= g;
                if (started) {
                  if (kOne && !wait_warp(&bar.o_step, (steps - 1) & 1)) return false;
                  tc_fence_after();
                  const uint32_t o_at = tmem + lanes + S::kO + (kOne ? 0 : stream * DP);
#pragma unroll 1
                  for (int d = 0; d < D; d += 16) {
                    float o[16];
                    tmem_load(o, o_at + d);
                    tmem_wait();
                    tmem_loaded(o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] *= g;
                    tmem_store(o_at + d, o);
                  }
                }
              }
              const float off = m == -INFINITY ? 0.0f : kWeightBias - m;
              float sum[4] = {0, 0, 0, 0};
              auto put = [&](float (&v)[32], int c) {
                tmem_loaded(v);
                const uint32_t word = kMasked ? seen(c) : 0u;
                uint32_t p[16];
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                  float v0 = kCapped ? capped(v[e]) : v[e], v1 = kCapped ? capped(v[e + 1]) : v[e + 1];
                  if (kMasked) {
                    v0 = word >> e & 1u ? v0 : -INFINITY;
                    v1 = word >> (e + 1) & 1u ? v1 : -INFINITY;
                  }
                  fma2(v0, v1, kCapped ? kLog2e : unit2, off);
                  v0 = ex2(v0);
                  v1 = ex2(v1);
                  add2(sum[e % 4], sum[e % 4 + 1], v0, v1);
                  p[e / 2] = f16x2_from_f32(v0, v1);
                }
                tmem_store(s_at + 16 * c, p);
              };
#pragma unroll 1
              for (int c = 0; c < NC; c += 2) {
                tmem_load(y, s_at + 32 * (c + 1));
                put(x, c);
                tmem_wait();
                if (c + 2 < NC) tmem_load(x, s_at + 32 * (c + 2));
                put(y, c + 1);
                tmem_wait();
              }
              l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
              return true;
            };
            using T = std::true_type;
            using F = std::false_type;
            if (cap > 0.0f) ok = weigh(T{}, T{});
            else ok = full ? weigh(F{}, F{}) : weigh(T{}, F{});
            if (!ok) break;
            // blocks of V that are NaN, where this row sees them
            if (about.x | about.y) {
#pragma unroll 1
              for (int c = 0; c < BN; ++c) {
                const int32_t t = t0 + c;
                if (tile.nan[c / S::kWarpTokens] && t < hi && (t >= lo || t < sink)) poison |= tile.nan_blocks[c];
              }
            }
            __syncwarp();
            tmem_wait_stores();
          }
          started = true;
          ++steps;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar.p_full + buf);
        }
        if (!ok) break;
        // -- the segment's end --
        if (started) {
          if (!wait_warp(bar.o_full + (kOne ? 0 : stream), o_count++ & 1)) break;
          tc_fence_after();
        }
        bool two = false;      // the second stream has a part too
        float m1 = -INFINITY, l1 = 0.0f;
        if (kTurns) {
          if (stream == 1) {
            const int r = quarter * 32 + lane;
            sh.m[r] = m;
            sh.l[r] = l;
            sh.poison[r] = poison;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.merge);
          if (!wait_warp(&bar.merge, merges++ & 1)) break;
          two = n > 1;
          if (stream == 0 && two) {
            m1 = sh.m[local];
            l1 = sh.l[local];
            poison |= sh.poison[local];
          }
        }
        // the products of this segment's queries are done: the next ones may come
        cp_async_wait<0>();
        if (!final) fetch(sh.next[warp]);
        if (busy && (!kTurns || stream == 0)) {
          const bool whole = part.u == 0 && part.end == s.units;
          const float top = fmaxf(m, m1);
          // nothing above -inf: the sums are zeros, or NaN where every score was NaN, which has to stay
          const float g0 = top == -INFINITY ? 1.0f : ex2(m - top), g1 = top == -INFINITY ? 1.0f : ex2(m1 - top);
          const float sum = two ? g0 * l + g1 * l1 : l;
          const float scale = whole ? (sum == 0.0f ? 0.0f : gv / sum) : 1.0f;
          const float w0 = (two ? g0 : 1.0f) * scale, w1 = g1 * scale;
          float* const part_o = whole ? nullptr : part_of(a, blockIdx.x, s.start < 0 ? 0 : 1, S::kRows, DP);
          const uint32_t o_at = tmem + lanes + S::kO + (kOne || kTurns ? 0 : stream * DP);
#pragma unroll 1
          for (int d = 0; d < D; d += 32) {  // (head_dim may end in the middle: what lies past it is not stored)
            float o[32] = {};
            __syncwarp();
            if (started) {
              tmem_load(o, o_at + d);
              tmem_wait();
              tmem_loaded(o);
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= w0;
            if (two) {
              float x[32];
              tmem_load(x, o_at + DP + d);
              tmem_wait();
              tmem_loaded(x);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] += w1 * x[i];
            }
            if (poison >> (d / 16) & 3u) {
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = poison >> (d / 16 + i / 16) & 1u ? NAN : o[i];
            }
            if (alive && whole) {
              uint4* const dst = reinterpret_cast<uint4*>(out + d * 2);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float v0 = o[8 * k + 2 * i], v1 = o[8 * k + 2 * i + 1];
                  y[i] = a.bf16 ? bf16x2_from_f32(v0, v1) : f16x2_from_f32(v0, v1);
                }
                if (k < 2 || d + 16 < D) dst[k] = make_uint4(y[0], y[1], y[2], y[3]);
              }
            } else if (alive) {
              float4* dst = reinterpret_cast<float4*>(part_o + static_cast<int64_t>(local) * DP + d);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (i < 4 || d + 16 < D) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
          }
          if (alive) {
            if (whole) {
              if (lse) *lse = sum == 0.0f ? -INFINITY : (top - kWeightBias) * (1.0f / kLog2e) + logf(sum);
            } else {
              part_o[S::kRows * DP + local] = top;
              part_o[S::kRows * (DP + 1) + local] = sum;
            }
          }
          tc_fence_before();  // (these reads come before the next segment's products)
        }
        tiles += n;
      } else if (!final) {
        cp_async_wait<0>();
        fetch(sh.next[warp]);
      }
      if (final) break;
      __syncwarp();
    }
    cp_async_wait<0>();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && sh.dead) flag(a.status, NVFP4_DEV_TIMEOUT);
  if (warp == kProductWarp) {
    tc_fence_after();
    tmem_free(tmem);
  }
}

// The parts of the segment that run blockIdx.x begins and others continue, added in the runs' order, a row to a warp.
constexpr int kJoinRows = 8;
template <int DP, int MT>
__global__ void __launch_bounds__(256) join_kernel(const PrefillArgs a) {
  using S = Shape<DP, MT>;
  const PrefillCut c = reinterpret_cast<const PrefillCut*>(static_cast<const uint8_t*>(a.workspace) + NVFP4_COUNTER_BYTES)[blockIdx.x];
  if (c.last < 0) return;
  const Request q = request_of(a, c.b);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = a.D;
  const int32_t r0 = c.t * S::kRows, rows = q.n * a.G - r0;
  const int64_t first = blockIdx.x;
  const float gv = __ldg(a.v_scale);
  for (int k = 0; k < kJoinRows / 8; ++k) {
    const int local = blockIdx.y * kJoinRows + warp * (kJoinRows / 8) + k;
    if (local >= rows) return;
    auto part = [&](int64_t i) { return part_of(a, i, i == first ? 1 : 0, S::kRows, DP); };
    float top = -INFINITY;
    for (int64_t i = first + lane; i <= c.last; i += 32) top = fmaxf(top, part(i)[S::kRows * DP + local]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    // nothing above -inf: the sums are zeros, or NaN where every score was NaN, which has to stay
    const bool none = top == -INFINITY;
    float sum = 0.0f;
    float4 v[DP / 128 + 1] = {};
#pragma unroll 4
    for (int64_t i = first; i <= c.last; ++i) {
      const float* p = part(i);
      const float g = none ? 1.0f : ex2(p[S::kRows * DP + local] - top);
      sum += g * p[S::kRows * (DP + 1) + local];
#pragma unroll
      for (int e = 0; e < (DP + 127) / 128; ++e) {
        const int d = e * 128 + lane * 4;
        if (d < D) {
          const float4 x = *reinterpret_cast<const float4*>(p + static_cast<int64_t>(local) * DP + d);
          v[e].x += g * x.x; v[e].y += g * x.y; v[e].z += g * x.z; v[e].w += g * x.w;
        }
      }
    }
    const float f = sum == 0.0f ? 0.0f : gv / sum;
    const int32_t token = div_q32(r0 + local, a.div_g);
    const int64_t row = (q.q0 + token) * a.Hq + static_cast<int64_t>(c.h) * a.G + (r0 + local - token * a.G);
#pragma unroll
    for (int e = 0; e < (DP + 127) / 128; ++e) {
      const int d = e * 128 + lane * 4;
      if (d < D) {
        uint2 w;
        w.x = a.bf16 ? bf16x2_from_f32(v[e].x * f, v[e].y * f) : f16x2_from_f32(v[e].x * f, v[e].y * f);
        w.y = a.bf16 ? bf16x2_from_f32(v[e].z * f, v[e].w * f) : f16x2_from_f32(v[e].z * f, v[e].w * f);
        *reinterpret_cast<uint2*>(a.out + (row * D + d) * 2) = w;
      }
    }
    if (lane == 0 && a.lse) a.lse[row] = sum == 0.0f ? -INFINITY : (top - kWeightBias) * (1.0f / kLog2e) + logf(sum);
  }
}

template <int DP, int MT, int E>
nvfp4_status launch_t(PrefillArgs a, cudaStream_t stream) {
  using S = Shape<DP, MT>;
  const char* fn = "nvfp4_paged_attention_prefill";
  const auto kern = prefill_kernel<DP, MT, E>;
  const size_t smem = S::kBytes + 1024;
  static_assert(S::kBytes >= kMaxScanBatch * 4, "the requests' tiles are counted where the tiles will be");
  int64_t grid;
  if (nvfp4_status st = resident_ctas(reinterpret_cast<const void*>(kern), kThreads, smem, 1, fn, &grid)) return st;
  a.parts_offset = NVFP4_COUNTER_BYTES + (grid * sizeof(PrefillCut) + 127) / 128 * 128;
  kern<<<static_cast<int>(grid), kThreads, smem, stream>>>(a);
  if (nvfp4_status st = check_launch(fn)) return st;
  if (a.max_pages * a.ps <= static_cast<int64_t>(kWholeUnits) * S::BN) return NVFP4_OK;  // no segment is cut
  join_kernel<DP, MT><<<dim3(static_cast<unsigned>(grid), S::kRows / kJoinRows), 256, 0, stream>>>(a);
  return check_launch(fn);
}

template <int DP, int MT>
nvfp4_status launch_e(const PrefillArgs& a, cudaStream_t s) {
  // 16-byte copies of codes and 4-byte copies of scales
  auto even = [](const nvfp4_paged_cache& c) { return reinterpret_cast<uintptr_t>(c.sf) % 4 == 0 && c.sf_page_stride % 4 == 0; };
  return a.D % 64 == 0 && even(a.kc) && even(a.vc) ? launch_t<DP, MT, 32>(a, s) : launch_t<DP, MT, 16>(a, s);
}

}  // namespace

int64_t prefill_workspace_bytes(int32_t D) {
  const int64_t dp = D <= 64 ? 64 : (D <= 128 ? 128 : 256), rows = D <= 128 ? 256 : 128, n = sm_count();
  return NVFP4_COUNTER_BYTES + (n * sizeof(PrefillCut) + 127) / 128 * 128 + 2 * n * rows * (dp + 2) * 4;
}

nvfp4_status launch_prefill(PrefillArgs a, cudaStream_t stream) {
  a.pool_pages = a.kc.num_pages < a.vc.num_pages ? a.kc.num_pages : a.vc.num_pages;
  const int64_t strides[4] = {a.kc.data_page_stride, a.vc.data_page_stride, a.kc.sf_page_stride, a.vc.sf_page_stride};
  for (int64_t s : strides)
    if (s > static_cast<int64_t>(UINT32_MAX)) return fail(NVFP4_ERR_UNSUPPORTED, "nvfp4_paged_attention_prefill: a page stride above 4 GiB");
  a.k_stride = static_cast<uint32_t>(strides[0]);
  a.v_stride = static_cast<uint32_t>(strides[1]);
  a.k_sf_stride = static_cast<uint32_t>(strides[2]);
  a.v_sf_stride = static_cast<uint32_t>(strides[3]);
  a.pipe = pipe_test_from_env();
  a.pipe.wait_limit = std::min(a.pipe.wait_limit, kNapLimit);
  a.few_rows = few_rows_of(a.nnz * a.G, a.D, a.B, a.H, a.max_pages * a.ps);
  if (a.few_rows > 0) {
    AttentionArgs f{};
    f.q = a.q; f.q_row_bytes = a.q_row_bytes;
    f.kc = a.kc; f.vc = a.vc;
    f.ps = a.ps; f.Hq = a.Hq; f.H = a.H; f.G = a.G; f.D = a.D; f.layout = a.layout; f.B = a.B;
    f.bf16 = a.bf16; f.table64 = a.table64;
    f.div_ps = a.div_ps;
    f.block_tables = a.block_tables; f.max_pages = a.max_pages; f.seq_lens = a.seq_lens;
    f.k_scale = a.k_scale; f.v_scale = a.v_scale;
    f.sm_scale = a.sm_scale; f.soft_cap = a.soft_cap;
    f.window_left = a.window_left; f.sink = a.sink;
    f.out = a.out; f.lse = a.lse; f.status = a.status; f.workspace = a.workspace;
    f.qo_indptr = a.qo_indptr; f.nnz = a.nnz; f.causal = a.causal;
    f.most_rows = a.few_rows;
    if (nvfp4_status st = launch_attention(f, stream)) return st;
  }
  // 256 rows of a segment share the decoded tiles; requests of fewer rows than 128 have no use for them
  const bool two = a.nnz * a.G > static_cast<int64_t>(a.B) * 128;
  if (a.D > 128) return launch_e<256, 1>(a, stream);
  if (a.D > 64) return two ? launch_e<128, 2>(a, stream) : launch_e<128, 1>(a, stream);
  return two ? launch_e<64, 2>(a, stream) : launch_e<64, 1>(a, stream);
}

}  // namespace nvfp4
