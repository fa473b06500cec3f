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
// A CTA (one to an SM) has three kinds of warps, which wait for one another on mbarriers only:
//   load     (8 warps, in two groups that take every second tile) pages are looked up, codes and scales loaded two
//            tiles ahead into registers, decoded to e2m1 * S, exact in binary16, and written to shared memory in
//            the tensor cores' order;
//   product  (one thread) S = Q K^T and O += P V by tcgen05.mma, sums in tensor memory;
//   softmax  (8 warps, a row to a thread) S from tensor memory, its running maximum and sum, P in binary16 back to
//            tensor memory over S; at a segment's end O to the output. They also bring the next queries.
// Two streams keep the tensor cores busy while the other one is at its weights: the two halves of 256 rows over the
// same tiles, or the same 128 rows over every second tile, joined at the end. head_dim above 128 leaves tensor
// memory for one stream: there S of the next tile is computed meanwhile.
//
// Queries are scaled row by row by a power of two into binary16 (what is below 2^-38 of a row's largest element is
// lost), weights are rounded to binary16 (2^-11 relative), as in attention.cu, and so are the running maximum and
// sum kept. A NaN block scale of V is taken as 0 in the product and the outputs that see it are set to NaN: a weight
// of 0 would not keep it from rows that do not.
#include "attention.h"
#include "softmax.cuh"
#include "tcgen05.cuh"

#include <cfloat>

namespace nvfp4 {
namespace {

constexpr int kSoftmaxWarps = 8;
constexpr int kLoadWarps = 4;   // of a group
constexpr int kLoadGroups = 2;
constexpr int kProductWarp = kSoftmaxWarps + kLoadGroups * kLoadWarps;
constexpr int kWarps = kProductWarp + 4;  // (three of the last warpgroup have nothing to do)
// Registers of a thread of each warpgroup: the launch's 96 for 640 threads, dealt out again. 2 x 144 + 2 x 72 + 48 =
// 5 x 96.
constexpr int kLaunchRegisters = 96, kSoftmaxRegisters = 144, kLoadRegisters = 72, kProductRegisters = 48;
static_assert(2 * kSoftmaxRegisters + 2 * kLoadRegisters + kProductRegisters <= 5 * kLaunchRegisters, "more than the launch has");
constexpr int kThreads = kWarps * 32;
constexpr int kMeta = 4;          // tiles whose masks are kept
constexpr int kSegmentCost = 2;   // what a segment's queries and outputs count for, in tiles
constexpr int kWholeUnits = 8;    // a segment of so few tiles is not cut

// DP: head_dim rounded up to 64, 128 or 256. MT: 128 rows of a segment, or twice as many.
template <int DP, int MT>
struct Shape {
  static constexpr int BN = DP > 128 ? 64 : 128;     // positions of a tile
  static constexpr int kRows = 128 * MT;
  static constexpr int kQBytes = 128 * DP * 2;       // of 128 rows
  static constexpr int kTileBytes = BN * DP * 2;
  static constexpr int kK = MT * kQBytes, kV = kK + 2 * kTileBytes, kBytes = kV + 2 * kTileBytes;
  static constexpr int kWarpTokens = BN / kLoadWarps;
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
  return {p0, static_cast<int32_t>(p1 - p0), n > reach ? static_cast<int32_t>(reach) : n};
}

// Positions that rows [r0, r1) of a request see: t < hi and (t >= lo or t < sink).
struct Sight {
  int32_t hi, lo, sink;
};
__device__ __forceinline__ Sight sight_of(const PrefillArgs& a, const Request& q, int64_t r0, int64_t r1) {
  const int32_t first = q.L - q.n + static_cast<int32_t>(quotient64(r0, a.G));
  const int32_t last = q.L - q.n + static_cast<int32_t>(quotient64(r1 - 1, a.G));
  Sight s;
  s.hi = a.causal ? max(last + 1, 0) : q.L;
  s.lo = a.window_left >= 0 && first > a.window_left ? min(first - a.window_left, s.hi) : 0;
  s.sink = min(a.sink, s.lo);
  return s;
}
template <int BN>
__device__ __forceinline__ bool sees(const Sight& s, int32_t t0) {  // some position of the tile at t0
  return t0 < s.hi && (t0 + BN > s.lo || t0 < s.sink);
}

// A segment, and the place of its first tile relative to the run's first.
struct Segment {
  int32_t b, t, h, units;
  int64_t start;
  Request q;
  Sight see;
  int32_t first_units, gap;
};

template <class S>
__device__ __forceinline__ void fill(const PrefillArgs& a, Segment& s) {
  const int64_t rows = static_cast<int64_t>(s.q.n) * a.G, r0 = static_cast<int64_t>(s.t) * S::kRows;
  s.see = sight_of(a, s.q, r0, min(rows, r0 + S::kRows));
  s.first_units = (s.see.sink + S::BN - 1) / S::BN;
  s.gap = max(s.see.lo / S::BN - s.first_units, 0);
  s.units = s.see.hi > 0 ? (s.see.hi - 1) / S::BN + 1 - s.gap : 0;
}
template <class S>
__device__ __forceinline__ int32_t tiles_of(const PrefillArgs& a, const Request& q) {
  return static_cast<int32_t>((static_cast<int64_t>(q.n) * a.G + S::kRows - 1) / S::kRows);
}
__device__ __forceinline__ int32_t places_of(int32_t units) { return units + kSegmentCost; }
// The next segment (the caller knows that there is one).
template <class S>
__device__ __forceinline__ void next_segment(const PrefillArgs& a, Segment& s) {
  s.start += places_of(s.units);
  if (++s.h < a.H) return;
  s.h = 0;
  if (static_cast<int64_t>(++s.t) * S::kRows >= static_cast<int64_t>(s.q.n) * a.G) {
    s.t = 0;
    do s.q = request_of(a, ++s.b);
    while (s.q.n == 0);
  }
  fill<S>(a, s);
}
// The units [u, end) of a segment that are this run's of `run` places; `mine`: it is, wholly, if it is not cut.
struct Portion {
  int32_t u, end;
  bool mine;
};
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
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_full[2], q_full, o_step, merge, done;
};
struct Shared {
  Barriers bar;
  Segment first;                      // the run's
  uint32_t tmem;
  int32_t dead;                       // a wait has run out
  uint32_t live[kMeta][kLoadWarps];   // positions of a tile that are on a page of the pool
  uint32_t nan[kMeta][kLoadWarps];    // a warp's V scales hold NaN
  uint16_t nan_blocks[kMeta][128];    // which blocks of a position (where its warp's nan is set)
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

// E: elements of a row that a lane decodes, 32 (two blocks, 16-byte loads) or 16.
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
  const uint32_t limit = a.pipe.wait_limit;

  // -- the run: tiles of all requests, then places of all tiles --
  int64_t c0, run, ncta;
  Cut cut;
  {
    int32_t* cum = reinterpret_cast<int32_t*>(smem);
    const int per = (a.B + kThreads - 1) / kThreads;
    const int lo = min(a.B, tid * per), hi = min(a.B, lo + per);
    int32_t local = 0;
    for (int b = lo; b < hi; ++b) {
      const Request q = request_of(a, b);
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
    __syncthreads();
    const int32_t tiles = cum[a.B - 1];
    const int32_t per2 = (tiles + kThreads - 1) / kThreads;
    const int32_t f0 = static_cast<int32_t>(min(static_cast<int64_t>(tiles), static_cast<int64_t>(tid) * per2));
    const int32_t f1 = static_cast<int32_t>(min(static_cast<int64_t>(tiles), static_cast<int64_t>(f0) + per2));
    Segment s;
    s.h = 0;
    // every tile of this thread's slice, until `stop` says so
    auto walk = [&](auto stop) {
      int32_t x = 0, y = a.B - 1;
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
        if (static_cast<int64_t>(++s.t) * S::kRows >= static_cast<int64_t>(s.q.n) * a.G) {
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
      mbar_init(bar.k_full + i, kLoadWarps);
      mbar_init(bar.v_full + i, kLoadWarps);
      mbar_init(bar.k_empty + i, 1);
      mbar_init(bar.v_empty + i, 1);
      mbar_init(bar.s_full + i, 1);
      mbar_init(bar.p_full + i, 4);
      mbar_init(bar.o_full + i, 1);
    }
    mbar_init(&bar.q_full, kOne ? 4 : kSoftmaxWarps);
    mbar_init(&bar.o_step, 1);
    mbar_init(&bar.merge, kSoftmaxWarps);
    mbar_init(&bar.done, 1);
    sh.dead = 0;
    fence_mbar_init();
  }
  if (warp == kProductWarp) tmem_alloc(&sh.tmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;

  // A bounded wait; when it runs out, or another role's has, everyone returns.
  auto wait = [&](uint64_t* b, uint32_t parity) -> bool {
    for (uint32_t i = 0; i < limit; ++i) {
      if (mbar_try_wait(b, parity)) return true;
      if ((i & 15) == 15 && *static_cast<volatile int32_t*>(&sh.dead)) return false;
    }
    if (!*static_cast<volatile int32_t*>(&sh.dead)) flag(a.status, NVFP4_DEV_TIMEOUT);
    *static_cast<volatile int32_t*>(&sh.dead) = 1;
    return false;
  };
  auto wait_warp = [&](uint64_t* b, uint32_t parity) -> bool { return __all_sync(0xFFFFFFFFu, wait(b, parity)); };
  auto more = [&](const Segment& s) { return s.start + places_of(s.units) < run; };
  const int D = a.D;
  const uint32_t base = smem_addr(smem);

  if (warp >= kProductWarp) {
    // ---- product ----
    set_registers<kProductRegisters, false>();
    if (warp == kProductWarp && lane == 0) {
      const uint32_t shape_s = mma_shape(BN, false), shape_o = mma_shape(D, true);
      uint32_t unit = 0, q_count = 0;       // tiles so far, segments so far
      uint32_t p_count[2] = {0, 0};
      auto issue_s = [&](int half, int buf, uint32_t g) {
        const uint32_t q = base + half * S::kQBytes, k = base + S::kK + (g & 1) * S::kTileBytes;
        for (int i = 0; i < D / 16; ++i)
          mma_ss(tmem + buf * BN, smem_operand(q + (i >> 2) * 16384 + (i & 3) * 32, 16),
                 smem_operand(k + (i >> 2) * (BN * 128) + (i & 3) * 32, 16), shape_s, i > 0);
        mma_commit(bar.s_full + buf);
      };
      auto issue_o = [&](int stream, int buf, uint32_t g, bool sum) {
        const uint32_t v = base + S::kV + (g & 1) * S::kTileBytes;
        for (int i = 0; i < BN / 16; ++i)
          mma_ts(tmem + S::kO + stream * DP, tmem + buf * BN + 8 * i, smem_operand(v + i * 2048, BN * 128), shape_o, sum || i > 0);
      };
      auto k_ready = [&](uint32_t g) { return wait(bar.k_full + (g & 1), (g >> 1) & 1); };
      auto v_ready = [&](uint32_t g) { return wait(bar.v_full + (g & 1), (g >> 1) & 1); };
      auto p_ready = [&](int buf) {
        if (!wait(bar.p_full + buf, p_count[buf]++ & 1)) return false;
        tc_fence_after();
        return true;
      };
      Segment s = sh.first;
      for (bool ok = true; ok;) {
        const Portion part = portion_of(s, run);
        const int32_t n = part.end - part.u;
        if (n > 0) {
          auto tile = [&](int32_t k) {  // position of the portion's tile k
            const int32_t u = part.u + k;
            return (u < s.first_units ? u : u + s.gap) * BN;
          };
          ok = wait(&bar.q_full, q_count++ & 1);
          if (ok) tc_fence_after();
          if constexpr (kTwo) {
            const int64_t rows = static_cast<int64_t>(s.q.n) * a.G, r0 = static_cast<int64_t>(s.t) * S::kRows;
            Sight see[2];
            int32_t last[2];  // a half's last tile
            for (int i = 0; i < 2; ++i) {
              see[i] = {0, 0, 0};
              if (r0 + 128 * i < rows) see[i] = sight_of(a, s.q, r0 + 128 * i, min(rows, r0 + 128 * i + 128));
              last[i] = n - 1;
              while (last[i] >= 0 && !sees<BN>(see[i], tile(last[i]))) --last[i];
            }
            bool sum[2] = {false, false};
            ok = ok && k_ready(unit);
            if (ok) {
              tc_fence_after();
              for (int i = 0; i < 2; ++i)
                if (sees<BN>(see[i], tile(0))) issue_s(i, i, unit);
              mma_commit(bar.k_empty + (unit & 1));
            }
            for (int32_t k = 0; ok && k < n; ++k) {
              const uint32_t g = unit + k;
              bool has_k = false;
              ok = v_ready(g);
              for (int i = 0; ok && i < 2; ++i) {
                if (sees<BN>(see[i], tile(k))) {
                  ok = p_ready(i);
                  if (!ok) break;
                  issue_o(i, i, g, sum[i]);
                  sum[i] = true;
                  if (k == last[i]) mma_commit(bar.o_full + i);
                }
                if (i == 1) mma_commit(bar.v_empty + (g & 1));
                if (k + 1 < n && (i == 1 || sees<BN>(see[i], tile(k + 1)))) {
                  if (!has_k) {
                    ok = has_k = k_ready(g + 1);
                    if (!ok) break;
                    tc_fence_after();
                  }
                  if (sees<BN>(see[i], tile(k + 1))) issue_s(i, i, g + 1);
                  if (i == 1) mma_commit(bar.k_empty + ((g + 1) & 1));
                }
              }
            }
          } else {
            // (in one stream, S of the next tile goes ahead of O of this one; in two, S of the one after the next
            // follows O of this one, whose P it overwrites)
            constexpr int kAhead = 2;
            for (int32_t k = 0; ok && k < n + kAhead; ++k) {
              auto start_s = [&](int32_t j) {
                if (!k_ready(unit + j)) return false;
                tc_fence_after();
                issue_s(0, j & 1, unit + j);
                mma_commit(bar.k_empty + ((unit + j) & 1));
                return true;
              };
              if (kOne) {
                if (k < n) ok = start_s(k);
              } else if (k < 2 && k < n) {
                ok = start_s(k);
              }
              const int32_t j = kOne ? k - 1 : k - 2;  // the tile whose O is next
              if (!ok || j < 0 || j >= n) continue;
              const uint32_t g = unit + j;
              ok = v_ready(g) && p_ready(j & 1);
              if (!ok) break;
              tc_fence_after();
              issue_o(kOne ? 0 : j & 1, j & 1, g, kOne ? j > 0 : j > 1);
              mma_commit(bar.v_empty + (g & 1));
              if (kOne) mma_commit(&bar.o_step);
              if (kOne ? j == n - 1 : j >= n - 2) mma_commit(bar.o_full + (kOne ? 0 : j & 1));
              if (!kOne && j + 2 < n) ok = start_s(j + 2);
            }
          }
          unit += n;
        }
        if (!more(s)) break;
        next_segment<S>(a, s);
      }
      // nothing of this CTA is under way any more when it ends
      mma_commit(&bar.done);
      for (uint32_t i = 0; i < kWaitLimit && !mbar_try_wait(&bar.done, 0); ++i) {}
    }
  } else if (warp >= kSoftmaxWarps) {
    // ---- load ----
    set_registers<kLoadRegisters, false>();
    constexpr int TW = S::kWarpTokens;
    constexpr int kLanes = DP / E;             // of a row
    constexpr int kStep = 32 / kLanes;         // rows at a time
    constexpr int kItems = TW / kStep;         // of a lane, in a tile
    constexpr int kWords = E / 8;
    const int group = (warp - kSoftmaxWarps) / kLoadWarps, w = (warp - kSoftmaxWarps) % kLoadWarps;
    const int my_row = lane / kLanes, my_part = lane % kLanes;
    const bool in_row = my_part * E < D;
    Segment s = sh.first;
    Portion part = portion_of(s, run);
    int32_t u = part.u + group, end = part.end;
    uint32_t unit = group;
    bool any = true;
    // to a tile of this group, or past the run's end
    auto settle = [&] {
      while (u >= end) {
        if (!more(s)) {
          any = false;
          return;
        }
        const int32_t rest = u - end;
        next_segment<S>(a, s);
        part = portion_of(s, run);
        u = part.u + rest;
        end = part.end;
      }
    };
    constexpr uint32_t kDead = 0xFFFFFFFFu;
    uint32_t page = kDead, row = 0;  // of position `lane` of this warp's part of the tile looked up
    bool ahead = false;
    auto look_up = [&] {
      ahead = any;
      page = kDead;
      if (!any) return;
      const int32_t t = (u < s.first_units ? u : u + s.gap) * BN + w * TW + lane;
      if (lane < TW && t < s.see.hi && t < s.q.L && (t >= s.see.lo || t < s.see.sink)) {
        const int32_t col = div_q32(t, a.div_ps), slot = t - col * a.ps;
        const int64_t at = s.b * a.max_pages + col;
        const int64_t p = a.table64 ? __ldg(static_cast<const int64_t*>(a.block_tables) + at)
                                    : static_cast<int64_t>(__ldg(static_cast<const int32_t*>(a.block_tables) + at));
        if (p >= 0 && p < a.pool_pages) page = static_cast<uint32_t>(p);
        else flag(a.status, NVFP4_DEV_BAD_PAGE);
        row = a.layout == NVFP4_NHD ? slot * a.H + s.h : s.h * a.ps + slot;
      }
    };
    uint32_t kr[kItems][kWords], vr[kItems][kWords], ks[kItems], vs[kItems];
    uint32_t live = 0;
    auto load_codes = [&](const nvfp4_paged_cache& c, uint32_t (&r)[kItems][kWords]) {
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const uint32_t p = __shfl_sync(0xFFFFFFFFu, page, i * kStep + my_row), rw = __shfl_sync(0xFFFFFFFFu, row, i * kStep + my_row);
        const bool in = p != kDead && in_row;
        const uint8_t* src = c.data + static_cast<uint64_t>(p) * c.data_page_stride + static_cast<uint64_t>(rw) * (D / 2) + my_part * (E / 2);
        if constexpr (E == 32) {
          const uint4 x = in ? __ldg(reinterpret_cast<const uint4*>(src)) : uint4{};
          r[i][0] = x.x; r[i][1] = x.y; r[i][2] = x.z; r[i][3] = x.w;
        } else {
          const uint2 x = in ? __ldg(reinterpret_cast<const uint2*>(src)) : uint2{};
          r[i][0] = x.x; r[i][1] = x.y;
        }
      }
    };
    auto load_scales = [&](const nvfp4_paged_cache& c, uint32_t (&r)[kItems]) {
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const uint32_t p = __shfl_sync(0xFFFFFFFFu, page, i * kStep + my_row), rw = __shfl_sync(0xFFFFFFFFu, row, i * kStep + my_row);
        const bool in = p != kDead && in_row;
        const uint8_t* src = c.sf + static_cast<uint64_t>(p) * c.sf_page_stride + static_cast<uint64_t>(rw) * (D / 16) + my_part * (E / 16);
        if constexpr (E == 32) r[i] = in ? static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(src))) : 0u;
        else r[i] = in ? static_cast<uint32_t>(__ldg(src)) : 0u;
      }
    };
    // Decoded rows to a tile's atoms. Lanes of a row whose chunks would meet in the same banks store them in
    // another order (DP = 128: 8 lanes are two rows of two atoms; 256: one row of four).
    auto store = [&](uint32_t tile, const uint32_t (&r)[kItems][kWords], const uint32_t (&sc)[kItems]) {
      if (!in_row) return;
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const int rw = w * TW + i * kStep + my_row;
        if constexpr (E == 32) {
          const int atom = my_part >> 1;
          const uint32_t at = tile + atom * (BN * 128) + rw * 128;
          const int turn = DP == 128 ? 2 * (atom & 1) : (DP == 256 ? atom : 0);
          const uint32_t s2 = f16x2_from_e4m3x2(sc[i]);
          const uint32_t s_lo = low_twice(s2), s_hi = high_twice(s2);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int c = j ^ turn;  // the chunk of this lane's four that it stores now
            uint32_t word = r[i][j], scale = j < 2 ? s_lo : s_hi;
            if (DP == 128) {
              word = turn ? r[i][j ^ 2] : word;
              scale = turn ? (j < 2 ? s_hi : s_lo) : scale;
            } else if (DP == 256) {
              const uint32_t x0 = turn & 1 ? r[i][j ^ 1] : word, x1 = turn & 1 ? r[i][j ^ 3] : r[i][j ^ 2];
              word = turn & 2 ? x1 : x0;
              scale = turn & 2 ? (j < 2 ? s_hi : s_lo) : scale;
            }
            uint32_t x[4];
            f16x2x4_from_e2m1x8(word, x[0], x[1], x[2], x[3]);
            const uint32_t dst = at + (((4 * (my_part & 1) + c) ^ (rw & 7)) << 4);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(hmul2_rn(x[0], scale)), "r"(hmul2_rn(x[1], scale)),
                         "r"(hmul2_rn(x[2], scale)), "r"(hmul2_rn(x[3], scale)) : "memory");
          }
        } else {
          const uint32_t at = tile + (my_part >> 2) * (BN * 128) + rw * 128;
          const uint32_t scale = f16x2_from_e4m3x2(sc[i] * 0x0101u);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t x[4];
            f16x2x4_from_e2m1x8(r[i][j], x[0], x[1], x[2], x[3]);
            const uint32_t dst = at + (((2 * (my_part & 3) + j) ^ (rw & 7)) << 4);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(hmul2_rn(x[0], scale)), "r"(hmul2_rn(x[1], scale)),
                         "r"(hmul2_rn(x[2], scale)), "r"(hmul2_rn(x[3], scale)) : "memory");
          }
        }
      }
    };
    auto publish = [&](uint64_t* full) {
      fence_async_proxy();
      __syncwarp();
      if (lane == 0) mbar_arrive(full);
    };
    settle();
    look_up();
    if (ahead) {
      live = __ballot_sync(0xFFFFFFFFu, page != kDead);
      load_codes(a.kc, kr);
      load_scales(a.kc, ks);
      load_scales(a.vc, vs);
      load_codes(a.vc, vr);
    }
    bool have = ahead;
    if (have) {
      u += kLoadGroups;
      settle();
      look_up();
    }
    while (have) {
      if (a.pipe.stall) break;  // (a test: nothing comes, and every wait runs out)
      const uint32_t stage = unit & 1, parity = ((unit >> 1) & 1) ^ 1, meta = unit & (kMeta - 1);
      if (!wait_warp(bar.k_empty + stage, parity)) break;
      // what the softmax has to know of this tile; NaN scales of V are taken out
      uint32_t bad = 0;
#pragma unroll
      for (int i = 0; i < kItems; ++i) bad |= ((vs[i] & 0x7F7Fu) + 0x0101u) & 0x8080u;
      const bool any_nan = __any_sync(0xFFFFFFFFu, bad != 0);
      if (any_nan) {
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
          uint32_t blocks = 0;
          for (int k = 0; k < E / 16; ++k)
            if ((vs[i] >> (8 * k) & 0x7Fu) == 0x7Fu) {
              blocks |= 1u << (my_part * (E / 16) + k);
              vs[i] &= ~(0xFFu << (8 * k));
            }
          for (int o = 1; o < kLanes; o <<= 1) blocks |= __shfl_xor_sync(0xFFFFFFFFu, blocks, o);
          if (my_part == 0) sh.nan_blocks[meta][w * TW + i * kStep + my_row] = static_cast<uint16_t>(blocks);
        }
      }
      if (lane == 0) {
        sh.live[meta][w] = live;
        sh.nan[meta][w] = any_nan;
      }
      store(base + S::kK + stage * S::kTileBytes, kr, ks);
      publish(bar.k_full + stage);
      uint32_t vs_now[kItems];
#pragma unroll
      for (int i = 0; i < kItems; ++i) vs_now[i] = vs[i];
      if (ahead) {
        live = __ballot_sync(0xFFFFFFFFu, page != kDead);
        load_codes(a.kc, kr);
        load_scales(a.kc, ks);
        load_scales(a.vc, vs);
      }
      if (!wait_warp(bar.v_empty + stage, parity)) break;
      store(base + S::kV + stage * S::kTileBytes, vr, vs_now);
      publish(bar.v_full + stage);
      have = ahead;
      if (have) {
        load_codes(a.vc, vr);
        u += kLoadGroups;
        settle();
        look_up();
      }
      unit += kLoadGroups;
    }
  } else {
    // ---- softmax ----
    set_registers<kSoftmaxRegisters, true>();
    if (!kOne || warp < 4) {
    const int stream = warp >> 2, quarter = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(quarter) << 21;  // this warp's lanes of tensor memory
    const float gk = __ldg(a.k_scale), gv = __ldg(a.v_scale);
    const float cap = a.soft_cap;
    uint32_t unit = 0, q_count = 0, o_count = 0, merges = 0, steps = 0;
    uint32_t s_count[2] = {0, 0};
    Segment s = sh.first;
    for (;;) {
      const Portion part = portion_of(s, run);
      const int32_t n = part.end - part.u;
      const int64_t rows = static_cast<int64_t>(s.q.n) * a.G, r0 = static_cast<int64_t>(s.t) * S::kRows;
      const int local = (kTwo ? 128 * stream : 0) + quarter * 32 + lane;  // this thread's row of the segment
      const bool alive = r0 + local < rows;
      const int64_t token = quotient64(r0 + local, a.G);
      const int32_t head = static_cast<int32_t>(r0 + local - token * a.G);
      uint8_t* const out = a.out + ((s.q.q0 + token) * a.Hq + static_cast<int64_t>(s.h) * a.G + head) * D * 2;
      float* const lse = a.lse ? a.lse + (s.q.q0 + token) * a.Hq + static_cast<int64_t>(s.h) * a.G + head : nullptr;
      if (n == 0 && part.mine && stream == (kTwo ? stream : 0) && alive) {  // nothing that any row sees
        for (int i = 0; i < D / 8; ++i) reinterpret_cast<uint4*>(out)[i] = uint4{};
        if (lse) *lse = -INFINITY;
      }
      if (n > 0) {
        // -- the queries: in binary16, each row scaled by a power of two --
        {
          const int width = D / 8;
          int log_t = 0;
          while ((1 << log_t) < width) ++log_t;
          const int T = 1 << log_t, j = lane & (T - 1), step = 32 >> log_t;
          const int per_warp = kTurns ? 16 : 32;
          const int q_row = kTurns ? warp * 16 : (kTwo ? warp * 32 : quarter * 32);  // this warp's first
#pragma unroll 1
          for (int i0 = 0; i0 < per_warp; i0 += 4 * step) {
            uint4 raw[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int i = q_row + i0 + k * step + (lane >> log_t);
              raw[k] = uint4{};
              if (i0 + k * step < per_warp && r0 + i < rows && j < width) {
                const int64_t tk = quotient64(r0 + i, a.G);
                const int64_t hd = static_cast<int64_t>(s.h) * a.G + (r0 + i - tk * a.G);
                raw[k] = __ldg(reinterpret_cast<const uint4*>(a.q + (s.q.q0 + tk) * a.q_row_bytes + hd * D * 2) + j);
              }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (i0 + k * step >= per_warp) break;
              const int i = q_row + i0 + k * step + (lane >> log_t);
              const uint32_t x[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
              float v[8], top = 0.0f;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                v[2 * e] = a.bf16 ? __uint_as_float(x[e] << 16) : f32_from_f16_lo(x[e]);
                v[2 * e + 1] = a.bf16 ? f32_from_bf16_hi(x[e]) : f32_from_f16_hi(x[e]);
                top = max3(top, fabsf(v[2 * e]), fabsf(v[2 * e + 1]));
              }
              for (int o = T >> 1; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
              const int e2 = top > 0.0f && top <= FLT_MAX ? ilogbf(top) - 14 : 0;
              float f = ldexpf(a.sm_scale, e2) * gk;
              // 2^-e2 as two factors (it may be out of range by itself), with f's sign: f is not negative from
              // here on, and a maximum of scores is one of logits; f = 0 is a query of zeros
              float f1 = __int_as_float((127 - e2 / 2) << 23);
              const float f2 = __int_as_float((127 - (e2 - e2 / 2)) << 23);
              if (f < 0.0f) f1 = -f1;
              if (f == 0.0f) f1 = 0.0f;
              f = f == 0.0f ? 1.0f : fabsf(f);
              if (j < width) {
                uint32_t y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = f16x2_from_f32(v[2 * e] * f1 * f2, v[2 * e + 1] * f1 * f2);
                const int r = i & 127;
                const uint32_t dst = base + (i >> 7) * S::kQBytes + (j >> 3) * 16384 + r * 128 + (((j & 7) ^ (r & 7)) << 4);
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]) : "memory");
              }
              if (j == 0) sh.factor[i] = f;
            }
          }
          fence_async_proxy();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.q_full);
          if (!wait_warp(&bar.q_full, q_count++ & 1)) break;
        }
        // -- this row --
        const float f = sh.factor[local];
        const float unit2 = cap > 0.0f ? kLog2e : f * kLog2e;  // what turns x into base-2 logarithms
        const int32_t p = s.q.L - s.q.n + static_cast<int32_t>(token);
        const int32_t hi = !alive ? 0 : (a.causal ? min(max(p + 1, 0), s.q.L) : s.q.L);
        const int32_t lo = a.window_left >= 0 && p > a.window_left ? p - a.window_left : 0;
        const int32_t sink = a.window_left >= 0 ? a.sink : 0;
        const bool busy = __any_sync(0xFFFFFFFFu, alive);
        const int32_t all_hi = __reduce_min_sync(0xFFFFFFFFu, alive ? hi : INT32_MAX);
        const int32_t all_lo = __reduce_max_sync(0xFFFFFFFFu, alive ? lo : 0);
        Sight see{0, 0, 0};  // of this stream's rows
        if (kTwo && r0 + 128 * stream < rows)
          see = sight_of(a, s.q, r0 + 128 * stream, min(rows, r0 + 128 * stream + 128));
        float m = -INFINITY, l = 0.0f;
        uint32_t poison = 0;
        bool started = false, ok = true;
        for (int32_t k = kTurns ? stream : 0; k < n; k += kTurns ? 2 : 1) {
          const int32_t u = part.u + k;
          const int32_t t0 = (u < s.first_units ? u : u + s.gap) * BN;
          if (kTwo && !sees<BN>(see, t0)) continue;
          const int buf = kTwo ? stream : k & 1;
          ok = wait_warp(bar.s_full + buf, s_count[buf]++ & 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t meta = (unit + k) & (kMeta - 1);
          const uint32_t s_at = tmem + lanes + buf * BN;
          if (busy) {
            // which positions: a word for 32 of them
            uint32_t words[BN / 32];
            bool full = t0 + BN <= all_hi && (t0 >= all_lo || t0 + BN <= sink);
#pragma unroll
            for (int c = 0; c < BN / 32; ++c) {
              words[c] = S::kWarpTokens == 32 ? sh.live[meta][c] : sh.live[meta][2 * c] | sh.live[meta][2 * c + 1] << 16;
              full = full && words[c] == ~0u;
            }
            if (!full) {
#pragma unroll
              for (int c = 0; c < BN / 32; ++c) {
                const int32_t t = t0 + 32 * c;
                words[c] &= low_bits(hi - t) & (~low_bits(lo - t) | low_bits(sink - t));
              }
            }
            auto weigh = [&](auto masked_, auto capped_) {
              constexpr bool kMasked = decltype(masked_)::value, kCapped = decltype(capped_)::value;
              constexpr int NC = BN / 32;
              float v[2][32];
              tmem_load(v[0], s_at);
              tmem_wait(v[0]);
              float top = -INFINITY;
#pragma unroll
              for (int c = 0; c < NC; ++c) {
                float (&x)[32] = v[c & 1];
                tmem_load(v[(c + 1) & 1], s_at + (c + 1 < NC ? 32 * (c + 1) : 0));  // (the first again, for the weights)
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                  const float x0 = kMasked && !(words[c] >> i & 1u) ? -INFINITY : x[i];
                  const float x1 = kMasked && !(words[c] >> (i + 1) & 1u) ? -INFINITY : x[i + 1];
                  top = max3(top, x0, x1);
                }
                tmem_wait(v[(c + 1) & 1]);
              }
              top = (kCapped ? soft_capped(top * f, cap) : top) * unit2;
              const bool rises = top > m + kSlack;  // (by row: a result does not depend on other rows)
              if (__any_sync(0xFFFFFFFFu, rises)) {
                const float g = rises ? ex2(m - top) : 1.0f;
                m = rises ? top : m;
                l *= g;
                if (started) {
                  if (kOne && !wait_warp(&bar.o_step, (steps - 1) & 1)) return false;
                  tc_fence_after();
                  const uint32_t o_at = tmem + lanes + S::kO + (kOne ? 0 : stream * DP);
                  for (int d = 0; d < D; d += 16) {
                    float o[16];
                    tmem_load(o, o_at + d);
                    tmem_wait(o);
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] *= g;
                    tmem_store(o_at + d, o);
                  }
                }
              }
              const float off = m == -INFINITY ? 0.0f : kWeightBias - m;
              float sums[4] = {0, 0, 0, 0};
#pragma unroll
              for (int c = 0; c < NC; ++c) {
                float (&x)[32] = v[(NC + c) & 1];
                if (c + 1 < NC) tmem_load(v[(NC + c + 1) & 1], s_at + 32 * (c + 1));
                uint32_t y[16];
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                  float p01[2];
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    float z = kCapped ? soft_capped(x[i + e] * f, cap) : x[i + e];
                    if (kMasked && !(words[c] >> (i + e) & 1u)) z = -INFINITY;
                    p01[e] = ex2(__fmaf_rn(z, unit2, off));
                    sums[(i + e) & 3] += p01[e];
                  }
                  y[i / 2] = f16x2_from_f32(p01[0], p01[1]);
                }
                if (kCapped) __syncwarp();
                tmem_store(s_at + 16 * c, y);
                if (c + 1 < NC) tmem_wait(v[(NC + c + 1) & 1]);
              }
              l += (sums[0] + sums[1]) + (sums[2] + sums[3]);
              return true;
            };
            using T = std::true_type;
            using F = std::false_type;
            if (cap > 0.0f) ok = weigh(T{}, T{});
            else ok = full ? weigh(F{}, F{}) : weigh(T{}, F{});
            if (!ok) break;
            // blocks of V that are NaN, where this row sees them
            for (int w = 0; w < kLoadWarps; ++w) {
              if (!sh.nan[meta][w]) continue;
              for (int i = 0; i < S::kWarpTokens; ++i) {
                const int c = w * S::kWarpTokens + i, t = t0 + c;
                if (t < hi && (t >= lo || t < sink)) poison |= sh.nan_blocks[meta][c];
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
          for (int d = 0; d < D; d += 16) {
            float o[16] = {};
            __syncwarp();
            if (started) {
              tmem_load(o, o_at + d);
              tmem_wait(o);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= w0;
            if (two) {
              float x[16];
              tmem_load(x, o_at + DP + d);
              tmem_wait(x);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] += w1 * x[i];
            }
            if (poison >> (d / 16) & 1u) {
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = NAN;
            }
            if (alive && whole) {
              uint32_t y[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
                y[i] = a.bf16 ? bf16x2_from_f32(o[2 * i], o[2 * i + 1]) : f16x2_from_f32(o[2 * i], o[2 * i + 1]);
              uint4* dst = reinterpret_cast<uint4*>(out + d * 2);
              dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
              dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
            } else if (alive) {
              float4* dst = reinterpret_cast<float4*>(part_o + static_cast<int64_t>(local) * DP + d);
#pragma unroll
              for (int i = 0; i < 4; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
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
        unit += n;
      }
      if (!more(s)) break;
      next_segment<S>(a, s);
    }
    // the run's last segment, if others continue it
    if (tid == 0 && s.units > kWholeUnits && s.start >= 0 && s.start < run && s.start + s.units > run) {
      PrefillCut* const cuts = reinterpret_cast<PrefillCut*>(static_cast<uint8_t*>(a.workspace) + NVFP4_COUNTER_BYTES);
      cuts[blockIdx.x] = {s.b, s.t, s.h, static_cast<int32_t>(cut.run_of(c0 + s.start + s.units - 1))};
    }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kProductWarp) {
    tc_fence_after();
    tmem_free(tmem);
  }
}

// The parts of the segment that run blockIdx.x begins and others continue, added in the runs' order; a warp takes
// four of its rows, 32 rows to a CTA.
constexpr int kJoinRows = 32;
template <int DP, int MT>
__global__ void __launch_bounds__(256) join_kernel(const PrefillArgs a) {
  using S = Shape<DP, MT>;
  const PrefillCut c = reinterpret_cast<const PrefillCut*>(static_cast<const uint8_t*>(a.workspace) + NVFP4_COUNTER_BYTES)[blockIdx.x];
  if (c.last < 0) return;
  const Request q = request_of(a, c.b);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = a.D;
  const int64_t rows = static_cast<int64_t>(q.n) * a.G, r0 = static_cast<int64_t>(c.t) * S::kRows;
  const int64_t first = blockIdx.x;
  const float gv = __ldg(a.v_scale);
  for (int k = 0; k < 4; ++k) {
    const int local = blockIdx.y * kJoinRows + warp * 4 + k;
    if (r0 + local >= rows) return;
    auto part = [&](int64_t i) { return part_of(a, i, i == first ? 1 : 0, S::kRows, DP); };
    float top = -INFINITY;
    for (int64_t i = first + lane; i <= c.last; i += 32) top = fmaxf(top, part(i)[S::kRows * DP + local]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
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
    const int64_t token = quotient64(r0 + local, a.G);
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
  // 16-byte loads of codes and 2-byte loads of scales
  auto even = [](const nvfp4_paged_cache& c) { return reinterpret_cast<uintptr_t>(c.sf) % 2 == 0 && c.sf_page_stride % 2 == 0; };
  return a.D % 32 == 0 && even(a.kc) && even(a.vc) ? launch_t<DP, MT, 32>(a, s) : launch_t<DP, MT, 16>(a, s);
}

}  // namespace

int64_t prefill_workspace_bytes(int32_t D) {
  const int64_t dp = D <= 64 ? 64 : (D <= 128 ? 128 : 256), rows = D <= 128 ? 256 : 128, n = sm_count();
  return NVFP4_COUNTER_BYTES + (n * sizeof(PrefillCut) + 127) / 128 * 128 + 2 * n * rows * (dp + 2) * 4;
}

nvfp4_status launch_prefill(PrefillArgs a, cudaStream_t stream) {
  a.pool_pages = a.kc.num_pages < a.vc.num_pages ? a.kc.num_pages : a.vc.num_pages;
  a.pipe = pipe_test_from_env();
  // 256 rows of a segment share the decoded tiles; requests of fewer rows than 128 have no use for them
  const bool two = a.nnz * a.G > static_cast<int64_t>(a.B) * 128;
  if (a.D > 128) return launch_e<256, 1>(a, stream);
  if (a.D > 64) return two ? launch_e<128, 2>(a, stream) : launch_e<128, 1>(a, stream);
  return two ? launch_e<64, 2>(a, stream) : launch_e<64, 1>(a, stream);
}

}  // namespace nvfp4
