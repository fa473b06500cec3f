// pages.cu -- which pages of a paged NVFP4 key cache a query should read.
//
// Bounds of a page p and KV head h, over its live slots t:
//   lo[d] = min_t (e2m1 * S)[t, d],  hi[d] = max_t (e2m1 * S)[t, d]     (binary16, exact)
// Score of a page for the query heads g of the KV head's group, an upper bound of q . k there
// (up to the positive factor gs_k):
//   s = max_g sum_d (max(q_d, 0) hi[d] + min(q_d, 0) lo[d])
// The products are exact in binary32 (11 by 11 bits, one of the two is zero); the sum has a
// fixed order, so that the selection is reproducible: in each group of eight elements two
// chains, of the even and of the odd elements, then their sum; the D/8 group sums, filled up
// with zeros to a power of two, add by halves (t[i] += t[i + n/2]).
#include "attention.h"
#include "scan.cuh"

namespace nvfp4 {
namespace {

__device__ __forceinline__ int64_t table_entry(const void* tables, int32_t is64, int64_t at) {
  return is64 ? __ldg(static_cast<const int64_t*>(tables) + at)
              : __ldg(static_cast<const int32_t*>(tables) + at);
}

// ---- bounds -----------------------------------------------------------------------------
//
// Reading the keys is the floor: 9/16 byte an element, and 4 bytes written for page_size of them. A
// thread has one column, a 16-element block of a head, and slots of one page; kBatch slots are
// loaded before the first is decoded. Pages of more than kMaxSlots slots give a column to several
// threads.

constexpr int kBoundsThreads = 256;
constexpr int kBatch = 8;
constexpr int kMaxSlots = 8;  // that a thread has of a column, where there are threads for it
constexpr int kMaxBoundsStages = 4;
// Shared memory of the ring: three CTAs to an SM, or what two stages of one larger page need.
constexpr int64_t kBoundsRing = 72 * 1024, kBoundsMostRing = 160 * 1024;

// (NaN if either is)
__device__ __forceinline__ uint32_t hmin2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A CTA takes `pages` items (pages of requests) at a time, of `tile` columns in `slices` threads
// each; their product is at most kBoundsThreads. Thread: (item, slice, column), column fastest.
struct BoundsShape {
  int col, slice, item;
};
__device__ __forceinline__ BoundsShape bounds_shape(const BoundsArgs& a) {
  const int tid = threadIdx.x;
  return {tid % a.tile, tid / a.tile % a.slices, tid / (a.tile * a.slices)};
}

// Item `item` of all pages to be done: its physical page (-1: none, or outside the pool) and live slots.
struct BoundsItem {
  int64_t page;
  int32_t n;
};

__device__ __forceinline__ int64_t bounds_len(const BoundsArgs& a, int32_t b) {
  return min(static_cast<int64_t>(__ldg(a.seq_lens + b)), a.max_pages * a.ps);
}
__device__ __forceinline__ int32_t bounds_first(const BoundsArgs& a, int32_t b) {
  return a.first_positions ? div_q32(max(__ldg(a.first_positions + b), 0), a.div_ps) : 0;
}
__device__ __forceinline__ int32_t scan_items(const BoundsArgs& a, int32_t* cum) {
  block_inclusive_scan(cum, a.B, [&](int32_t b) {
    const int64_t len = bounds_len(a, b);
    if (blockIdx.x == 0 && __ldg(a.seq_lens + b) > a.max_pages * a.ps) flag(a.status, NVFP4_DEV_LEN_CLAMPED);
    const int32_t pages = len > 0 ? div_q32(static_cast<int32_t>(len - 1), a.div_ps) + 1 : 0;
    return max(pages - bounds_first(a, b), 0);
  });
  return cum[a.B - 1];
}
__device__ __forceinline__ BoundsItem find_item(const BoundsArgs& a, const int32_t* cum, int64_t item, int32_t total) {
  if (item >= total) return {-1, 0};
  const int32_t b = scan_find(cum, a.B, static_cast<int32_t>(item));
  const int32_t col = static_cast<int32_t>(item) - (b > 0 ? cum[b - 1] : 0) + bounds_first(a, b);
  int64_t page = table_entry(a.block_tables, a.table64, b * a.max_pages + col);
  if (page < 0 || page >= a.kc.num_pages) {
    flag(a.status, NVFP4_DEV_BAD_PAGE);
    page = -1;
  }
  return {page, static_cast<int32_t>(min(static_cast<int64_t>(a.ps), bounds_len(a, b) - static_cast<int64_t>(col) * a.ps))};
}

// Bounds of a thread's slots of one column: block of slot t at `at + t * step` of codes and scales
// (global or shared memory).
struct ColumnBounds {
  uint32_t lo[8], hi[8];
};
__device__ __forceinline__ void clear(ColumnBounds& v) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    v.lo[e] = 0x7C007C00u;  // +inf, -inf: what a slice without slots leaves
    v.hi[e] = 0xFC00FC00u;
  }
}
__device__ __forceinline__ void add_slots(ColumnBounds& r, const uint8_t* codes, const uint8_t* scales, int32_t at,
                                          int32_t step, int32_t first, int32_t stride, int32_t n) {
  for (int32_t t0 = first; t0 < n; t0 += kBatch * stride) {
    uint2 c[kBatch];
    uint32_t s[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int32_t t = min(t0 + k * stride, n - 1);  // (past the end: the last slot again)
      const int32_t blk = at + t * step;
      c[k] = reinterpret_cast<const uint2*>(codes)[blk];
      s[k] = scales[blk];
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const uint32_t S2 = f16x2_from_e4m3x2(s[k] * 0x0101u);
      uint32_t v[8];
      f16x2x4_from_e2m1x8(c[k].x, v[0], v[1], v[2], v[3]);
      f16x2x4_from_e2m1x8(c[k].y, v[4], v[5], v[6], v[7]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = hmul2_rn(v[e], S2);
        r.lo[e] = hmin2(r.lo[e], v[e]);
        r.hi[e] = hmax2(r.hi[e], v[e]);
      }
    }
  }
}

// Join the slices of a column through s_part [16][kBoundsThreads] into slice 0; the whole CTA calls it.
__device__ __forceinline__ void join_slices(const BoundsArgs& a, ColumnBounds& r, uint32_t* s_part, int slice, bool mine) {
  const int tid = threadIdx.x;
  __syncthreads();  // what the last join left has been read
  if (mine && slice > 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s_part[e * kBoundsThreads + tid] = r.lo[e];
      s_part[(8 + e) * kBoundsThreads + tid] = r.hi[e];
    }
  }
  __syncthreads();
  if (mine && slice == 0) {
    for (int q = 1; q < a.slices; ++q) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        r.lo[e] = hmin2(r.lo[e], s_part[e * kBoundsThreads + tid + q * a.tile]);
        r.hi[e] = hmax2(r.hi[e], s_part[(8 + e) * kBoundsThreads + tid + q * a.tile]);
      }
    }
  }
}

__device__ __forceinline__ void write_column(const BoundsArgs& a, const ColumnBounds& r, int64_t page, int32_t h, int32_t j) {
  uint4* lo = reinterpret_cast<uint4*>(a.bounds + (page * a.H + h) * 2 * a.D + 16 * j);
  uint4* hi = reinterpret_cast<uint4*>(a.bounds + ((page * a.H + h) * 2 + 1) * a.D + 16 * j);
  lo[0] = make_uint4(r.lo[0], r.lo[1], r.lo[2], r.lo[3]);
  lo[1] = make_uint4(r.lo[4], r.lo[5], r.lo[6], r.lo[7]);
  hi[0] = make_uint4(r.hi[0], r.hi[1], r.hi[2], r.hi[3]);
  hi[1] = make_uint4(r.hi[4], r.hi[5], r.hi[6], r.hi[7]);
}

// Pages that cannot be copied in bulk (alignment, size): straight from global memory. The threads of
// a column join in shared memory.
__global__ void __launch_bounds__(kBoundsThreads) page_key_bounds_kernel(const BoundsArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  int32_t* cum = reinterpret_cast<int32_t*>(smem);
  __shared__ uint32_t s_part[16 * kBoundsThreads];
  const int32_t total = scan_items(a, cum), nb = a.D / 16, columns = a.H * nb;
  const BoundsShape me = bounds_shape(a);
  for (int64_t item0 = static_cast<int64_t>(blockIdx.x) * a.pages; item0 < total;
       item0 += static_cast<int64_t>(gridDim.x) * a.pages) {
    const BoundsItem it = me.item < a.pages ? find_item(a, cum, item0 + me.item, total) : BoundsItem{-1, 0};
    for (int32_t c0 = 0; c0 < columns; c0 += a.tile) {
      const int32_t w = c0 + me.col, h = w / nb, j = w - h * nb;
      const bool mine = it.page >= 0 && w < columns;
      ColumnBounds r;
      clear(r);
      if (mine)
        add_slots(r, a.kc.data + it.page * a.kc.data_page_stride, a.kc.sf + it.page * a.kc.sf_page_stride,
                  a.layout == NVFP4_NHD ? w : h * a.ps * nb + j, a.layout == NVFP4_NHD ? columns : nb, me.slice,
                  a.slices, it.n);
      if (a.slices > 1) join_slices(a, r, s_part, me.slice, mine);
      if (mine && me.slice == 0) write_column(a, r, it.page, h, j);
    }
  }
}

// The same from a ring of stages, each `pages` items' codes and scales in bulk copies: a page is
// contiguous in either layout, and copies in flight are not bound by registers or by the number of
// loads that an SM tracks. One warp keeps the ring filled; the others take a job at a time, 32/S
// columns (of one page or, where it has fewer, of several) with S lanes to a column (S = 1, 2 or 4, about eight slots each), and are bound
// to one another by the stages' barriers alone. The S lanes join by halves: one keeps the lower
// bounds and gives the upper ones away, so that each ends with 32/S bytes of the result.
//
// Per 32 blocks of 16 elements: two loads, nine conversions, eight products, 16 minima and maxima.
// They bound it: 200 K tokens of 8 heads of 128 elements in pages of 32 take 41 us (3.4 TB/s, the
// ALU pipe two thirds busy), in pages of 16 41 us (4.0 TB/s); direct loads took them at 2.2 TB/s.
// With a CTA-wide barrier at a stage's start and end and the join in shared memory it was 50 us,
// with two larger CTAs to an SM and six stages 45 us.
constexpr int kRingWarps = 8;
constexpr int kRingPages = 32;  // most items of a stage: one to a lane

template <int S>
__device__ __forceinline__ void add_ring_slots(ColumnBounds& r, const uint2* c, const uint8_t* s, int32_t inc, int32_t n) {
  auto add = [&](const uint2 (&w)[kBatch], const uint32_t (&f)[kBatch]) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const uint32_t S2 = f16x2_from_e4m3x2(f[k] * 0x0101u);
      uint32_t v[8];
      f16x2x4_from_e2m1x8(w[k].x, v[0], v[1], v[2], v[3]);
      f16x2x4_from_e2m1x8(w[k].y, v[4], v[5], v[6], v[7]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = hmul2_rn(v[e], S2);
        r.lo[e] = hmin2(r.lo[e], v[e]);
        r.hi[e] = hmax2(r.hi[e], v[e]);
      }
    }
  };
  // slots 0, S, 2 S, .. below n, `inc` blocks apart
#pragma unroll 1
  while (n > 0) {
    uint2 w[kBatch];
    uint32_t f[kBatch];
    if (n > (kBatch - 1) * S) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        w[k] = c[k * inc];
        f[k] = s[k * inc];
      }
    } else {
      const int32_t last = (n - 1) / S;  // (past the end: the last slot again)
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        w[k] = c[min(k, last) * inc];
        f[k] = s[min(k, last) * inc];
      }
    }
    add(w, f);
    n -= kBatch * S;
    c += kBatch * inc;
    s += kBatch * inc;
  }
}

template <int S>
__global__ void __launch_bounds__((kRingWarps + 1) * 32, 3) page_key_bounds_ring_kernel(const BoundsArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(8) uint64_t s_full[kMaxBoundsStages], s_empty[kMaxBoundsStages];
  __shared__ BoundsItem s_item[kMaxBoundsStages][kRingPages];
  int32_t* cum = reinterpret_cast<int32_t*>(smem + a.stages * a.stage_bytes);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(s_full + s, a.pages);
      mbar_init(s_empty + s, kRingWarps);
    }
    fence_mbar_init();
  }
  const int32_t total = scan_items(a, cum), nb = a.D / 16, columns = a.H * nb;  // ends with a barrier
  const int64_t step = static_cast<int64_t>(gridDim.x) * a.pages, from = static_cast<int64_t>(blockIdx.x) * a.pages;
  int s = 0;
  uint32_t phase = 0;
  if (warp == kRingWarps) {  // the copies: lane p < pages has item p of a stage
    const bool stall = a.pipe.stall != 0;  // test control: withhold the first stage
    int32_t filled = 0;                    // stages filled, up to a.stages
    for (int64_t item0 = from; item0 < total; item0 += step) {
      const BoundsItem it = lane < a.pages ? find_item(a, cum, item0 + lane, total) : BoundsItem{-1, 0};
      if (filled == a.stages) {
        const bool ok = mbar_wait(s_empty + s, phase ^ 1u, a.pipe.wait_limit);
        if (__any_sync(0xFFFFFFFFu, !ok)) {
          if (lane == 0) flag(a.status, NVFP4_DEV_TIMEOUT);
          break;
        }
      } else {
        ++filled;
      }
      if (lane < a.pages && !(stall && item0 == from)) {
        s_item[s][lane] = it;
        if (it.page >= 0) {
          uint8_t* dst = smem + s * a.stage_bytes + lane * (a.code_bytes + a.scale_bytes);
          mbar_arrive_expect_tx(s_full + s, a.code_bytes + a.scale_bytes);
          bulk_g2s(dst, a.kc.data + it.page * a.kc.data_page_stride, a.code_bytes, s_full + s);
          bulk_g2s(dst + a.code_bytes, a.kc.sf + it.page * a.kc.sf_page_stride, a.scale_bytes, s_full + s);
        } else {
          mbar_arrive(s_full + s);
        }
      }
      if (++s == a.stages) {
        s = 0;
        phase ^= 1u;
      }
    }
    // No copy may still be landing in this CTA's shared memory when it exits: the last fill of each
    // stage. (Stages below s were filled in this round of the ring, those from s on in the last one.)
    for (int q = 0; q < a.stages; ++q) {
      if (q >= filled || (stall && q == 0)) continue;
      mbar_wait(s_full + q, q < s ? phase : phase ^ 1u, a.pipe.wait_limit);
    }
    return;
  }
  constexpr int kColumns = 32 / S;
  const int slice = lane / kColumns, in_group = lane % kColumns;
  const int32_t all = a.pages * columns;  // a stage's columns
  const bool nhd = a.layout == NVFP4_NHD;
  const int32_t slot_step = nhd ? columns : nb;
  for (int64_t item0 = from; item0 < total; item0 += step) {
    const bool ok = mbar_wait(s_full + s, phase, a.pipe.wait_limit);
    if (__any_sync(0xFFFFFFFFu, !ok)) {
      if (lane == 0) flag(a.status, NVFP4_DEV_TIMEOUT);
      return;
    }
    for (int32_t c0 = warp * kColumns; c0 < all; c0 += kRingWarps * kColumns) {
      const int32_t p = min(div_q32(c0 + in_group, a.div_columns), a.pages - 1);
      const int32_t w = c0 + in_group - p * columns;
      const BoundsItem it = s_item[s][p];
      const bool mine = it.page >= 0 && w < columns;
      if (__any_sync(0xFFFFFFFFu, mine)) {
        const int32_t h = div_q32(w, a.div_nb), j = w - h * nb;
        ColumnBounds r;
        clear(r);
        if (mine) {
          const uint8_t* codes = smem + s * a.stage_bytes + p * (a.code_bytes + a.scale_bytes);
          const int32_t at = (nhd ? w : h * a.ps * nb + j) + slice * slot_step;
          add_ring_slots<S>(r, reinterpret_cast<const uint2*>(codes) + at, codes + a.code_bytes + at, S * slot_step,
                            it.n - slice);
        }
        uint16_t* out = a.bounds + (it.page * a.H + h) * 2 * a.D + 16 * j;
        if (S == 1) {
          if (mine) write_column(a, r, it.page, h, j);
        } else {
          const bool upper = lane & 16;
          uint32_t x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, upper ? r.lo[e] : r.hi[e], 16);
            x[e] = upper ? hmax2(r.hi[e], got) : hmin2(r.lo[e], got);
          }
          if (upper) out += a.D;
          if (S == 2) {
            if (mine) {
              reinterpret_cast<uint4*>(out)[0] = make_uint4(x[0], x[1], x[2], x[3]);
              reinterpret_cast<uint4*>(out)[1] = make_uint4(x[4], x[5], x[6], x[7]);
            }
          } else {
            const bool second = lane & 8;
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, second ? x[e] : x[4 + e], 8);
              const uint32_t keep = second ? x[4 + e] : x[e];
              y[e] = upper ? hmax2(keep, got) : hmin2(keep, got);
            }
            if (mine) reinterpret_cast<uint4*>(out)[second] = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(s_empty + s);  // the stage has been read
    if (++s == a.stages) {
      s = 0;
      phase ^= 1u;
    }
  }
}

// ---- scores -----------------------------------------------------------------------------
//
// A unit is kUnitPages pages of one (request, KV head). All units are cut into equal runs, one for each
// warp; a warp holds its query heads in registers (as positive and negative parts) and passes
// over the pages' bounds once, T lanes to a page (T = D/8 rounded up), each lane eight elements.
// A lane's bounds come through its own ring of stages in shared memory (cp.async; no other lane
// reads them, so a wait is all the synchronization there is). The lanes' parts of a unit's sums are
// joined together at its end: 17 shuffles for eight pages and four heads of 128 elements, 32 if each
// row of pages is joined by itself. Reading the bounds, 4 D bytes a page and head, is the floor.
// 158 registers (G <= 4) admit twelve warps to an SM, 232 (G <= 8) eight; they wait for their copies most,
// and 45 and 41 % of the issue slots are used, the 2 G D multiply-adds (packed two by two) first among the
// instructions. With the selection, at D = 128, in calls back to back: 512 lists of 346 pages on average, G = 4, 31 us (2.95 TB/s of bounds); 512
// lists of 2270 pages 138 us (4.3); 32 lists of 7200 pages, G = 8, 55 us (2.1). Two lanes to a page
// would need no shuffles but takes 16 % longer: the rows then lie 4 D bytes apart in shared memory.

constexpr int kScoreWarps = 4;
constexpr int kScoreBytes = 8192;  // a warp's ring
constexpr int kUnitPages = 8;

// Unsigned keys in the order of the scores.
__device__ __forceinline__ uint32_t key_of(float s) {
  const uint32_t u = __float_as_uint(s + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
constexpr uint32_t kForced = 0xFFFFFFFFu;  // a page that is selected before all others

__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}
__device__ __forceinline__ uint64_t widen2(uint32_t h) {
  return pack2(f32_from_f16_lo(h), f32_from_f16_hi(h));
}

// The selection is launched while the scores are still being computed, and waits for them.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void wait_for_scores() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ int32_t pages_of(const SelectArgs& a, int32_t b) {
  const int64_t len = min(static_cast<int64_t>(max(__ldg(a.seq_lens + b), 0)), a.max_pages * a.ps);
  return static_cast<int32_t>((len + a.ps - 1) / a.ps);
}

template <int GC, int T, int R>
__global__ void __launch_bounds__(kScoreWarps * 32, GC == 4 ? 3 : 2) page_scores_kernel(const SelectArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kPages = 32 / T, kStep = kPages * R;  // pages of a row of lanes, and of a step
  constexpr int kStage = 1024 * R, kStages = kScoreBytes / kStage;
  constexpr int kRows = kUnitPages / kPages, kIts = kUnitPages / kStep;  // rows and steps of a unit
  constexpr int kAhead = (kIts + kStages - 2) / kIts;  // units that the copies are ahead at a unit's end
  static_assert(kIts >= 1 && (kAhead + 1) * kUnitPages <= 64 && kRows * GC == T * (GC / 4), "");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % T, group = lane / T;
  int32_t* cum = reinterpret_cast<int32_t*>(smem + kScoreWarps * kScoreBytes);
  block_inclusive_scan(cum, a.B, [&](int32_t b) {
    if (blockIdx.x == 0 && __ldg(a.seq_lens + b) > a.max_pages * a.ps) flag(a.status, NVFP4_DEV_LEN_CLAMPED);
    return (pages_of(a, b) + kUnitPages - 1) / kUnitPages;
  });
  const int64_t total = static_cast<int64_t>(cum[a.B - 1]) * a.H;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kScoreWarps;
  const int64_t me = static_cast<int64_t>(blockIdx.x) * kScoreWarps + warp;
  launch_dependents();
  int64_t u = total * me / warps;
  const int64_t u_end = total * (me + 1) / warps;
  if (u >= u_end) return;
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem + warp * kScoreBytes)) + lane * 16;

  // the list of unit u: units run over requests, then heads, then pages
  int32_t b = scan_find(cum, a.B, static_cast<int32_t>(u / a.H));
  int32_t units = cum[b] - (b > 0 ? cum[b - 1] : 0);
  int64_t in_request = u - static_cast<int64_t>(b > 0 ? cum[b - 1] : 0) * a.H;
  int32_t h = static_cast<int32_t>(in_request / units), first = static_cast<int32_t>(in_request % units);

  const bool active = 8 * sub < a.D;
  const uint64_t page_bytes = static_cast<uint64_t>(a.H) * 4 * a.D;
  for (;;) {
    const int32_t n = pages_of(a, b);
    const int32_t last = static_cast<int32_t>(min(static_cast<int64_t>(units), first + (u_end - u)));
    uint32_t* keys = a.scores + (static_cast<int64_t>(b) * a.H + h) * a.pitch;
    for (int32_t g0 = 0; g0 < a.G; g0 += GC) {
      uint64_t qp[GC][4], qn[GC][4];
#pragma unroll
      for (int g = 0; g < GC; ++g) {
        uint4 w{};
        if (active && g0 + g < a.G)
          w = __ldg(reinterpret_cast<const uint4*>(
              a.q + b * a.q_row_bytes + ((static_cast<int64_t>(h) * a.G + g0 + g) * a.D + 8 * sub) * 2));
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = a.bf16 ? __uint_as_float(ww[i] << 16) : f32_from_f16_lo(ww[i]);
          const float y = a.bf16 ? f32_from_bf16_hi(ww[i]) : f32_from_f16_hi(ww[i]);
          qp[g][i] = pack2(fmaxf(x, 0.0f), fmaxf(y, 0.0f));
          qn[g][i] = pack2(fminf(x, 0.0f), fminf(y, 0.0f));
        }
      }
      // A unit's entries of the block table are read a unit before its first copy; `bad` has its pages
      // outside the pool (copied as zeros), eight bits to a unit, the newest unit lowest.
      const uint8_t* base = reinterpret_cast<const uint8_t*>(a.bounds + static_cast<int64_t>(h) * 2 * a.D + (active ? 8 * sub : 0));
      const int32_t units_here = last - first;
      int32_t to_issue = 0, entry = -1;
      int64_t next = -1;
      uint64_t bad = 0;
      auto read_entry = [&](int32_t unit) {
        next = -1;
        if (unit < units_here && lane < kUnitPages && (first + unit) * kUnitPages + lane < n)
          next = table_entry(a.block_tables, a.table64, b * a.max_pages + (first + unit) * kUnitPages + lane);
      };
      auto issue = [&](int step) {  // step `step` of unit `to_issue`
        if (step == 0) {
          const bool live = to_issue < units_here && lane < kUnitPages && (first + to_issue) * kUnitPages + lane < n;
          const bool ok = next >= 0 && next < a.num_pages;
          entry = live && ok ? static_cast<int32_t>(next) : -1;
          const uint32_t out = __ballot_sync(0xFFFFFFFFu, live && !ok);
          if (out && lane == 0) flag(a.status, NVFP4_DEV_BAD_PAGE);
          bad = bad << kUnitPages | out;
          read_entry(to_issue + 1);
        }
        if (to_issue < units_here) {
          const uint32_t dst = ring + (to_issue * kIts + step) % kStages * kStage;
#pragma unroll
          for (int q = 0; q < R; ++q) {
            const int32_t page = __shfl_sync(0xFFFFFFFFu, entry, step * kStep + q * kPages + group);
            const uint8_t* src = base + static_cast<uint64_t>(max(page, 0)) * page_bytes;
            const int bytes = page >= 0 && active ? 16 : 0;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + q * 1024), "l"(src), "r"(bytes) : "memory");
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + q * 1024 + 512), "l"(src + 2 * a.D), "r"(bytes) : "memory");
          }
        }
        if (step == kIts - 1) ++to_issue;
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      read_entry(0);
#pragma unroll
      for (int s = 0; s < kStages - 1; ++s) issue(s % kIts);
#pragma unroll 1
      for (int32_t unit = 0; unit < units_here; ++unit) {
        float v[kRows * GC];  // the lane's part of each sum of the unit
#pragma unroll
        for (int step = 0; step < kIts; ++step) {
          asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
          const uint8_t* st = smem + warp * kScoreBytes + (unit * kIts + step) % kStages * kStage + lane * 16;
          uint4 lw[R], hw[R];
#pragma unroll
          for (int q = 0; q < R; ++q) {
            lw[q] = *reinterpret_cast<const uint4*>(st + q * 1024);
            hw[q] = *reinterpret_cast<const uint4*>(st + q * 1024 + 512);
          }
          issue((step + kStages - 1) % kIts);
#pragma unroll
          for (int q = 0; q < R; ++q) {
            const uint64_t lo[4] = {widen2(lw[q].x), widen2(lw[q].y), widen2(lw[q].z), widen2(lw[q].w)};
            const uint64_t hi[4] = {widen2(hw[q].x), widen2(hw[q].y), widen2(hw[q].z), widen2(hw[q].w)};
#pragma unroll
            for (int g = 0; g < GC; ++g) {
              uint64_t acc = 0;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                fma2(acc, qp[g][i], hi[i]);
                fma2(acc, qn[g][i], lo[i]);
              }
              float x, y;
              asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(acc));
              v[(step * R + q) * GC + g] = __fadd_rn(x, y);
            }
          }
        }
        // Sums over the T lanes by halves: a lane gives one half of its sums to its partner and keeps
        // the other, so that at the end lane `sub` has row sub / 4 and the heads sub % 4 (of GC = 4;
        // two heads of GC = 8). Then the maximum over the heads.
#pragma unroll
        for (int s = 1; 1 << s <= T; ++s) {
          const int o = T >> s;
          const bool up = lane & o;
#pragma unroll
          for (int k = 0; k < kRows * GC / 2; ++k) {
            if (k < kRows * GC >> s) {
              const float low = v[k], high = v[k + (kRows * GC >> s)];
              v[k] = __fadd_rn(up ? high : low, __shfl_xor_sync(0xFFFFFFFFu, up ? low : high, o));
            }
          }
        }
        float best = -INFINITY;
#pragma unroll
        for (int k = 0; k < GC / 4; ++k)
          if (g0 + (lane & 3) * (GC / 4) + k < a.G) best = fmaxf(best, v[k]);
        best = fmaxf(best, __shfl_xor_sync(0xFFFFFFFFu, best, 2));
        best = fmaxf(best, __shfl_xor_sync(0xFFFFFFFFu, best, 1));
        const int p = (sub >> 2) * kPages + group;
        const int32_t j = (first + unit) * kUnitPages + p;
        if ((lane & 3) == 0 && j < n) {
          const bool outside = bad >> (kAhead * kUnitPages + p) & 1u;
          uint32_t key = key_of(outside ? -INFINITY : best);
          if (g0 > 0) key = max(key, keys[j]);
          if (!outside && (j < a.sink || j >= n - a.recent)) key = kForced;
          keys[j] = key;
        }
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    u += last - first;
    if (u >= u_end) break;
    first = 0;
    if (++h == a.H) {
      h = 0;
      do {
        ++b;
        units = cum[b] - cum[b - 1];
      } while (units == 0);
    }
  }
}

// ---- selection --------------------------------------------------------------------------
//
// One CTA for each list. The k-th largest key is found by its digits, from the highest bit in
// which the keys differ: a histogram of a digit in shared memory, the bin that holds the k-th,
// and so on inside that bin, until the bin is wanted as a whole. Then one pass in page order
// writes the pages above it and the first ones equal to it. It is a chain of short steps with a barrier
// or two between them: by itself, from cold caches, 9 us for 512 lists of up to 1024 pages and 11 us for 32
// lists of 7200, which leave four fifths of the SMs idle. 512 lists of up to 1024 pages take 4.6 us less in CTAs of 128 threads than of 512 (31.0 and
// 35.6 us with the scores), 16 lists of the same length 1.2 us more (12.0 and 10.8).

constexpr int kSelectThreads = 512, kShortThreads = 128;
constexpr int kDigit = 9, kBins = 1 << kDigit;
constexpr int kPerThread = 16;  // keys that a thread has in registers

// Sum of v[0 .. warp) over the warps' totals v (one for each warp, THREADS / 32 of them), and
// of all of them; every lane of a warp calls it.
template <int THREADS>
__device__ __forceinline__ uint32_t sum_before(const uint32_t* v, int warp, uint32_t* all) {
  const int lane = threadIdx.x & 31;
  const uint32_t x = lane < THREADS / 32 ? v[lane] : 0u;
  *all = __reduce_add_sync(0xFFFFFFFFu, x);
  return __reduce_add_sync(0xFFFFFFFFu, lane < warp ? x : 0u);
}

__device__ __forceinline__ uint32_t warp_sum(uint32_t v) { return __reduce_add_sync(0xFFFFFFFFu, v); }

template <int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == kShortThreads ? 6 : 2) select_pages_kernel(const SelectArgs a) {
  __shared__ uint32_t s_hist[kBins], s_red[4][THREADS / 32], s_bin, s_above, s_in_bin;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t item = blockIdx.x;
  const int32_t b = static_cast<int32_t>(item / a.H);
  const int32_t n = pages_of(a, b);
  const int32_t count = min(n, a.k);
  int32_t* out = a.selected + item * a.k;
  const uint32_t* keys = a.scores + item * a.pitch;
  wait_for_scores();  // (on every path: what follows this kernel in the stream follows the scores too)
  if (tid == 0) a.num_selected[item] = count;
  for (int32_t i = count + tid; i < a.k; i += THREADS) out[i] = -1;
  if (count == n) {
    for (int32_t j = tid; j < n; j += THREADS) out[j] = j;
    return;
  }
  // A thread's keys are neighbours, so that page order is thread order: `each_n` of them, in
  // registers; of a list longer than THREADS * kPerThread the rest is read again each time.
  constexpr int32_t kTile = THREADS * kPerThread;
  int32_t each_n = (n + THREADS - 1) / THREADS;
  each_n = each_n > 2 ? min((each_n + 3) & ~3, kPerThread) : each_n;
  uint32_t mine[kPerThread];
#pragma unroll
  for (int i = 0; i < kPerThread; i += 4) {
    const int32_t j = tid * each_n + i;
    uint4 v{};
    if (each_n > 2) {
      if (i < each_n && j < n) v = __ldcg(reinterpret_cast<const uint4*>(keys + j));  // (rows are padded to four)
    } else if (i == 0) {
      if (j < n) v.x = __ldcg(keys + j);
      if (each_n > 1 && j + 1 < n) v.y = __ldcg(keys + j + 1);
    }
    mine[i] = v.x; mine[i + 1] = v.y; mine[i + 2] = v.z; mine[i + 3] = v.w;
  }
  auto each = [&](auto body) {  // of this thread's keys
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      if (i >= each_n) break;
      if (tid * each_n + i < n) body(mine[i]);
    }
    for (int32_t t = kTile; t < n; t += kTile)
      for (int i = 0; i < kPerThread; ++i) {
        const int32_t j = t + tid * kPerThread + i;
        if (j < n) body(__ldcg(keys + j));
      }
  };
  uint32_t lo = 0xFFFFFFFFu, hi = 0, forced = 0;
  each([&](uint32_t k) {
    if (k == kForced) {
      ++forced;
    } else {
      lo = min(lo, k);
      hi = max(hi, k);
    }
  });
  lo = __reduce_min_sync(0xFFFFFFFFu, lo);
  hi = __reduce_max_sync(0xFFFFFFFFu, hi);
  forced = warp_sum(forced);
  if (lane == 0) {
    s_red[0][warp] = lo;
    s_red[1][warp] = hi;
    s_red[2][warp] = forced;
  }
  __syncthreads();
  lo = __reduce_min_sync(0xFFFFFFFFu, s_red[0][lane % (THREADS / 32)]);
  hi = __reduce_max_sync(0xFFFFFFFFu, s_red[1][lane % (THREADS / 32)]);
  sum_before<THREADS>(s_red[2], 0, &forced);
  // keys >= floor_ are taken, of those in [floor_, ceil_] the first `want` in page order
  uint32_t floor_ = kForced, ceil_ = kForced, want = count;
  if (forced < static_cast<uint32_t>(count)) {
    want = count - forced;
    // digits of key - base, `left` bits of them
    uint32_t base = lo, left = 32 - __clz(hi - lo);
    floor_ = lo;
    ceil_ = hi;
    uint32_t in_range = n - forced;
    while (left > 0 && in_range > want) {
      const uint32_t shift = left > kDigit ? left - kDigit : 0;
      for (int i = tid; i < kBins; i += THREADS) s_hist[i] = 0;
      __syncthreads();
      each([&](uint32_t k) {
        if (k >= floor_ && k <= ceil_) atomicAdd(s_hist + ((k - base) >> shift), 1u);
      });
      __syncthreads();
      // the bin of the want-th largest: bins from the top, kEach of them to a thread
      constexpr int kEach = kBins / THREADS;
      uint32_t c[kEach], own = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) own += c[i] = s_hist[kBins - 1 - (tid * kEach + i)];
      uint32_t sum = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += x;
      }
      if (lane == 31) s_red[3][warp] = sum;
      __syncthreads();
      uint32_t all;
      sum += sum_before<THREADS>(s_red[3], warp, &all);
      sum -= own;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        if (sum < want && sum + c[i] >= want) {
          s_bin = kBins - 1 - (tid * kEach + i);
          s_above = sum;
          s_in_bin = c[i];
        }
        sum += c[i];
      }
      __syncthreads();
      base += s_bin << shift;
      want -= s_above;
      in_range = s_in_bin;
      floor_ = base;
      const uint32_t top = base + ((1u << shift) - 1u);
      ceil_ = min(ceil_, top);
      left = shift;
      __syncthreads();
    }
  }
  // One pass in page order. taken = keys above the range, and the first `want` inside it.
  uint32_t base_above = 0, base_in = 0;
  for (int32_t t = 0; t < n; t += kTile) {
    uint32_t above = 0, in = 0;
    uint32_t k[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int32_t j = t + tid * each_n + i;
      k[i] = t == 0 ? mine[i] : (j < n ? __ldcg(keys + j) : 0u);
      if (i < each_n && j < n) {
        above += k[i] > ceil_;
        in += k[i] >= floor_ && k[i] <= ceil_;
      }
    }
    uint32_t sa = above, si = in;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, sa, o), y = __shfl_up_sync(0xFFFFFFFFu, si, o);
      if (lane >= o) {
        sa += x;
        si += y;
      }
    }
    __syncthreads();
    if (lane == 31) {
      s_red[0][warp] = sa;
      s_red[1][warp] = si;
    }
    __syncthreads();
    uint32_t a_all, i_all;
    uint32_t na = base_above + sa - above + sum_before<THREADS>(s_red[0], warp, &a_all);
    uint32_t ni = base_in + si - in + sum_before<THREADS>(s_red[1], warp, &i_all);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int32_t j = t + tid * each_n + i;
      if (i >= each_n || j >= n) continue;
      const bool is_above = k[i] > ceil_, is_in = k[i] >= floor_ && k[i] <= ceil_;
      if (is_above || (is_in && ni < want)) out[na + min(ni, want)] = j;
      na += is_above;
      ni += is_in;
    }
    base_above += a_all;
    base_in += i_all;
  }
}

template <int GC, int T>
nvfp4_status launch_scores(const SelectArgs& a, cudaStream_t stream) {
  const auto kern = page_scores_kernel<GC, T, GC == 4 ? 2 : 1>;
  const size_t smem = kScoreWarps * kScoreBytes + static_cast<size_t>(a.B) * 4;
  int64_t cap;
  if (nvfp4_status st = resident_ctas(reinterpret_cast<const void*>(kern), kScoreWarps * 32, smem, 32,
                                      "nvfp4_select_pages", &cap))
    return st;
  const int64_t most = (static_cast<int64_t>(a.B) * a.H * ((a.max_pages + kUnitPages - 1) / kUnitPages) + kScoreWarps - 1) / kScoreWarps;
  const int grid = static_cast<int>(most < cap ? most : cap);
  if (grid > 0) kern<<<grid, kScoreWarps * 32, smem, stream>>>(a);
  return check_launch("nvfp4_select_pages");
}

template <int GC>
nvfp4_status launch_scores_t(const SelectArgs& a, cudaStream_t stream) {
  if (a.D <= 64) return launch_scores<GC, 8>(a, stream);
  if (a.D <= 128) return launch_scores<GC, 16>(a, stream);
  return launch_scores<GC, 32>(a, stream);
}

}  // namespace

nvfp4_status launch_page_key_bounds(BoundsArgs a, cudaStream_t stream) {
  const int32_t columns = a.H * (a.D / 16);
  const int64_t codes = static_cast<int64_t>(a.ps) * a.H * (a.D / 2), scales = codes / 8;
  const bool ring = codes % 16 == 0 && scales % 16 == 0 && (codes + scales) * 2 <= kBoundsMostRing &&
                    reinterpret_cast<uintptr_t>(a.kc.sf) % 16 == 0 && a.kc.sf_page_stride % 16 == 0;
  size_t smem = static_cast<size_t>(a.B) * 4;
  int threads = kBoundsThreads;
  auto kern = page_key_bounds_kernel;
  if (ring) {
    a.code_bytes = static_cast<uint32_t>(codes);
    a.scale_bytes = static_cast<uint32_t>(scales);
    const int S = a.ps < 2 * kMaxSlots ? 1 : (a.ps < 4 * kMaxSlots ? 2 : 4);
    // a job for each warp, where the ring holds them
    a.pages = (kRingWarps * (32 / S) + columns - 1) / columns;
    if (a.pages > kRingPages) a.pages = kRingPages;
    while (a.pages > 1 && a.pages * (codes + scales) * 2 > kBoundsRing) --a.pages;
    a.stage_bytes = (a.pages * (a.code_bytes + a.scale_bytes) + 127) / 128 * 128;
    a.stages = static_cast<int32_t>(kBoundsRing / a.stage_bytes);
    a.stages = a.stages < 2 ? 2 : (a.stages > kMaxBoundsStages ? kMaxBoundsStages : a.stages);
    a.pipe = pipe_test_from_env();
    a.div_nb = make_div(a.D / 16);
    a.div_columns = make_div(columns);
    smem += static_cast<size_t>(a.stages) * a.stage_bytes;
    threads = (kRingWarps + 1) * 32;
    kern = S == 1 ? page_key_bounds_ring_kernel<1> : (S == 2 ? page_key_bounds_ring_kernel<2> : page_key_bounds_ring_kernel<4>);
  } else {
    a.tile = columns < kBoundsThreads ? columns : kBoundsThreads;
    a.slices = (a.ps + kMaxSlots - 1) / kMaxSlots;
    const int32_t most_slices = kBoundsThreads / a.tile;
    if (a.slices > most_slices) a.slices = most_slices;
    a.pages = kBoundsThreads / (a.tile * a.slices);
    if (a.pages > kBoundsThreads / 16) a.pages = kBoundsThreads / 16;
  }
  int64_t cap;
  if (nvfp4_status st = resident_ctas(reinterpret_cast<const void*>(kern), threads, smem, 32,
                                      "nvfp4_page_key_bounds", &cap))
    return st;
  const int64_t most = (a.B * a.max_pages + a.pages - 1) / a.pages;
  const int grid = static_cast<int>(most < cap ? most : cap);
  kern<<<grid, threads, smem, stream>>>(a);
  return check_launch("nvfp4_page_key_bounds");
}

// Keys of a list are 16-byte aligned.
static int64_t key_pitch(int64_t max_pages) { return (max_pages + 3) & ~int64_t(3); }

int64_t select_workspace_bytes(int32_t B, int32_t H, int64_t max_pages) {
  return static_cast<int64_t>(B) * H * key_pitch(max_pages) * 4;
}

nvfp4_status launch_select_pages(SelectArgs a, cudaStream_t stream) {
  a.pitch = key_pitch(a.max_pages);
  const nvfp4_status st = a.G <= 4 ? launch_scores_t<4>(a, stream) : launch_scores_t<8>(a, stream);
  if (st != NVFP4_OK) return st;
  cudaLaunchConfig_t config{};
  // lists that a small CTA holds in registers, and more of them than wide CTAs fit at once
  int64_t wide;
  if (nvfp4_status e = resident_ctas(reinterpret_cast<const void*>(select_pages_kernel<kSelectThreads>), kSelectThreads,
                                     0, 32, "nvfp4_select_pages", &wide))
    return e;
  const int64_t lists = static_cast<int64_t>(a.B) * a.H;
  const bool is_short = lists > wide && a.max_pages <= kShortThreads * kPerThread;
  config.gridDim = dim3(static_cast<unsigned>(lists));
  config.blockDim = dim3(is_short ? kShortThreads : kSelectThreads);
  config.stream = stream;
  cudaLaunchAttribute overlap{};
  overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  overlap.val.programmaticStreamSerializationAllowed = 1;
  config.attrs = &overlap;
  config.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(
      &config, is_short ? select_pages_kernel<kShortThreads> : select_pages_kernel<kSelectThreads>, a);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(NVFP4_ERR_CUDA, std::string("nvfp4_select_pages: ") + cudaGetErrorString(e));
  }
  return NVFP4_OK;
}

}  // namespace nvfp4
