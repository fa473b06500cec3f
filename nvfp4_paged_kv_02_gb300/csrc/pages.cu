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
// Reading the keys bounds it: 9/16 byte an element, and 4 bytes written for page_size of them.
// A thread has one column, a 16-element block of a head, and its slots of one page; kBatch slots
// are loaded before the first is decoded. Pages of more than kMaxSlots slots give a column to
// several threads, which join in shared memory.

constexpr int kBoundsThreads = 256;
constexpr int kBatch = 8;
constexpr int kMaxSlots = 32;

__device__ __forceinline__ uint32_t hmin2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A CTA takes `pages` items of `tile` columns in `slices` threads each (their product is at most
// kBoundsThreads); tiles x items make its work. Thread: (item, slice, column), column fastest.
template <bool SLICED>
__global__ void __launch_bounds__(kBoundsThreads) page_key_bounds_kernel(const BoundsArgs a) {
  extern __shared__ int32_t s_cum[];
  __shared__ uint32_t s_part[SLICED ? 16 * kBoundsThreads : 1];
  const int tid = threadIdx.x, nb = a.D / 16;
  const int64_t reach = a.max_pages * a.ps;
  auto len_of = [&](int32_t b) { return min(static_cast<int64_t>(__ldg(a.seq_lens + b)), reach); };
  auto first_of = [&](int32_t b) {  // first page
    return a.first_positions ? div_q32(max(__ldg(a.first_positions + b), 0), a.div_ps) : 0;
  };
  block_inclusive_scan(s_cum, a.B, [&](int32_t b) {
    const int64_t len = len_of(b);
    if (blockIdx.x == 0 && __ldg(a.seq_lens + b) > reach) flag(a.status, NVFP4_DEV_LEN_CLAMPED);
    const int32_t pages = len > 0 ? div_q32(static_cast<int32_t>(len - 1), a.div_ps) + 1 : 0;
    return max(pages - first_of(b), 0);
  });
  const int32_t total = s_cum[a.B - 1];
  const int32_t columns = a.H * nb;
  const int my_col = tid % a.tile, my_slice = tid / a.tile % a.slices, my_item = tid / (a.tile * a.slices);
  const bool in_team = my_item < a.pages;

  for (int64_t item0 = static_cast<int64_t>(blockIdx.x) * a.pages; item0 < total;
       item0 += static_cast<int64_t>(gridDim.x) * a.pages) {
    const int32_t item = static_cast<int32_t>(min(item0 + my_item, static_cast<int64_t>(total - 1)));
    const bool live = in_team && item0 + my_item < total;
    const int32_t b = scan_find(s_cum, a.B, item);
    const int32_t col = item - (b > 0 ? s_cum[b - 1] : 0) + first_of(b);
    int64_t page = live ? table_entry(a.block_tables, a.table64, b * a.max_pages + col) : -1;
    if (page < 0 || page >= a.kc.num_pages) {
      if (live) flag(a.status, NVFP4_DEV_BAD_PAGE);
      page = -1;
    }
    const int32_t n = static_cast<int32_t>(min(static_cast<int64_t>(a.ps), len_of(b) - static_cast<int64_t>(col) * a.ps));
    const uint8_t* codes = a.kc.data + page * a.kc.data_page_stride;
    const uint8_t* scales = a.kc.sf + page * a.kc.sf_page_stride;
    for (int32_t c0 = 0; c0 < columns; c0 += a.tile) {
      const int32_t w = c0 + my_col;
      const bool mine = page >= 0 && w < columns;
      const int32_t h = w / nb, j = w - h * nb;
      // block of slot t: at + t * step
      const int32_t at = a.layout == NVFP4_NHD ? w : h * a.ps * nb + j;
      const int32_t step = a.layout == NVFP4_NHD ? columns : nb;
      uint32_t lo[8], hi[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        lo[e] = 0x7C007C00u;  // +inf, -inf: what a slice without slots leaves
        hi[e] = 0xFC00FC00u;
      }
      if (mine) {
        for (int32_t t0 = my_slice; t0 < n; t0 += kBatch * a.slices) {
          uint2 c[kBatch];
          uint32_t s[kBatch];
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const int32_t t = min(t0 + k * a.slices, n - 1);  // (past the end: the last slot again)
            const int32_t blk = at + t * step;
            c[k] = __ldg(reinterpret_cast<const uint2*>(codes) + blk);
            s[k] = __ldg(scales + blk);
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
              lo[e] = hmin2(lo[e], v[e]);
              hi[e] = hmax2(hi[e], v[e]);
            }
          }
        }
      }
      if (SLICED) {
        __syncthreads();  // what the last tile left has been read
        if (mine) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            s_part[e * kBoundsThreads + tid] = lo[e];
            s_part[(8 + e) * kBoundsThreads + tid] = hi[e];
          }
        }
        __syncthreads();
        if (mine && my_slice == 0) {
          for (int q = 1; q < a.slices; ++q) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              lo[e] = hmin2(lo[e], s_part[e * kBoundsThreads + tid + q * a.tile]);
              hi[e] = hmax2(hi[e], s_part[(8 + e) * kBoundsThreads + tid + q * a.tile]);
            }
          }
        }
      }
      if (mine && my_slice == 0) {
        uint4* dst = reinterpret_cast<uint4*>(a.bounds + (page * a.H + h) * 2 * a.D + 16 * j);
        uint4* dst_hi = reinterpret_cast<uint4*>(a.bounds + ((page * a.H + h) * 2 + 1) * a.D + 16 * j);
        dst[0] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        dst[1] = make_uint4(lo[4], lo[5], lo[6], lo[7]);
        dst_hi[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        dst_hi[1] = make_uint4(hi[4], hi[5], hi[6], hi[7]);
      }
    }
  }
}

// ---- scores -----------------------------------------------------------------------------
//
// A unit is kUnitPages pages of one (request, KV head). All units are cut into equal runs, one for each
// warp; a warp holds its query heads in registers (as positive and negative parts) and passes
// over the pages' bounds once, T lanes to a page (T = D/8 rounded up), each lane eight elements.
// A lane's bounds come through its own ring of stages in shared memory (cp.async; no other lane
// reads them, so a wait is all the synchronization there is). Reading the bounds bounds it, 4 D
// bytes a page and head; the 2 G D multiply-adds are packed two by two.

constexpr int kScoreWarps = 4;
constexpr int kScoreStages = 8;
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

__device__ __forceinline__ int32_t pages_of(const SelectArgs& a, int32_t b) {
  const int64_t len = min(static_cast<int64_t>(max(__ldg(a.seq_lens + b), 0)), a.max_pages * a.ps);
  return static_cast<int32_t>((len + a.ps - 1) / a.ps);
}

template <int GC, int T>
__global__ void __launch_bounds__(kScoreWarps * 32, GC == 4 ? 3 : 2) page_scores_kernel(const SelectArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kPages = 32 / T;  // of an iteration
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % T, group = lane / T;
  int32_t* cum = reinterpret_cast<int32_t*>(smem + kScoreWarps * kScoreStages * 1024);
  block_inclusive_scan(cum, a.B, [&](int32_t b) {
    if (blockIdx.x == 0 && __ldg(a.seq_lens + b) > a.max_pages * a.ps) flag(a.status, NVFP4_DEV_LEN_CLAMPED);
    return (pages_of(a, b) + kUnitPages - 1) / kUnitPages;
  });
  const int64_t total = static_cast<int64_t>(cum[a.B - 1]) * a.H;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kScoreWarps;
  const int64_t me = static_cast<int64_t>(blockIdx.x) * kScoreWarps + warp;
  int64_t u = total * me / warps;
  const int64_t u_end = total * (me + 1) / warps;
  if (u >= u_end) return;
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem + warp * kScoreStages * 1024)) + lane * 16;

  // the list of unit u: units run over requests, then heads, then pages
  int32_t b = scan_find(cum, a.B, static_cast<int32_t>(u / a.H));
  int32_t units = cum[b] - (b > 0 ? cum[b - 1] : 0);
  int64_t in_request = u - static_cast<int64_t>(b > 0 ? cum[b - 1] : 0) * a.H;
  int32_t h = static_cast<int32_t>(in_request / units), first = static_cast<int32_t>(in_request % units);

  const bool active = 8 * sub < a.D;
  for (;;) {
    const int32_t n = pages_of(a, b);
    const int32_t last = static_cast<int32_t>(min(static_cast<int64_t>(units), first + (u_end - u)));
    uint32_t* keys = a.scores + (static_cast<int64_t>(b) * a.H + h) * a.max_pages;
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
      // iterations: kPages pages each, kIts of them to a unit
      constexpr int kIts = kUnitPages / kPages;
      const int32_t it_end = (last - first) * kIts;
      int32_t issued = 0, entry_unit = -1, entry = -1;
      auto issue = [&] {
        if (issued < it_end) {
          const int32_t unit = issued / kIts;
          if (unit != entry_unit) {  // the unit's pages, one to a lane
            entry_unit = unit;
            const int32_t col = (first + unit) * kUnitPages + lane;
            entry = -1;
            if (lane < kUnitPages && col < n) {
              const int64_t page = table_entry(a.block_tables, a.table64, b * a.max_pages + col);
              if (page >= 0 && page < a.num_pages) entry = static_cast<int32_t>(page);
              else flag(a.status, NVFP4_DEV_BAD_PAGE);
            }
          }
          const int32_t page = __shfl_sync(0xFFFFFFFFu, entry, issued % kIts * kPages + group);
          const bool live = page >= 0 && active;
          const uint16_t* src = a.bounds + ((static_cast<int64_t>(live ? page : 0) * a.H + h) * 2 * a.D + (live ? 8 * sub : 0));
          const uint32_t dst = ring + issued % kScoreStages * 1024;
          const int bytes = live ? 16 : 0;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 512), "l"(src + a.D), "r"(bytes) : "memory");
        }
        ++issued;
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      for (int s = 0; s < kScoreStages - 1; ++s) issue();
      float mine = -INFINITY;
      for (int32_t it = 0; it < it_end; ++it) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kScoreStages - 2) : "memory");
        const uint8_t* st = smem + warp * kScoreStages * 1024 + it % kScoreStages * 1024 + lane * 16;
        const uint4 lw = *reinterpret_cast<const uint4*>(st), hw = *reinterpret_cast<const uint4*>(st + 512);
        issue();
        const uint64_t lo[4] = {widen2(lw.x), widen2(lw.y), widen2(lw.z), widen2(lw.w)};
        const uint64_t hi[4] = {widen2(hw.x), widen2(hw.y), widen2(hw.z), widen2(hw.w)};
        float v[GC];
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
          v[g] = __fadd_rn(x, y);
        }
        // Sums over the T lanes by halves. While a lane has several heads left it gives half of them
        // to its partner and keeps the other half.
        int cnt = GC, mine_g = 0;
#pragma unroll
        for (int o = T / 2; o >= 1; o /= 2) {
          if (cnt > 1) {
            cnt /= 2;
            const bool up = lane & o;
#pragma unroll
            for (int k = 0; k < GC / 2; ++k) {
              if (k < cnt) {
                const float give = up ? v[k] : v[k + cnt], keep = up ? v[k + cnt] : v[k];
                v[k] = __fadd_rn(keep, __shfl_xor_sync(0xFFFFFFFFu, give, o));
              }
            }
            if (up) mine_g += cnt;
          } else {
            v[0] = __fadd_rn(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], o));
          }
        }
        // the maximum over the heads: lanes that differ in the bits that chose a head
        float best = -INFINITY;
#pragma unroll
        for (int k = 0; k < (GC > T ? GC / T : 1); ++k)
          best = fmaxf(best, g0 + mine_g + k < a.G ? v[k] : -INFINITY);
#pragma unroll
        for (int o = T / 2; o >= (T > GC ? T / GC : 1); o /= 2) best = fmaxf(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
        // lane l keeps the score of the unit's page l
        const float got = __shfl_sync(0xFFFFFFFFu, best, lane % kPages * T);
        if (lane / kPages == it % kIts) mine = got;
        if (it % kIts == kIts - 1) {
          const int32_t j = (first + it / kIts) * kUnitPages + lane;
          if (lane < kUnitPages && j < n) {
            // (a page outside the pool was copied as zeros: it comes last)
            const int64_t page = table_entry(a.block_tables, a.table64, b * a.max_pages + j);
            const bool bad = page < 0 || page >= a.num_pages;
            uint32_t key = bad ? key_of(-INFINITY) : key_of(mine);
            if (g0 > 0) key = max(key, keys[j]);
            if (j < a.sink || j >= n - a.recent) key = kForced;
            keys[j] = key;
          }
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
// writes the pages above it and the first ones equal to it.

constexpr int kSelectThreads = 512;
constexpr int kDigit = 9, kBins = 1 << kDigit;
constexpr int kPerThread = 16;  // keys that a thread has in registers

__device__ __forceinline__ uint32_t warp_sum(uint32_t v) { return __reduce_add_sync(0xFFFFFFFFu, v); }

__global__ void __launch_bounds__(kSelectThreads) select_pages_kernel(const SelectArgs a) {
  __shared__ uint32_t s_hist[kBins], s_red[4][kSelectThreads / 32], s_bin, s_above, s_in_bin;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t item = blockIdx.x;
  const int32_t b = static_cast<int32_t>(item / a.H);
  const int32_t n = pages_of(a, b);
  const int32_t count = min(n, a.k);
  int32_t* out = a.selected + item * a.k;
  const uint32_t* keys = a.scores + item * a.max_pages;
  if (tid == 0) a.num_selected[item] = count;
  for (int32_t i = count + tid; i < a.k; i += kSelectThreads) out[i] = -1;
  if (count == n) {
    for (int32_t j = tid; j < n; j += kSelectThreads) out[j] = j;
    return;
  }
  // A thread's keys are neighbours, so that page order is thread order: `each_n` of them, in
  // registers; of a list longer than kSelectThreads * kPerThread the rest is read again each time.
  constexpr int32_t kTile = kSelectThreads * kPerThread;
  const int32_t each_n = min((n + kSelectThreads - 1) / kSelectThreads, kPerThread);
  uint32_t mine[kPerThread];
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int32_t j = tid * each_n + i;
    mine[i] = i < each_n && j < n ? __ldcg(keys + j) : 0u;
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
  forced = 0;
  for (int w = 0; w < kSelectThreads / 32; ++w) {
    lo = min(lo, s_red[0][w]);
    hi = max(hi, s_red[1][w]);
    forced += s_red[2][w];
  }
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
      for (int i = tid; i < kBins; i += kSelectThreads) s_hist[i] = 0;
      __syncthreads();
      each([&](uint32_t k) {
        if (k >= floor_ && k <= ceil_) atomicAdd(s_hist + ((k - base) >> shift), 1u);
      });
      __syncthreads();
      // the bin of the want-th largest: bins from the top, kBins = kSelectThreads of them
      static_assert(kBins == kSelectThreads, "one bin to a thread");
      const uint32_t c = s_hist[kBins - 1 - tid];
      uint32_t sum = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += x;
      }
      if (lane == 31) s_red[3][warp] = sum;
      __syncthreads();
      uint32_t before = 0;
      for (int w = 0; w < warp; ++w) before += s_red[3][w];
      sum += before;
      if (sum >= want && sum - c < want) {
        s_bin = kBins - 1 - tid;
        s_above = sum - c;
        s_in_bin = c;
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
    uint32_t a_all = 0, i_all = 0, na = base_above + sa - above, ni = base_in + si - in;
    for (int w = 0; w < kSelectThreads / 32; ++w) {
      if (w < warp) {
        na += s_red[0][w];
        ni += s_red[1][w];
      }
      a_all += s_red[0][w];
      i_all += s_red[1][w];
    }
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
  const auto kern = page_scores_kernel<GC, T>;
  const size_t smem = kScoreWarps * kScoreStages * 1024 + static_cast<size_t>(a.B) * 4;
  if (nvfp4_status st = set_dynamic_smem(reinterpret_cast<const void*>(kern), smem, "nvfp4_select_pages")) return st;
  const int64_t cap = static_cast<int64_t>(sm_count()) *
                      blocks_per_sm(reinterpret_cast<const void*>(kern), kScoreWarps * 32, smem);
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
  a.tile = columns < kBoundsThreads ? columns : kBoundsThreads;
  a.slices = (a.ps + kMaxSlots - 1) / kMaxSlots;
  const int32_t most_slices = kBoundsThreads / a.tile;
  if (a.slices > most_slices) a.slices = most_slices;
  a.pages = kBoundsThreads / (a.tile * a.slices);
  const auto kern = a.slices > 1 ? page_key_bounds_kernel<true> : page_key_bounds_kernel<false>;
  const void* f = reinterpret_cast<const void*>(kern);
  const size_t smem = static_cast<size_t>(a.B) * 4;
  if (nvfp4_status st = set_dynamic_smem(f, smem, "nvfp4_page_key_bounds")) return st;
  const int64_t cap = static_cast<int64_t>(sm_count()) * blocks_per_sm(f, kBoundsThreads, smem);
  const int64_t most = (a.B * a.max_pages + a.pages - 1) / a.pages;
  const int grid = static_cast<int>(most < cap ? most : cap);
  kern<<<grid, kBoundsThreads, smem, stream>>>(a);
  return check_launch("nvfp4_page_key_bounds");
}

int64_t select_workspace_bytes(int32_t B, int32_t H, int64_t max_pages) {
  return static_cast<int64_t>(B) * H * max_pages * 4;
}

nvfp4_status launch_select_pages(const SelectArgs& a, cudaStream_t stream) {
  const nvfp4_status st = a.G <= 4 ? launch_scores_t<4>(a, stream) : launch_scores_t<8>(a, stream);
  if (st != NVFP4_OK) return st;
  select_pages_kernel<<<a.B * a.H, kSelectThreads, 0, stream>>>(a);
  return check_launch("nvfp4_select_pages");
}

}  // namespace nvfp4
