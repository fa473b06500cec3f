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

namespace nvfp4 {
namespace {

__device__ __forceinline__ int64_t table_entry(const void* tables, int32_t is64, int64_t at) {
  return is64 ? __ldg(static_cast<const int64_t*>(tables) + at)
              : __ldg(static_cast<const int32_t*>(tables) + at);
}

// ---- bounds -----------------------------------------------------------------------------

constexpr int kBoundsThreads = 128;

// A CTA walks the pages of request blockIdx.y; a thread has one 16-element block of one head.
__global__ void __launch_bounds__(kBoundsThreads) page_key_bounds_kernel(const BoundsArgs a) {
  const int32_t b = blockIdx.y, nb = a.D / 16;
  int64_t len = __ldg(a.seq_lens + b);
  const int64_t reach = a.max_pages * a.ps;
  if (len > reach) {
    if (threadIdx.x == 0 && blockIdx.x == 0) flag(a.status, NVFP4_DEV_LEN_CLAMPED);
    len = reach;
  }
  const int64_t from = a.first_positions ? max(__ldg(a.first_positions + b), 0) : 0;
  for (int64_t col = from / a.ps + blockIdx.x; col * a.ps < len; col += gridDim.x) {
    const int64_t page = table_entry(a.block_tables, a.table64, b * a.max_pages + col);
    if (page < 0 || page >= a.kc.num_pages) {
      if (threadIdx.x == 0) flag(a.status, NVFP4_DEV_BAD_PAGE);
      continue;
    }
    const int32_t n = static_cast<int32_t>(min(static_cast<int64_t>(a.ps), len - col * a.ps));
    for (int32_t w = threadIdx.x; w < a.H * nb; w += kBoundsThreads) {
      const int32_t h = w / nb, j = w - h * nb;
      uint32_t lo[8], hi[8];
      for (int32_t t = 0; t < n; ++t) {
        const int64_t r = a.layout == NVFP4_NHD ? static_cast<int64_t>(t) * a.H + h
                                                : static_cast<int64_t>(h) * a.ps + t;
        const uint2 c = __ldg(reinterpret_cast<const uint2*>(
            a.kc.data + page * a.kc.data_page_stride + r * (a.D / 2)) + j);
        const uint32_t s = __ldg(a.kc.sf + page * a.kc.sf_page_stride + r * nb + j);
        const uint32_t S2 = f16x2_from_e4m3x2(s * 0x0101u);
        uint32_t v[8];
        f16x2x4_from_e2m1x8(c.x, v[0], v[1], v[2], v[3]);
        f16x2x4_from_e2m1x8(c.y, v[4], v[5], v[6], v[7]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[e] = hmul2_rn(v[e], S2);
          asm("min.f16x2 %0, %1, %2;" : "=r"(lo[e]) : "r"(t ? lo[e] : v[e]), "r"(v[e]));
          asm("max.f16x2 %0, %1, %2;" : "=r"(hi[e]) : "r"(t ? hi[e] : v[e]), "r"(v[e]));
        }
      }
      uint4* dst = reinterpret_cast<uint4*>(a.bounds + (page * a.H + h) * 2 * a.D + 16 * j);
      uint4* dst_hi = reinterpret_cast<uint4*>(a.bounds + ((page * a.H + h) * 2 + 1) * a.D + 16 * j);
      dst[0] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      dst[1] = make_uint4(lo[4], lo[5], lo[6], lo[7]);
      dst_hi[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      dst_hi[1] = make_uint4(hi[4], hi[5], hi[6], hi[7]);
    }
  }
}

// ---- selection --------------------------------------------------------------------------

constexpr int kSelectThreads = 256;

// Unsigned keys in the order of the scores.
__device__ __forceinline__ uint32_t key_of(float s) {
  const uint32_t u = __float_as_uint(s + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// A CTA scores the pages of one (request, KV head), a page to T lanes, finds the k-th largest
// key by its bytes, and writes the pages above it and the first ones equal to it.
__global__ void __launch_bounds__(kSelectThreads) select_pages_kernel(const SelectArgs a) {
  const int64_t item = blockIdx.x;
  const int32_t b = static_cast<int32_t>(item / a.H), h = static_cast<int32_t>(item % a.H);
  const int64_t reach = a.max_pages * a.ps;
  int64_t len = max(__ldg(a.seq_lens + b), 0);
  if (len > reach) {
    if (threadIdx.x == 0 && h == 0) flag(a.status, NVFP4_DEV_LEN_CLAMPED);
    len = reach;
  }
  const int64_t n = (len + a.ps - 1) / a.ps;
  const int32_t count = static_cast<int32_t>(min(n, static_cast<int64_t>(a.k)));
  int32_t* out = a.selected + item * a.k;
  uint32_t* keys = a.scores + item * a.max_pages;
  if (threadIdx.x == 0) a.num_selected[item] = count;
  for (int32_t i = count + threadIdx.x; i < a.k; i += kSelectThreads) out[i] = -1;

  const int slices = a.D / 8;
  int T = 1;
  while (T < slices) T *= 2;
  const int sub = threadIdx.x % 32;  // one warp to a page; lanes take groups of eight
  for (int64_t j = threadIdx.x / 32; j < n; j += kSelectThreads / 32) {
    const int64_t page = table_entry(a.block_tables, a.table64, b * a.max_pages + j);
    float best = -INFINITY;
    if (page < 0 || page >= a.num_pages) {
      if (sub == 0) flag(a.status, NVFP4_DEV_BAD_PAGE);
    } else {
      for (int32_t g = 0; g < a.G; ++g) {
        float s = 0.0f;
        if (sub < slices) {
          const uint16_t* lo = a.bounds + (page * a.H + h) * 2 * a.D + 8 * sub;
          const uint16_t* hi = lo + a.D;
          const uint8_t* q = a.q + b * a.q_row_bytes + ((static_cast<int64_t>(h) * a.G + g) * a.D + 8 * sub) * 2;
          float chain[2] = {0.0f, 0.0f};
          for (int e = 0; e < 8; ++e) {
            const uint32_t w = reinterpret_cast<const uint16_t*>(q)[e];
            const float x = a.bf16 ? __uint_as_float(w << 16) : f32_from_f16_lo(w);
            chain[e & 1] = __fadd_rn(chain[e & 1], __fmul_rn(x, f32_from_f16_lo(x > 0.0f ? hi[e] : lo[e])));
          }
          s = __fadd_rn(chain[0], chain[1]);
        }
        for (int o = T / 2; o > 0; o /= 2) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, o));
        best = fmaxf(best, s);
      }
    }
    if (j < a.sink || j >= n - a.recent) best = INFINITY;
    if (sub == 0) keys[j] = key_of(best);
  }
  __syncthreads();
  if (count == n) {
    for (int64_t j = threadIdx.x; j < n; j += kSelectThreads) out[j] = static_cast<int32_t>(j);
    return;
  }
  __shared__ uint32_t s_hist[256];
  __shared__ uint32_t s_prefix, s_want, s_base[2], s_warp[2][kSelectThreads / 32];
  if (threadIdx.x == 0) {
    s_prefix = 0;
    s_want = count;  // keys still to be taken among those that share the prefix
  }
  for (int shift = 24; shift >= 0; shift -= 8) {
    s_hist[threadIdx.x] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix, mask = shift == 24 ? 0u : ~((1u << (shift + 8)) - 1u);
    for (int64_t j = threadIdx.x; j < n; j += kSelectThreads)
      if ((keys[j] & mask) == prefix) atomicAdd(s_hist + ((keys[j] >> shift) & 255u), 1u);
    __syncthreads();
    if (threadIdx.x == 0) {
      uint32_t want = s_want;
      int d = 255;
      while (s_hist[d] < want) want -= s_hist[d--];
      s_want = want;
      s_prefix = prefix | (static_cast<uint32_t>(d) << shift);
    }
    __syncthreads();
  }
  // in page order: every key above the k-th, and the first s_want of those equal to it
  const uint32_t kth = s_prefix, ties = s_want;
  if (threadIdx.x < 2) s_base[threadIdx.x] = 0;
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int64_t j0 = 0; j0 < n; j0 += kSelectThreads) {
    const int64_t j = j0 + threadIdx.x;
    const uint32_t key = j < n ? keys[j] : 0u;
    const bool eq = j < n && key == kth, gt = j < n && key > kth;
    const uint32_t beq = __ballot_sync(0xFFFFFFFFu, eq), bgt = __ballot_sync(0xFFFFFFFFu, gt);
    if (lane == 0) {
      s_warp[0][warp] = __popc(beq);
      s_warp[1][warp] = __popc(bgt);
    }
    __syncthreads();
    uint32_t neq = s_base[0], ngt = s_base[1], alleq = neq, allgt = ngt;
    for (int w = 0; w < kSelectThreads / 32; ++w) {
      if (w < warp) {
        neq += s_warp[0][w];
        ngt += s_warp[1][w];
      }
      alleq += s_warp[0][w];
      allgt += s_warp[1][w];
    }
    const uint32_t below = (1u << lane) - 1u;
    neq += __popc(beq & below);
    ngt += __popc(bgt & below);
    if (gt || (eq && neq < ties)) out[ngt + min(neq, ties)] = static_cast<int32_t>(j);
    __syncthreads();
    if (threadIdx.x == 0) {
      s_base[0] = alleq;
      s_base[1] = allgt;
    }
    __syncthreads();
  }
}

}  // namespace

nvfp4_status launch_page_key_bounds(const BoundsArgs& a, cudaStream_t stream) {
  const int64_t per = 8 * static_cast<int64_t>(sm_count()) / a.B + 1;
  const int gx = static_cast<int>(a.max_pages < per ? a.max_pages : per);
  page_key_bounds_kernel<<<dim3(gx, a.B), kBoundsThreads, 0, stream>>>(a);
  return check_launch("nvfp4_page_key_bounds");
}

int64_t select_workspace_bytes(int32_t B, int32_t H, int64_t max_pages) {
  return static_cast<int64_t>(B) * H * max_pages * 4;
}

nvfp4_status launch_select_pages(const SelectArgs& a, cudaStream_t stream) {
  select_pages_kernel<<<a.B * a.H, kSelectThreads, 0, stream>>>(a);
  return check_launch("nvfp4_select_pages");
}

}  // namespace nvfp4
