// attention.cu -- attention of one new token per request over a paged NVFP4 cache.
//
// For request b, query head i of KV head h = i / G (G = Hq / H), over the live tokens t:
//   x_t = sm_scale * gs_k * sum_d q[d] (e2m1 * S)_K[t, d]      (soft cap c: c tanh(x_t / c))
//   out = gs_v * sum_t exp(x_t - m) (e2m1 * S)_V[t, :] / l,    m = max x_t, l = sum exp(x_t - m)
//   lse = m + log(l)
// in one pass with a running maximum and sum; statistics and sums are binary32, e2m1 * S is
// exact. No live token: out = 0, lse = -inf.
#include "attention.h"

#include <cfloat>

namespace nvfp4 {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxPerLane = kAttnMaxHeadDim / 64;

__device__ __forceinline__ float f32_of16(const uint8_t* p, bool bf16) {
  const uint32_t w = *reinterpret_cast<const uint16_t*>(p);
  return bf16 ? __uint_as_float(w << 16) : f32_from_f16_lo(w);
}

__device__ __forceinline__ float2 code_pair(uint32_t byte, float s) {
  uint32_t h[4];
  f16x2x4_from_e2m1x8(byte, h[0], h[1], h[2], h[3]);
  return make_float2(f32_from_f16_lo(h[0]) * s, f32_from_f16_hi(h[0]) * s);
}

__device__ __forceinline__ float scale_of(uint32_t byte) {
  return f32_from_f16_lo(f16x2_from_e4m3x2(byte));
}

// One warp for each (request, query head); its lanes share the head dimension.
__global__ void __launch_bounds__(kWarps * 32) attention_kernel(const AttentionArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (item >= static_cast<int64_t>(a.B) * a.Hq) return;
  const int32_t b = static_cast<int32_t>(item / a.Hq), hq = static_cast<int32_t>(item % a.Hq);
  const int32_t h = hq / a.G, nbytes = a.D / 2;
  const int64_t reach = a.max_pages * a.ps;
  int64_t len = __ldg(a.seq_lens + b);
  if (len > reach) {
    if (lane == 0) flag(a.status, NVFP4_DEV_LEN_CLAMPED);
    len = reach;
  }
  const int64_t lo = a.window_left >= 0 ? max(int64_t(0), len - 1 - a.window_left) : 0;
  int64_t n = len;  // positions walked: tokens, or slots of the selected pages
  if (a.selected) n = static_cast<int64_t>(min(max(__ldg(a.num_selected + b * a.H + h), 0), a.max_selected)) * a.ps;

  float q[2 * kMaxPerLane], o[2 * kMaxPerLane], m = -INFINITY, l = 0.0f;
  for (int u = 0; u < kMaxPerLane; ++u) {
    const int byte = lane + 32 * u;
    const uint8_t* p = a.q + b * a.q_row_bytes + (static_cast<int64_t>(hq) * a.D + 2 * byte) * 2;
    q[2 * u] = byte < nbytes ? f32_of16(p, a.bf16) : 0.0f;
    q[2 * u + 1] = byte < nbytes ? f32_of16(p + 2, a.bf16) : 0.0f;
    o[2 * u] = o[2 * u + 1] = 0.0f;
  }
  // the query's power of two moves into the scale, so that no product overflows
  float top = 0.0f;
  for (int u = 0; u < 2 * kMaxPerLane; ++u) top = fmaxf(top, fabsf(q[u]));
  for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, s));
  const int e = top > 0.0f && top < INFINITY ? ilogbf(top) : 0;
  for (int u = 0; u < 2 * kMaxPerLane; ++u) q[u] = ldexpf(q[u], -e);
  const float scale = ldexpf(a.sm_scale, e) * __ldg(a.k_scale);
  for (int64_t i = a.selected ? 0 : lo; i < n; ++i) {
    int64_t col = i / a.ps, t = i;
    const int32_t slot = static_cast<int32_t>(i - col * a.ps);
    if (a.selected) {
      col = __ldg(a.selected + (static_cast<int64_t>(b) * a.H + h) * a.max_selected + col);
      if (col < 0 || col >= a.max_pages) {
        if (lane == 0) flag(a.status, NVFP4_DEV_BAD_PAGE);
        continue;
      }
      t = col * a.ps + slot;
    }
    if (t >= len) continue;
    const int64_t at = b * a.max_pages + col;
    const int64_t page = a.table64 ? reinterpret_cast<const int64_t*>(a.block_tables)[at]
                                   : reinterpret_cast<const int32_t*>(a.block_tables)[at];
    if (page < 0 || page >= a.kc.num_pages || page >= a.vc.num_pages) {
      if (lane == 0) flag(a.status, NVFP4_DEV_BAD_PAGE);
      continue;
    }
    const int64_t r = a.layout == NVFP4_NHD ? static_cast<int64_t>(slot) * a.H + h
                                            : static_cast<int64_t>(h) * a.ps + slot;
    const uint8_t* kd = a.kc.data + page * a.kc.data_page_stride + r * nbytes;
    const uint8_t* ks = a.kc.sf + page * a.kc.sf_page_stride + r * (a.D / 16);
    const uint8_t* vd = a.vc.data + page * a.vc.data_page_stride + r * nbytes;
    const uint8_t* vs = a.vc.sf + page * a.vc.sf_page_stride + r * (a.D / 16);
    float x = 0.0f;
    for (int u = 0; u < kMaxPerLane; ++u) {
      const int byte = lane + 32 * u;
      if (byte < nbytes) {
        const float2 k = code_pair(kd[byte], scale_of(ks[byte / 8]));
        x += q[2 * u] * k.x + q[2 * u + 1] * k.y;
      }
    }
    for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, s);
    x *= scale;
    if (a.soft_cap > 0.0f) x = a.soft_cap * tanhf(x / a.soft_cap);
    const float m2 = fmaxf(m, x), f = m2 == -INFINITY ? 1.0f : __expf(m - m2);
    const float p = m2 == -INFINITY ? 0.0f : __expf(x - m2);
    m = m2;
    l = l * f + p;
    for (int u = 0; u < kMaxPerLane; ++u) {
      const int byte = lane + 32 * u;
      if (byte < nbytes) {
        const float2 v = code_pair(vd[byte], scale_of(vs[byte / 8]));
        o[2 * u] = o[2 * u] * f + p * v.x;
        o[2 * u + 1] = o[2 * u + 1] * f + p * v.y;
      }
    }
  }
  const float inv = l == 0.0f ? 0.0f : __ldg(a.v_scale) / l;
  for (int u = 0; u < kMaxPerLane; ++u) {
    const int byte = lane + 32 * u;
    if (byte < nbytes) {
      uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + ((static_cast<int64_t>(b) * a.Hq + hq) * a.D + 2 * byte) * 2);
      *dst = a.bf16 ? bf16x2_from_f32(o[2 * u] * inv, o[2 * u + 1] * inv)
                    : f16x2_from_f32(o[2 * u] * inv, o[2 * u + 1] * inv);
    }
  }
  if (a.lse && lane == 0) a.lse[static_cast<int64_t>(b) * a.Hq + hq] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace

int64_t attention_workspace_bytes(int32_t, int32_t, int32_t) { return NVFP4_COUNTER_BYTES; }

nvfp4_status launch_attention(const AttentionArgs& a, cudaStream_t stream) {
  const int64_t items = static_cast<int64_t>(a.B) * a.Hq;
  const int grid = static_cast<int>((items + kWarps - 1) / kWarps);
  attention_kernel<<<grid, kWarps * 32, 0, stream>>>(a);
  return check_launch("nvfp4_paged_attention_decode");
}

}  // namespace nvfp4
