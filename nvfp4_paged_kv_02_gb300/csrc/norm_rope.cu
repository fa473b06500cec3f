// norm_rope.cu -- RMS norm of the query and key rows of each head, rotation by position, and
// quantize-append of the key and value rows, in one pass over a step's projections.
//
// For one row x of D elements (query or key of one head; w its norm's weights):
//   r = 1 / sqrt(sum(x^2) * (1/D) + eps),  y = (x * r) * w
//   pairs (y_a, y_b) of the first R elements:  (y_a c - y_b s,  y_b c + y_a s)
// with (c, s) from the row of the table at the token's position; the rest of y passes through.
// Pairs are (i, i + R/2), or (2i, 2i+1) when interleaved. The result is rounded once to the
// input type; a key row then goes through the append's block rule (append.cu), as the rounded
// row would if it were handed to the append. Value rows are quantized as they are.
//
// All of it is binary32 with one rounding per operation and a fixed order of the sum of
// squares, so that the codes (which jump at the format's borders) are reproducible: eight
// squares t[i] += t[i+4], t[i+2], t[i+1]; the two groups of eight that rotate together are
// added; the D/16 pair sums, filled up with zeros to a power of two, add by halves.
//
// T = D/16 rounded up to a power of two lanes work on one row; lane j holds the two groups of
// eight elements that rotate together: groups j and j + R/16 below R/16, else 2j and 2j+1. A
// rotation then needs no exchange, and the sum of squares is in-lane plus log2(T) shuffles. A
// key row's 16-element blocks are put together through shared memory.
#include "internal.h"
#include "quantize.cuh"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;

// Exact binary32 values of eight packed elements.
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& v, float x[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = BF16 ? __uint_as_float(w[k] << 16) : f32_from_f16_lo(w[k]);
    x[2 * k + 1] = BF16 ? f32_from_bf16_hi(w[k]) : f32_from_f16_hi(w[k]);
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float x[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    w[k] = BF16 ? bf16x2_from_f32(x[2 * k], x[2 * k + 1]) : f16x2_from_f32(x[2 * k], x[2 * k + 1]);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float sum_squares8(const float x[8]) {
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = __fmul_rn(x[i], x[i]);
#pragma unroll
  for (int h = 4; h >= 1; h /= 2) {
#pragma unroll
    for (int i = 0; i < h; ++i) t[i] = __fadd_rn(t[i], t[i + h]);
  }
  return t[0];
}

// (a c - b s, b c + a s), one rounding per operation.
__device__ __forceinline__ void rotate(float& a, float& b, float c, float s) {
  const float ra = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = ra;
}

__device__ __forceinline__ void load4(const float* p, float v[4]) {
  const float4 f = __ldg(reinterpret_cast<const float4*>(p));
  v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
}

template <bool BF16, int MODE>
__global__ void __launch_bounds__(kThreads) norm_rope_append_kernel(const NormRopeArgs a) {
  __shared__ Tables tab;
  __shared__ __align__(16) uint4 s_rows[kThreads / 32][64];  // a warp's rows, as groups of eight
  float gs[2];
  if (!load_scales(a.ap, gs)) return;
  fill_tables<MODE>(tab, gs);
  const TensorConsts tc[2] = {make_consts(gs[0]), make_consts(gs[1])};

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int T = 1 << a.log2_T, j = lane & (T - 1), nt = a.ap.D / 16, nr = a.rotary_dim / 16;
  const int per_warp = 32 >> a.log2_T;
  const int ga = j < nr ? j : 2 * j, gb = j < nr ? j + nr : 2 * j + 1;  // this lane's groups
  const int32_t H = a.ap.H, row_kinds = a.Hq + 2 * H;
  const int64_t rows = a.ap.nnz * row_kinds;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32) * per_warp;
  for (int64_t first = (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + warp) * per_warp;
       first < rows; first += step) {
    const int64_t row = first + (lane >> a.log2_T);
    bool live = row < rows && j < nt;
    const int64_t i = live ? div_q(row, a.div_rows) : 0;
    const int32_t rr = live ? static_cast<int32_t>(row - i * row_kinds) : 0;
    const int kind = rr < a.Hq ? 0 : (rr < a.Hq + H ? 1 : 2);  // query, key, value
    const int32_t h = kind == 0 ? rr : (kind == 1 ? rr - a.Hq : rr - a.Hq - H);
    const int32_t pos = __ldg(a.ap.positions + i);
    if (live && nr > 0 && (pos < 0 || pos >= a.num_positions)) {
      flag(a.ap.status, NVFP4_DEV_BAD_POSITION);
      live = false;
    }
    const uint8_t* src = kind == 0 ? a.q + i * a.q_row_bytes
                                   : (kind == 1 ? a.ap.k + i * a.ap.k_row_bytes
                                                : a.ap.v + i * a.ap.v_row_bytes);
    src += static_cast<int64_t>(h) * a.ap.D * 2;
    const int pa = kind == 2 ? 2 * j : ga, pb = kind == 2 ? 2 * j + 1 : gb;
    uint4 va{}, vb{};
    if (live) {
      va = reinterpret_cast<const uint4*>(src)[pa];
      vb = reinterpret_cast<const uint4*>(src)[pb];
    }
    float xa[8], xb[8];
    unpack8<BF16>(va, xa);
    unpack8<BF16>(vb, xb);
    const uint8_t* w = kind == 0 ? a.q_weight : a.k_weight;
    float sum = __fadd_rn(sum_squares8(xa), sum_squares8(xb));
    for (int o = T >> 1; o > 0; o >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xFFFFFFFFu, sum, o));
    if (live && kind != 2 && w != nullptr) {
      const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(sum, a.inv_d), a.eps)));
      float wa[8], wb[8];
      unpack8<BF16>(__ldg(reinterpret_cast<const uint4*>(w) + ga), wa);
      unpack8<BF16>(__ldg(reinterpret_cast<const uint4*>(w) + gb), wb);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xa[e] = __fmul_rn(__fmul_rn(xa[e], r), wa[e]);
        xb[e] = __fmul_rn(__fmul_rn(xb[e], r), wb[e]);
      }
    }
    if (live && kind != 2 && j < nr) {
      const float* cs = a.cos_sin + static_cast<int64_t>(pos) * a.rotary_dim;
      const float* sn = cs + a.rotary_dim / 2;
      float c[8], s[8];
      if (a.interleaved) {
        load4(cs + 4 * ga, c);
        load4(cs + 4 * gb, c + 4);
        load4(sn + 4 * ga, s);
        load4(sn + 4 * gb, s + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          rotate(xa[2 * e], xa[2 * e + 1], c[e], s[e]);
          rotate(xb[2 * e], xb[2 * e + 1], c[4 + e], s[4 + e]);
        }
      } else {
        load4(cs + 8 * j, c);
        load4(cs + 8 * j + 4, c + 4);
        load4(sn + 8 * j, s);
        load4(sn + 8 * j + 4, s + 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) rotate(xa[e], xb[e], c[e], s[e]);
      }
    }
    if (kind != 2) {
      va = pack8<BF16>(xa);
      vb = pack8<BF16>(xb);
    }
    if (live && kind == 0) {
      uint4* dst = reinterpret_cast<uint4*>(a.q_out + i * a.q_out_row_bytes +
                                            static_cast<int64_t>(h) * a.ap.D * 2);
      dst[ga] = va;
      dst[gb] = vb;
    }
    if (!__any_sync(0xFFFFFFFFu, live && kind != 0)) continue;
    uint4* buf = s_rows[warp] + (lane - j) * 2;
    if (j < nt) {
      buf[pa] = va;
      buf[pb] = vb;
    }
    __syncwarp();
    if (live && kind != 0) {
      const RowMeta m = resolve_row(a.ap, i);
      const int kv = kind - 1;
      if (m.flags & (1 << kv)) {
        U32x8 in;
        const uint4 lo = buf[2 * j], hi = buf[2 * j + 1];
        in.w[0] = lo.x; in.w[1] = lo.y; in.w[2] = lo.z; in.w[3] = lo.w;
        in.w[4] = hi.x; in.w[5] = hi.y; in.w[6] = hi.z; in.w[7] = hi.w;
        const BlockOut q = quantize_block<BF16, MODE>(in, tc[kv], tab, kv, a.ap.cap_a, a.ap.neg_zero);
        const nvfp4_paged_cache& c = kv ? a.ap.vc : a.ap.kc;
        const int64_t r = a.ap.layout == NVFP4_NHD ? static_cast<int64_t>(m.slot) * H + h
                                                   : static_cast<int64_t>(h) * a.ap.ps + m.slot;
        uint8_t* dst = c.data + m.page * c.data_page_stride + r * (a.ap.D / 2) + 8 * j;
        *reinterpret_cast<uint2*>(dst) = make_uint2(q.c0, q.c1);
        c.sf[m.page * c.sf_page_stride + r * nt + j] = static_cast<uint8_t>(q.s);
      }
    }
    __syncwarp();
  }
}

template <bool BF16, int MODE>
nvfp4_status launch_t(const NormRopeArgs& a, cudaStream_t stream) {
  const auto kern = norm_rope_append_kernel<BF16, MODE>;
  const int64_t rows = a.ap.nnz * (a.Hq + 2 * static_cast<int64_t>(a.ap.H));
  const int64_t per_cta = (kThreads / 32) * (32 >> a.log2_T);
  const int64_t need = (rows + per_cta - 1) / per_cta;
  const int64_t cap = static_cast<int64_t>(sm_count()) *
                      blocks_per_sm(reinterpret_cast<const void*>(kern), kThreads, 0);
  const int grid = static_cast<int>(need < cap ? need : cap);
  kern<<<grid, kThreads, 0, stream>>>(a);
  return check_launch("nvfp4_qk_norm_rope_append_paged");
}

template <bool BF16>
nvfp4_status launch_m(const NormRopeArgs& a, int mode, cudaStream_t s) {
  switch (mode) {
    case 0: return launch_t<BF16, 0>(a, s);
    case 1: return launch_t<BF16, 1>(a, s);
    case 2: return launch_t<BF16, 2>(a, s);
    case 3: return launch_t<BF16, 3>(a, s);
    default: return launch_t<BF16, 4>(a, s);
  }
}

}  // namespace

nvfp4_status launch_norm_rope_append(const NormRopeArgs& a, bool bf16, int mode,
                                     cudaStream_t stream) {
  return bf16 ? launch_m<true>(a, mode, stream) : launch_m<false>(a, mode, stream);
}

}  // namespace nvfp4
