// quantize.cuh -- what every quantizing kernel shares: one 16-element block to NVFP4 (E4M3
// scale, E2M1 codes; the arithmetic is described in append.cu) and the page and slot of an
// appended row.
#pragma once

#include <cfloat>

#include "internal.h"

namespace nvfp4 {

// Per-tensor constants for one block quantization.
struct TensorConsts {
  float gs;       // global decode scale
  uint32_t neg_gh2;  // -RN16(gs) in both binary16 halves (binary16 error)
  float g6, r6;   // fp32(6 gs) and its reciprocal
  float g4, r4;   // 4 gs and its reciprocal
  bool exact_rcp; // both divisors and reciprocals are normal: use div_rn_with_rcp
};

__device__ __forceinline__ TensorConsts make_consts(float gs) {
  TensorConsts c;
  c.gs = gs;
  const uint32_t gh = static_cast<uint32_t>(__half_as_ushort(__float2half_rn(gs))) ^ 0x8000u;
  c.neg_gh2 = gh | (gh << 16);
  c.g6 = __fmul_rn(6.0f, gs);
  c.g4 = __fmul_rn(4.0f, gs);
  c.r6 = __frcp_rn(c.g6);
  c.r4 = __frcp_rn(c.g4);
  const float lo = FLT_MIN, hi = FLT_MAX;
  c.exact_rcp = c.g6 >= lo && c.g6 <= hi && c.g4 >= lo && c.r6 >= lo && c.r6 <= hi &&
                c.r4 >= lo && c.r4 <= hi;
  return c;
}

// RN(a / b). EXACT: the caller knows that b and rb are normal (div_rn_with_rcp applies).
template <bool EXACT>
__device__ __forceinline__ float quotient(float a, float b, float rb, bool exact_rcp) {
  if (EXACT) return div_rn_with_rcp(a, b, rb);
  return exact_rcp ? div_rn_with_rcp(a, b, rb) : __fdiv_rn(a, b);
}

// Exact binary32 values of the 16 elements. For bf16 the low half is widened with an
// integer multiply by 2^16 (the FMA pipe) rather than a shift (the half-rate ALU pipe,
// which the E2M1 decodes already keep busy).
template <bool BF16>
__device__ __forceinline__ void unpack16(const U32x8& in, float x[16]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (BF16) {
      uint32_t lo;
      asm("mul.lo.u32 %0, %1, 65536;" : "=r"(lo) : "r"(in.w[k]));
      x[2 * k] = __uint_as_float(lo);
      x[2 * k + 1] = f32_from_bf16_hi(in.w[k]);
    } else {
      x[2 * k] = f32_from_f16_lo(in.w[k]);
      x[2 * k + 1] = f32_from_f16_hi(in.w[k]);
    }
  }
}

// Four element pairs (x[0..7]) with multiplier inv: the four code bytes, and the decoded
// values e2m1(q) as four half2. The decodes read the bytes of the packed word (which takes
// fewer integer instructions than decoding each conversion result).
__device__ __forceinline__ uint32_t encode8(const float* x, float inv, uint32_t v[4]) {
  uint32_t code;
  asm("{\n\t"
      ".reg .b64 ip, p0, p1, p2, p3;\n\t"
      ".reg .f32 y0, y1, y2, y3, y4, y5, y6, y7;\n\t"
      ".reg .b8 q0, q1, q2, q3, r0, r1, r2, r3;\n\t"
      "mov.b64 ip, {%5, %5};\n\t"
      "mov.b64 p0, {%6, %7};\n\t"
      "mov.b64 p1, {%8, %9};\n\t"
      "mov.b64 p2, {%10, %11};\n\t"
      "mov.b64 p3, {%12, %13};\n\t"
      "mul.rn.f32x2 p0, p0, ip;\n\t"
      "mul.rn.f32x2 p1, p1, ip;\n\t"
      "mul.rn.f32x2 p2, p2, ip;\n\t"
      "mul.rn.f32x2 p3, p3, ip;\n\t"
      "mov.b64 {y0, y1}, p0;\n\t"
      "mov.b64 {y2, y3}, p1;\n\t"
      "mov.b64 {y4, y5}, p2;\n\t"
      "mov.b64 {y6, y7}, p3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 q0, y1, y0;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 q1, y3, y2;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 q2, y5, y4;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 q3, y7, y6;\n\t"
      "mov.b32 %0, {q0, q1, q2, q3};\n\t"
      "mov.b32 {r0, r1, r2, r3}, %0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, r0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, r1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, r2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %4, r3;\n\t"
      "}"
      : "=r"(code), "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
      : "f"(inv), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]),
        "f"(x[7]));
  return code;
}

// Codes of a block without the decoded values (standard NVFP4).
__device__ __forceinline__ uint32_t codes8(const float* x, float inv) {
  uint32_t code;
  asm("{\n\t"
      ".reg .b64 ip, p0, p1, p2, p3;\n\t"
      ".reg .f32 y0, y1, y2, y3, y4, y5, y6, y7;\n\t"
      ".reg .b8 q0, q1, q2, q3;\n\t"
      "mov.b64 ip, {%1, %1};\n\t"
      "mov.b64 p0, {%2, %3};\n\t"
      "mov.b64 p1, {%4, %5};\n\t"
      "mov.b64 p2, {%6, %7};\n\t"
      "mov.b64 p3, {%8, %9};\n\t"
      "mul.rn.f32x2 p0, p0, ip;\n\t"
      "mul.rn.f32x2 p1, p1, ip;\n\t"
      "mul.rn.f32x2 p2, p2, ip;\n\t"
      "mul.rn.f32x2 p3, p3, ip;\n\t"
      "mov.b64 {y0, y1}, p0;\n\t"
      "mov.b64 {y2, y3}, p1;\n\t"
      "mov.b64 {y4, y5}, p2;\n\t"
      "mov.b64 {y6, y7}, p3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 q0, y1, y0;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 q1, y3, y2;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 q2, y5, y4;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 q3, y7, y6;\n\t"
      "mov.b32 %0, {q0, q1, q2, q3};\n\t"
      "}"
      : "=r"(code)
      : "f"(inv), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]),
        "f"(x[7]));
  return code;
}

// One candidate with the binary32 error: codes c0, c1 and the error sum. The terms and the
// tree are scalar: binary32 operations split across the two FMA pipes, which measured
// faster here than the packed two-lane forms.
template <bool MSE>
__device__ __forceinline__ float candidate_f32(const float x[16], float inv, uint32_t S2,
                                               float neg_gs, uint32_t& c0, uint32_t& c1) {
  uint32_t v[8];
  c0 = encode8(x, inv, v);
  c1 = encode8(x + 8, inv, v + 4);
  float t[16];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t w = hmul2_rn(v[k], S2);  // e2m1 * S, exact
    // each element error is rounded once: a fused multiply-add
    const float e0 = __fmaf_rn(f32_from_f16_lo(w), neg_gs, x[2 * k]);
    const float e1 = __fmaf_rn(f32_from_f16_hi(w), neg_gs, x[2 * k + 1]);
    t[2 * k] = MSE ? __fmul_rn(e0, e0) : fabsf(e0);
    t[2 * k + 1] = MSE ? __fmul_rn(e1, e1) : fabsf(e1);
  }
#pragma unroll
  for (int h = 8; h >= 1; h /= 2) {
#pragma unroll
    for (int i = 0; i < h; ++i) t[i] = __fadd_rn(t[i], t[i + h]);
  }
  return t[0];
}

// One candidate with the binary16 error: codes c0, c1 and the error sum (as a float).
// S2 = (S, S) and neg_gh2 = (-g_h, -g_h) as half2.
template <bool MSE>
__device__ __forceinline__ float candidate_f16(const float x[16], const uint32_t xh[8], float inv,
                                               uint32_t S2, uint32_t neg_gh2, uint32_t nzh2,
                                               uint32_t& c0, uint32_t& c1) {
  uint32_t t[8];
  c0 = encode8(x, inv, t);
  c1 = encode8(x + 8, inv, t + 4);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t w = hmul2_rn(t[k], S2);  // e2m1 * S, exact
    const uint32_t e = hfma2_rn(w, neg_gh2, xh[k]);  // x_h - w * g_h, one rounding
    if (MSE) {
      t[k] = hsq2_rn(e, nzh2);
    } else {
      asm("abs.f16x2 %0, %1;" : "=r"(t[k]) : "r"(e));
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) t[k] = hadd2_rn(t[k], t[k + 4]);
  t[0] = hadd2_rn(t[0], t[2]);
  t[1] = hadd2_rn(t[1], t[3]);
  t[0] = hadd2_rn(t[0], t[1]);
  const __half s = __hadd_rn(__ushort_as_half(static_cast<unsigned short>(t[0] & 0xFFFFu)),
                             __ushort_as_half(static_cast<unsigned short>(t[0] >> 16)));
  return __half2float(s);
}

// Per-CTA tables indexed by scale byte. The binary32-error recipes read both of a
// candidate's constants with one 8-byte shared-memory load (measured faster there; the
// other recipes measured faster with separate arrays).
union Tables {
  struct {
    float inv[2][256];         // 1 / (S * gs) per tensor
    uint32_t S2[256];          // (S, S) as half2 (binary16-error recipes)
  } split;                     // standard NVFP4 and the binary16-error recipes
  uint2 pair[2][256];          // binary32-error recipes: (bits of 1 / (S * gs), (S, S) as half2)
};

struct BlockOut {
  uint32_t c0, c1, s;
};

template <bool BF16, int MODE, bool EXACT = false>
__device__ __forceinline__ BlockOut quantize_block(const U32x8& in, const TensorConsts& tc,
                                                   const Tables& tab, int kv, float cap_a,
                                                   uint32_t nz) {
  float x[16];
  unpack16<BF16>(in, x);
  // max |x|: the standard and binary16-error recipes chain three-input maxima of
  // magnitudes (8 instead of 16, off the busy integer pipe's share); the binary32-error
  // recipes fold |x| into two-input maxima
  float amax;
  if (MODE == 0 || MODE >= 3) {
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(amax) : "f"(x[0]), "f"(x[1]), "f"(x[2]));
#pragma unroll
    for (int i = 3; i < 15; i += 2)
      asm("max.abs.f32 %0, %0, %1, %2;" : "+f"(amax) : "f"(x[i]), "f"(x[i + 1]));
    amax = fmaxf(amax, fabsf(x[15]));
  } else {
    amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
  }
  const float ra = fminf(quotient<EXACT>(amax, tc.g6, tc.r6, tc.exact_rcp), cap_a);
  BlockOut r;
  if (MODE == 0) {
    r.s = e4m3x2_from_f32(ra, 0.0f) & 0xFFu;
    const float inv = tab.split.inv[kv][r.s];
    r.c0 = codes8(x, inv);
    r.c1 = codes8(x + 8, inv);
    return r;
  }
  const float rb = fminf(quotient<EXACT>(amax, tc.g4, tc.r4, tc.exact_rcp), 448.0f);
  const uint32_t sab = e4m3x2_from_f32(ra, rb);
  // sb = sab >> 8 and sa = sab & 0xFF as multiplies (FMA pipe)
  uint32_t sb;
  asm("mul.hi.u32 %0, %1, 16777216;" : "=r"(sb) : "r"(sab));
  const uint32_t sa = sab - sb * 256u;
  uint32_t a0, a1, b0, b1;
  float ea, eb;
  if (MODE == 1 || MODE == 2) {
    const uint2 ta = tab.pair[kv][sa], tb = tab.pair[kv][sb];
    ea = candidate_f32<MODE == 2>(x, __uint_as_float(ta.x), ta.y, -tc.gs, a0, a1);
    eb = candidate_f32<MODE == 2>(x, __uint_as_float(tb.x), tb.y, -tc.gs, b0, b1);
  } else {
    uint32_t xh[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) xh[k] = BF16 ? f16x2_from_f32(x[2 * k], x[2 * k + 1]) : in.w[k];
    const uint32_t nzh2 = (nz >> 16) | nz;  // binary16 -0 in both halves
    ea = candidate_f16<MODE == 4>(x, xh, tab.split.inv[kv][sa], tab.split.S2[sa], tc.neg_gh2,
                                  nzh2, a0, a1);
    eb = candidate_f16<MODE == 4>(x, xh, tab.split.inv[kv][sb], tab.split.S2[sb], tc.neg_gh2,
                                  nzh2, b0, b1);
  }
  const bool take_b = eb < ea;
  r.c0 = take_b ? b0 : a0;
  r.c1 = take_b ? b1 : a1;
  r.s = take_b ? sb : sa;
  return r;
}

// The two global scales: from the arguments, or from device memory when given there.
// Returns false (and reports it) when a device-held scale is not positive finite.
__device__ __forceinline__ bool load_scales(const AppendArgs& a, float gs[2]) {
  gs[0] = a.gs[0];
  gs[1] = a.gs[1];
  if (a.gs_dev[0] != nullptr) {
    gs[0] = __ldg(a.gs_dev[0]);
    gs[1] = __ldg(a.gs_dev[1]);
    const bool ok = gs[0] > 0.0f && gs[0] <= FLT_MAX && gs[1] > 0.0f && gs[1] <= FLT_MAX;
    if (!ok) {
      if (threadIdx.x == 0 && blockIdx.x == 0) flag(a.status, NVFP4_DEV_BAD_SCALE);
      return false;
    }
  }
  return true;
}

// Fill the per-CTA tables for both tensors' global scales; ends with __syncthreads().
template <int MODE>
__device__ __forceinline__ void fill_tables(Tables& tab, const float gs[2]) {
  for (int s = threadIdx.x; s < 256; s += blockDim.x) {
    const uint32_t S2 = f16x2_from_e4m3x2(static_cast<uint32_t>(s) * 0x0101u);
    const float S = f32_from_f16_lo(S2);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const float den = __fmul_rn(S, gs[kv]);
      const float inv = den == 0.0f ? 0.0f : fminf(__frcp_rn(den), FLT_MAX);
      if (MODE == 1 || MODE == 2) {
        tab.pair[kv][s] = make_uint2(__float_as_uint(inv), S2);
      } else {
        tab.split.inv[kv][s] = inv;
        if (kv == 0) tab.split.S2[s] = S2;
      }
    }
  }
  __syncthreads();
}

// Destination of appended row i: request batch_indices[i], logical position positions[i],
// page kv_indices[kv_indptr[b] + pos / page_size], slot pos % page_size. Rows outside the
// described space or with a page outside a pool are reported and marked invalid.
struct RowMeta {
  int32_t page;   // physical page (valid only with flags bit 0 / bit 1)
  int32_t slot;   // slot inside the page
  int32_t flags;  // bit 0: K page valid, bit 1: V page valid
  int32_t pad;
};

__device__ __forceinline__ RowMeta resolve_row(const AppendArgs& a, int64_t i) {
  RowMeta m{0, 0, 0, 0};
  const int32_t b = __ldg(a.batch_indices + i);
  const int32_t pos = __ldg(a.positions + i);
  if (b < 0 || b >= a.batch_size) {
    flag(a.status, NVFP4_DEV_BAD_BATCH);
    return m;
  }
  const int64_t start = __ldg(a.kv_indptr + b);
  const int64_t npages = static_cast<int64_t>(__ldg(a.kv_indptr + b + 1)) - start;
  const int64_t lp = pos >= 0 ? div_q(pos, a.div_ps) : -1;
  bool ok = pos >= 0 && lp < npages && start >= 0 && start + lp < a.num_kv_indices;
  if (ok && a.kv_last_page_len) ok = pos < (npages - 1) * a.ps + __ldg(a.kv_last_page_len + b);
  if (!ok) {
    flag(a.status, NVFP4_DEV_BAD_POSITION);
    return m;
  }
  const int64_t page = __ldg(a.kv_indices + start + lp);
  m.page = static_cast<int32_t>(page);
  m.slot = static_cast<int32_t>(pos - lp * a.ps);
  const bool kok = page >= 0 && page < a.kc.num_pages;
  const bool vok = page >= 0 && page < a.vc.num_pages;
  if (!kok || !vok) flag(a.status, NVFP4_DEV_BAD_PAGE);
  m.flags = (kok ? 1 : 0) | (vok ? 2 : 0);
  return m;
}

}  // namespace nvfp4
