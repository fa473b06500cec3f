// softmax.cuh -- what the attention kernels share: asynchronous copies, the arithmetic of weights, the cut of a launch's work into
// equal runs, and a block of the cache as binary16.
#pragma once

#include <cstdint>

#include "device.cuh"

namespace nvfp4 {

// A weight is p = 2^(x log2 e - m + kWeightBias), where m follows the maximum only when that is more than kSlack
// above it: p <= 2^15, which binary16 holds.
constexpr float kWeightBias = 8.0f;
constexpr float kSlack = 7.0f;
constexpr float kLog2e = 1.4426950408889634f;

// Asynchronous copies to shared memory; not live: nothing is read, the destination is zero-filled.
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool live) {
  const int n = live ? BYTES : 0;  // 0: nothing is read, the destination is zero-filled
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(n), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// c tanh(x / c) by 1 - 2 / (e^(2x/c) + 1): absolute error a few 2^-24 of c.
__device__ __forceinline__ float soft_capped(float x, float cap) {
  const float e = ex2(x / cap * (2.0f * kLog2e));
  return cap * (1.0f - 2.0f / (e + 1.0f));
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// (x0, x1) = (x0, x1) * a + b, and (s0, s1) += (x0, x1), in one instruction each.
__device__ __forceinline__ void fma2(float& x0, float& x1, float a, float b) {
  asm("{\n\t.reg .b64 x, a, b;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 a, {%2, %2};\n\tmov.b64 b, {%3, %3};\n\t"
      "fma.rn.f32x2 x, x, a, b;\n\tmov.b64 {%0, %1}, x;\n\t}" : "+f"(x0), "+f"(x1) : "f"(a), "f"(b));
}
__device__ __forceinline__ void add2(float& s0, float& s1, float x0, float x1) {
  asm("{\n\t.reg .b64 s, x;\n\tmov.b64 s, {%0, %1};\n\tmov.b64 x, {%2, %3};\n\tadd.rn.f32x2 s, s, x;\n\t"
      "mov.b64 {%0, %1}, s;\n\t}" : "+f"(s0), "+f"(s1) : "f"(x0), "f"(x1));
}

// a / b, by 32-bit division where both are small.
__device__ __forceinline__ int64_t quotient64(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// The cut of `total` places into n runs: the first `more` runs have per + 1 places.
struct Cut {
  int64_t per, more;
  __device__ __forceinline__ int64_t begin(int64_t run) const { return run * per + min(run, more); }
  __device__ __forceinline__ int64_t run_of(int64_t place) const {
    const int64_t edge = more * (per + 1);
    return place < edge ? quotient64(place, per + 1) : more + quotient64(place - edge, per);
  }
};

// The codes of this lane's block of 16 elements, scaled: eight pairs.
__device__ __forceinline__ void decode16(uint32_t w0, uint32_t w1, uint32_t S2, uint32_t v[8]) {
  f16x2x4_from_e2m1x8(w0, v[0], v[1], v[2], v[3]);
  f16x2x4_from_e2m1x8(w1, v[4], v[5], v[6], v[7]);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = hmul2_rn(v[i], S2);
}

__device__ __forceinline__ uint32_t low_twice(uint32_t v) {
  uint32_t d;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {l, l};\n\t}" : "=r"(d) : "r"(v));
  return d;
}
__device__ __forceinline__ uint32_t high_twice(uint32_t v) {
  uint32_t d;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {h, h};\n\t}" : "=r"(d) : "r"(v));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

}  // namespace nvfp4
