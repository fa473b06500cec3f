// softmax.cuh -- what the attention kernels share: the arithmetic of weights, the cut of a launch's work into
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
