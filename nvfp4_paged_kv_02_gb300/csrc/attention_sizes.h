// attention_sizes.h -- what the kernel of single tokens (attention.cuh) can count, and which prompts' rows go to it.
// Plain arithmetic of the host, which a test compiles by itself.
#pragma once

#include <cstdint>

namespace nvfp4 {

// A CTA of that kernel counts its places (units of 32 positions and nine more of each list) in 32 bits. `lists`: of a
// launch, each of up to `reach` positions; at most 2^38 places, so 2^31 for a CTA where there are 128 or more.
inline bool places_countable(int64_t lists, int64_t reach) {
  return lists <= 0 || reach / 32 + 10 <= (int64_t(1) << 38) / lists;
}

// Requests of at most so many rows (8 or 16) of a KV head go to that kernel, which reads a cache faster than rows of 128
// can be made of it; 0: none do. `rows`: of all requests (query tokens times query heads of a KV head). They go where
// requests have few rows on average (drafts, or single tokens among them): 64 requests of four tokens, four query heads
// to a KV head, 105 K positions: 117 us without, 83 with both launches, in a CUDA graph; 90 in calls one after the other.
// Tables of up to 1024 positions stay: the second launch costs more (five requests of 1 to 9 tokens over up to 86
// positions: 14 us, with both 27). So does what that kernel could not count. A batch of single tokens beside long chunks
// has many rows on average and stays too.
inline int32_t few_rows_of(int64_t rows, int32_t head_dim, int32_t batch, int32_t kv_heads, int64_t reach) {
  const int64_t sixteen = head_dim <= 128 ? 16 : 8;
  if (rows > sixteen * batch || reach <= 1024 || !places_countable(static_cast<int64_t>(batch) * kv_heads, reach)) return 0;
  return sixteen == 16 && rows > 8 * static_cast<int64_t>(batch) ? 16 : 8;
}

}  // namespace nvfp4
