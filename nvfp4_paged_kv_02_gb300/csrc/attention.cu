// attention.cu -- attention of one new token per request: the choice of a kernel (attention.cuh), and its plain kind.
#include "attention.cuh"

namespace nvfp4 {
namespace {

// Query heads that one pass over the cache serves: eight, or sixteen where the accumulators of
// sixteen fit the registers (D <= 128).
int eights_of(int G, int D) { return G > 8 && D <= 128 ? 2 : 1; }

}  // namespace

int64_t attention_workspace_bytes(int32_t Hq, int32_t H, int32_t D) {
  const int64_t nw = (D + 63) / 64, heads = 8 * eights_of(Hq / H, D);
  const int64_t slot = heads * (64 * nw + 2) * 4;
  return NVFP4_COUNTER_BYTES + 2 * slot * kMaxCtasPerSm * sm_count();
}

nvfp4_status launch_attention(AttentionArgs a, cudaStream_t stream) {
  const int nt = a.qo_indptr ? a.most_rows / 8 : eights_of(a.G, a.D), nw = (a.D + 63) / 64;
  a.chunks = a.qo_indptr ? 1 : (a.G + 8 * nt - 1) / (8 * nt);
  a.chunk_heads = (a.G + a.chunks - 1) / a.chunks;
  const int64_t pool = a.kc.num_pages < a.vc.num_pages ? a.kc.num_pages : a.vc.num_pages;
  a.pool_pages = static_cast<uint32_t>(pool);
  const int64_t strides[4] = {a.kc.data_page_stride, a.vc.data_page_stride, a.kc.sf_page_stride, a.vc.sf_page_stride};
  for (int64_t s : strides)
    if (s > static_cast<int64_t>(UINT32_MAX)) return fail(NVFP4_ERR_UNSUPPORTED, "nvfp4_paged_attention_decode: a page stride above 4 GiB");
  a.k_stride = static_cast<uint32_t>(strides[0]);
  a.v_stride = static_cast<uint32_t>(strides[1]);
  a.k_sf_stride = static_cast<uint32_t>(strides[2]);
  a.v_sf_stride = static_cast<uint32_t>(strides[3]);
  // one offset serves K and V, and 32 bits hold it
  a.compact = strides[0] == strides[1] && strides[2] == strides[3] && strides[2] % 4 == 0 &&
              pool * (strides[0] / 16) <= static_cast<int64_t>(UINT32_MAX) &&
              pool * (strides[2] / 4) <= static_cast<int64_t>(UINT32_MAX);
  if (sm_count() * kMaxCtasPerSm * 4 > NVFP4_COUNTER_BYTES)
    return fail(NVFP4_ERR_UNSUPPORTED, "nvfp4_paged_attention_decode: more SMs than counters");
  // scale rows are copied 4 nw bytes at a time (nw = 3: 4), aligned to that
  auto scales_aligned = [&](uintptr_t n) {
    return reinterpret_cast<uintptr_t>(a.kc.sf) % n == 0 && reinterpret_cast<uintptr_t>(a.vc.sf) % n == 0 &&
           a.kc.sf_page_stride % n == 0 && a.vc.sf_page_stride % n == 0;
  };
  const bool full = a.D % 64 == 0 && scales_aligned(nw == 3 ? 4 : 4 * nw);
  if (a.qo_indptr) return launch_attention_tokens(a, nw, nt, full, stream);
  if (a.sink > 0) return launch_attention_sinks(a, nw, nt, full, stream);
  return launch_kind<kPlain>(a, nw, nt, full, stream);
}

}  // namespace nvfp4
