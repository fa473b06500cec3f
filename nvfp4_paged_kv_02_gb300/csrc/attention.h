// attention.h -- arguments of the operators that read a paged NVFP4 cache with a query:
// page bounds, page selection, attention of one new token per request and of several.
#pragma once

#include "attention_sizes.h"
#include "internal.h"

namespace nvfp4 {

// Largest head_dim of the attention kernels (their accumulators are held in registers).
constexpr int kAttnMaxHeadDim = 256;

struct AttentionArgs {
  const uint8_t* q;
  int64_t q_row_bytes;
  nvfp4_paged_cache kc, vc;
  int32_t ps, Hq, H, G, D, layout, B;
  int32_t bf16, table64;
  Div div_ps;
  const void* block_tables;
  int64_t max_pages;
  const int32_t* seq_lens;
  const int32_t* selected;      // [B, H, max_selected] logical pages, or null: all of them
  const int32_t* num_selected;  // [B, H]
  int32_t max_selected;
  const float* k_scale;
  const float* v_scale;
  float sm_scale, soft_cap;
  int32_t window_left, sink;  // with a window: the first `sink` positions too
  uint8_t* out;
  float* lse;  // may be null
  int32_t* status;
  void* workspace;
  // several query tokens of each request, in requests of at most most_rows (8 or 16) rows of a KV head (attention of
  // the last tokens): rows of query by qo_indptr; or null
  const int32_t* qo_indptr;
  int64_t nnz;
  int32_t causal, most_rows;
  // set at launch
  int32_t chunks, chunk_heads;  // passes over a KV head's query heads, and the heads of one
  uint32_t pool_pages;          // pages that both caches have
  uint32_t k_stride, v_stride, k_sf_stride, v_sf_stride;  // page strides, bytes
  int32_t compact;
  int32_t groups, log2_group;  // entries of the scan, and the requests to one
};
// Device memory that a launch needs, whatever the lengths.
int64_t attention_workspace_bytes(int32_t Hq, int32_t H, int32_t D);
nvfp4_status launch_attention(AttentionArgs a, cudaStream_t stream);
// its kinds, in translation units of their own (nw: head_dim / 64, rounded up; nt: eights of rows)
nvfp4_status launch_attention_sinks(const AttentionArgs& a, int nw, int nt, bool full, cudaStream_t stream);
nvfp4_status launch_attention_tokens(const AttentionArgs& a, int nw, int nt, bool full, cudaStream_t stream);

struct PrefillArgs {
  const uint8_t* q;
  int64_t q_row_bytes, nnz;
  nvfp4_paged_cache kc, vc;
  int32_t ps, Hq, H, G, D, layout, B;
  int32_t bf16, table64, causal;
  Div div_ps, div_g;
  const int32_t* qo_indptr;  // [B + 1]
  const void* block_tables;
  int64_t max_pages;
  const int32_t* seq_lens;
  const float* k_scale;
  const float* v_scale;
  float sm_scale, soft_cap;
  int32_t window_left, sink;
  uint8_t* out;
  float* lse;  // may be null
  int32_t* status;
  void* workspace;
  // set at launch
  int64_t pool_pages, parts_offset;
  int32_t few_rows;  // requests of so few rows are another kernel's
  uint32_t k_stride, v_stride, k_sf_stride, v_sf_stride;  // page strides, bytes
  PipeTest pipe;
};
// In the workspace, for each run: the segment that it begins and others continue, up to run `last` (-1: none).
struct PrefillCut {
  int32_t b, t, h, last;
};
int64_t prefill_workspace_bytes(int32_t D);
nvfp4_status launch_prefill(PrefillArgs a, cudaStream_t stream);

struct BoundsArgs {
  nvfp4_paged_cache kc;
  int32_t ps, H, D, layout, B, table64;
  Div div_ps;
  const void* block_tables;
  int64_t max_pages;
  const int32_t* seq_lens;
  const int32_t* first_positions;  // may be null: 0
  uint16_t* bounds;
  int32_t* status;
  // set at launch: a CTA's shape, or the ring's
  int32_t pages, tile, slices, stages;
  uint32_t code_bytes, scale_bytes, stage_bytes;
  Div div_nb, div_columns;
  PipeTest pipe;
};
nvfp4_status launch_page_key_bounds(BoundsArgs a, cudaStream_t stream);

struct SelectArgs {
  const uint8_t* q;
  int64_t q_row_bytes;
  int32_t bf16, Hq, H, G, D, ps, B, table64;
  const uint16_t* bounds;
  int64_t num_pages;
  const void* block_tables;
  int64_t max_pages;
  const int32_t* seq_lens;
  int32_t k, sink, recent;
  int32_t* selected;
  int32_t* num_selected;
  uint32_t* scores;  // workspace: [B, H, pitch]
  int32_t* status;
  int64_t pitch;  // set at launch
};
int64_t select_workspace_bytes(int32_t B, int32_t H, int64_t max_pages);
nvfp4_status launch_select_pages(SelectArgs a, cudaStream_t stream);

}  // namespace nvfp4
