// attention_tokens.cu -- the kernel of attention.cuh of several query tokens of each request.
#include "attention.cuh"

namespace nvfp4 {

nvfp4_status launch_attention_tokens(const AttentionArgs& a, int nw, int nt, bool full, cudaStream_t stream) {
  return launch_kind<kTokens>(a, nw, nt, full, stream);
}

}  // namespace nvfp4
