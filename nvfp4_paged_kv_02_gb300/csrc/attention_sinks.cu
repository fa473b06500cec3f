// attention_sinks.cu -- the kernel of attention.cuh with first tokens that stay beside a window.
#include "attention.cuh"

namespace nvfp4 {

nvfp4_status launch_attention_sinks(const AttentionArgs& a, int nw, int nt, bool full, cudaStream_t stream) {
  return launch_kind<kSinks>(a, nw, nt, full, stream);
}

}  // namespace nvfp4
