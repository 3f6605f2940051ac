// attn_scored_rot4.cu — attn_scored and attn_tree over caches with 4 bits per V
// code and the block-diagonal rotation; kernels in attn_scored_kernel.cuh.
#include "attn_scored_kernel.cuh"

namespace ckv {

cudaError_t launch_scored_rot4(const ScoredArgs& a, cudaStream_t stream) {
  return launch_scored_bits<4, 1>(a, stream);
}

}  // namespace ckv
