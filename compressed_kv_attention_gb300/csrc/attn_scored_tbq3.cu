// attn_scored_tbq3.cu — attn_scored and attn_tree over caches with 3 bits per V
// code; kernels in attn_scored_kernel.cuh.
#include "attn_scored_kernel.cuh"

namespace ckv {

cudaError_t launch_scored_tbq3(const ScoredArgs& a, cudaStream_t stream) {
  return launch_scored_bits<3, 0>(a, stream);
}

}  // namespace ckv
