// prefill_backward_fine.cu -- prefill_backward.cuh's kernels for calls whose sequences all take P and dS as two
// bf16 terms.
#include "prefill_backward.cuh"

namespace attn {

cudaError_t launch_backward_fine(const BackwardArgs& a, cudaStream_t stream) {
  return a.cu_q ? launch_all<true, false, true>(a, stream) : launch_all<false, false, true>(a, stream);
}

}  // namespace attn
