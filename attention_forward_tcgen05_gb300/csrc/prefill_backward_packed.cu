// prefill_backward_packed.cu -- prefill_backward.cuh's kernels for packed batches that may hold sequences of both
// forms, in one launch: as a launch each, one short sequence beside four of 1000 rows (32 heads of 128) made a call
// 37 us longer, so 3, and one without any 5.
#include "prefill_backward.cuh"

namespace attn {

cudaError_t launch_backward_packed(const BackwardArgs& a, cudaStream_t stream) {
  return launch_all<true, true, true>(a, stream);
}

}  // namespace attn
