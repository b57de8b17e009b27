// prefill_backward.cu -- prefill_backward.cuh's first kernel, and its kernels for fixed-length calls with P and
// dS rounded to bf16.
#include "prefill_backward.cuh"

namespace attn {

cudaError_t launch_backward_prep(const BackwardArgs& a, bool any, cudaStream_t stream) {
  return a.d == 64 ? launch_prep<64>(a, any, stream) : launch_prep<128>(a, any, stream);
}

cudaError_t launch_backward(const BackwardArgs& a, cudaStream_t stream) { return launch_all<false, true, false>(a, stream); }

}  // namespace attn
