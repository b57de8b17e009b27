// prefill_backward.cu -- prefill_backward.cuh's kernels with P and dS rounded to bf16.
#include "prefill_backward.cuh"

namespace attn {

int backward_tile_rows(int d, bool dkdv) { return tile_rows<false>(d, dkdv); }

cudaError_t launch_backward(const BackwardArgs& a, cudaStream_t stream) { return launch_all<false>(a, stream); }

}  // namespace attn
