// prefill_paged.cu -- prefill over a paged cache with bf16 outputs.
#include "prefill_paged.cuh"

namespace attn {

cudaError_t launch_prefill_paged(const PrefillArgs& a, cudaStream_t stream) {
  return launch_prefill_paged_t<false>(a, stream);
}

}  // namespace attn
