// prefill_paged_f32.cu -- prefill over a paged cache with fp32 outputs.
#include "prefill_paged.cuh"

namespace attn {

cudaError_t launch_prefill_paged_f32(const PrefillArgs& a, cudaStream_t stream) {
  return launch_prefill_paged_t<true>(a, stream);
}

}  // namespace attn
