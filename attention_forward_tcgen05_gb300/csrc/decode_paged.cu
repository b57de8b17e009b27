// decode_paged.cu -- one-token GQA decode over a paged cache (decode_paged.cuh).
#include "decode_paged.cuh"

namespace attn {

int decode_paged_slots(int d, int G, int sms) {
  return sms * decode_paged_ctas(d, G <= 8 ? 1 : 2);
}

cudaError_t launch_decode_paged(const DecodeArgs& a, cudaStream_t stream) {
  return launch_paged_decode<false>(a, stream);
}

}  // namespace attn
