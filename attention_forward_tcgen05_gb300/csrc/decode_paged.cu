// decode_paged.cu -- launches of the one-token decode over a paged cache (the kernel:
// decode_kernel.cuh with PAGED).
#include "decode_kernel.cuh"

namespace attn {

cudaError_t launch_decode_paged(const DecodeArgs& a, cudaStream_t stream) {
  switch (a.d) {
    case 64: return launch_decode_g<64, true>(a, stream);
    case 128: return launch_decode_g<128, true>(a, stream);
    case 256: return launch_decode_g<256, true>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
