// decode_window.cu -- one-token GQA decode over the last keys of a sequence and its first ones
// (decode_paged.cuh's kernel over the list of admitted keys), paged or dense.
//
// Of a sequence of L keys the token admits [max(0, L - window), L) and [0, n_sink): at most
// window + n_sink rows of K and V are read whatever L, and HBM bounds large batches as it does
// decode_paged.cu.  Masking in that kernel instead would read all L.
#include "decode_paged.cuh"

namespace attn {

cudaError_t launch_decode_window(const DecodeArgs& a, cudaStream_t stream) {
  return launch_paged_decode<true>(a, stream);
}

}  // namespace attn
