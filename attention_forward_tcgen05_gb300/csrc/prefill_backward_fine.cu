// prefill_backward_fine.cu -- prefill_backward.cuh's kernels for calls of few pairs of rows and keys, with P
// and dS as two bf16 terms.  Where few terms make up a gradient its error is not the usual mean of
// their roundings but may be that of one, up to 2^-8, as much again as the gradient's own.  Such a call is
// bound by its launches and one tile's chain, under which the further products are done.
#include "prefill_backward.cuh"

namespace attn {

int backward_fine_tile_rows(int d, bool dkdv) { return tile_rows<true>(d, dkdv); }

cudaError_t launch_backward_fine(const BackwardArgs& a, cudaStream_t stream) { return launch_all<true>(a, stream); }

}  // namespace attn
