// decode.cu -- launches of the one-token decode over a dense cache, and of the merge
// (the kernel: decode_kernel.cuh; over a paged cache: decode_paged.cu).
#include "decode_kernel.cuh"

namespace attn {
namespace {

template <int D>
__global__ void __launch_bounds__(128)
    merge_kernel(const float* __restrict__ part_o, const float* __restrict__ part_lse, void* o,
                 float* __restrict__ lse, int rows, int n_splits, int o_bf16, int heads,
                 const int* __restrict__ cu_q, int n_seq) {
  const int row = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= rows) return;
  // rows of tokens outside the packed batch have no partials and stay as they are
  if (cu_q != nullptr && (row / heads < cu_q[0] || row / heads >= cu_q[n_seq])) return;
  // heads > 0: lse [heads][rows / heads] (one row of it per head), else lse [rows]
  const size_t lse_row = heads > 0 ? (size_t)(row % heads) * (rows / heads) + row / heads : (size_t)row;
  merge_row<D>(part_o, part_lse, o, lse, (size_t)row, lse_row, n_splits, o_bf16, threadIdx.x & 31);
}

}  // namespace

cudaError_t launch_decode_split(const DecodeArgs& a, cudaStream_t stream) {
  switch (a.d) {
    case 64: return launch_decode_g<64, false>(a, stream);
    case 128: return launch_decode_g<128, false>(a, stream);
    case 256: return launch_decode_g<256, false>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_merge(const MergeArgs& a, cudaStream_t stream) {
  const int rows = a.B * a.Hq;
  const dim3 grid((rows + 3) / 4);
  const int heads = a.lse_by_head ? a.Hq : 0;
  switch (a.d) {
    case 64:
      merge_kernel<64><<<grid, 128, 0, stream>>>(a.part_o, a.part_lse, a.o, a.lse, rows, a.n_splits, a.o_bf16, heads,
                                            a.cu_q, a.n_seq);
      break;
    case 128:
      merge_kernel<128><<<grid, 128, 0, stream>>>(a.part_o, a.part_lse, a.o, a.lse, rows, a.n_splits, a.o_bf16, heads,
                                            a.cu_q, a.n_seq);
      break;
    case 256:
      merge_kernel<256><<<grid, 128, 0, stream>>>(a.part_o, a.part_lse, a.o, a.lse, rows, a.n_splits, a.o_bf16, heads,
                                            a.cu_q, a.n_seq);
      break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace attn
