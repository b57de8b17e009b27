// prefill_paged.cu -- launches of the prefill of new tokens over a paged cache (the
// kernel: prefill_kernel.cuh with PAGED).
//
// Packed varlen batches only.  The query heads of a KV head share a tile's rows
// (pack), so a chunk of a few tokens fills more of a tile and each K/V row is gathered
// once per group of heads.
#include "prefill_kernel.cuh"

namespace attn {
namespace {

template <int D, bool WIN, bool SPLIT, bool H>
cudaError_t launch_t(const PrefillArgs& a, cudaStream_t stream) {
  using C = PrefillCfg<D, H>;
  auto kern = fmha_fwd_kernel<D, WIN, SPLIT, H, true>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  const int G = a.pack, TR = kPrefillTileM / G * G;
  const long long rows = (long long)a.Sq * G;
  const long long n_blocks_q = (rows + C::NQ * TR - 1) / (C::NQ * TR);
  const int n_splits = SPLIT ? a.n_splits : 1;
  const long long units = n_blocks_q * (a.Hq / G) * a.B * n_splits;
  if (units > 0x7FFFFFFFLL || rows > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  kern<<<(unsigned)units, C::kThreads, C::kSmemBytes, stream>>>(
      a.tm_q, a.tm_k, a.tm_v, a.tm_o, a.o_tma, a.o, a.lse, a.Hq, a.Hkv, a.Sq, a.Skv, a.causal, a.o_bf16, a.scale,
      (a.Hq / G) * a.B, a.err, a.cu_q, a.kv_lens, a.total_q, a.window, a.n_sink, G, n_splits, a.split_min,
      a.part_o, a.part_lse, 0, 0, a.kv);
  return cudaGetLastError();
}

template <int D, bool H>
cudaError_t launch_d(const PrefillArgs& a, cudaStream_t stream) {
  if constexpr (!H) {
    if (a.window > 0) return launch_t<D, true, false, false>(a, stream);
  }
  return a.n_splits > 1 ? launch_t<D, false, true, H>(a, stream) : launch_t<D, false, false, H>(a, stream);
}

}  // namespace

cudaError_t launch_prefill_paged(const PrefillArgs& a, cudaStream_t stream) {
  switch (a.d) {
    case 64: return a.halves ? launch_d<64, true>(a, stream) : launch_d<64, false>(a, stream);
    case 128: return a.halves ? launch_d<128, true>(a, stream) : launch_d<128, false>(a, stream);
    case 256: return launch_d<256, false>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
