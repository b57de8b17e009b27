// prefill_paged.cuh -- launches of the prefill of new tokens over a paged cache (the
// kernel: prefill_kernel.cuh with PAGED), for bf16 outputs (prefill_paged.cu) and fp32 ones
// (prefill_paged_f32.cu).
//
// Packed varlen batches only.  The query heads of a KV head share a tile's rows
// (pack), so a chunk of a few tokens fills more of a tile and each K/V row is gathered
// once per group of heads.
//
// What bounds it and what was measured (GB300, device time; floor in brackets).  Steps of 256
// rows x 128 keys at d = 128 take 1.75 us.  In a 2,000-row chunk of a 32k-key prompt (656 us and
// a merge; 675 [469] together, 707 a call in a long series, where the power cap lowers the
// clock) the tensor pipe is active 62 % of the time, issue slots 45 %, the exponential unit 31 %:
// no unit is full, and the chain of a tile (S from TMEM, maximum, exponentials, P to TMEM, the
// next product) is the time.  One head per tile over a dense cache takes 808 us: a group's keys
// are then read once per head.  Tensor copies against gathers:
// 164 against 248 us for eight ragged chunks (145 GFLOP) from pages of 16.  A unit's start and
// end take 7 us; with 3.5 units an SM that is a sixth of the eight chunks' 145 us [78].  fp32
// outputs: 199 us, 5e-6 of O off against 1.6e-3 with P in one term.
#pragma once
#include "prefill_kernel.cuh"

namespace attn {
namespace {

template <int D, bool WIN, bool SPLIT, bool H, bool FINE>
cudaError_t launch_t(const PrefillArgs& a, cudaStream_t stream) {
  using C = PrefillCfg<D, H>;
  auto kern = fmha_fwd_kernel<D, WIN, SPLIT, H, true, FINE>;
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

template <int D, bool H, bool FINE>
cudaError_t launch_d(const PrefillArgs& a, cudaStream_t stream) {
  if constexpr (!H) {
    if (a.window > 0) return launch_t<D, true, false, false, FINE>(a, stream);
  }
  return a.n_splits > 1 ? launch_t<D, false, true, H, FINE>(a, stream) : launch_t<D, false, false, H, FINE>(a, stream);
}

template <bool FINE>
cudaError_t launch_prefill_paged_t(const PrefillArgs& a, cudaStream_t stream) {
  switch (a.d) {
    case 64: return a.halves ? launch_d<64, true, FINE>(a, stream) : launch_d<64, false, FINE>(a, stream);
    case 128: return a.halves ? launch_d<128, true, FINE>(a, stream) : launch_d<128, false, FINE>(a, stream);
    case 256: return launch_d<256, false, FINE>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace
}  // namespace attn
