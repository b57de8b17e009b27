// prefill.cu -- launches of the single-CTA prefill over dense keys (the kernel:
// prefill_kernel.cuh; over a paged cache: prefill_paged.cu).
#include "prefill_kernel.cuh"

namespace attn {
namespace {

// Skv == 0: no key at all, O = 0 and LSE = -inf for every row.
__global__ void fill_empty_kernel(void* o, float* lse, size_t n_o, size_t n_lse, int o_bf16) {
  const size_t stride = (size_t)gridDim.x * blockDim.x;
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n_o; i += stride) {
    if (o_bf16) reinterpret_cast<uint16_t*>(o)[i] = 0;
    else reinterpret_cast<float*>(o)[i] = 0.f;
  }
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n_lse; i += stride)
    lse[i] = -INFINITY;
}

// SMs of the current device
int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

// One launch of grid CTAs over units [unit0, ...) with configuration H.
template <int D, bool H>
cudaError_t launch_prefill_grid(const PrefillArgs& a, cudaStream_t stream, long long unit0, long long grid,
                                int row_halves) {
  using C = PrefillCfg<D, H>;
  auto kern = fmha_fwd_kernel<D, false, false, false, false, false>;
  if constexpr (H) {
    kern = a.n_splits > 1 ? fmha_fwd_kernel<D, false, true, true, false, false> : fmha_fwd_kernel<D, false, false, true, false, false>;
  } else {
    if (a.window > 0) kern = fmha_fwd_kernel<D, true, false, false, false, false>;
    else if (a.n_splits > 1) kern = fmha_fwd_kernel<D, false, true, false, false, false>;
  }
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  if (grid <= 0) return cudaSuccess;
  const int G = a.pack;
  const int n_splits = a.n_splits > 1 ? a.n_splits : 1;
  kern<<<(unsigned)grid, C::kThreads, C::kSmemBytes, stream>>>(
      a.tm_q, a.tm_k, a.tm_v, a.tm_o, a.o_tma, a.o, a.lse, a.Hq, a.Hkv, a.Sq, a.Skv, a.causal, a.o_bf16, a.scale,
      (a.Hq / G) * a.B, a.err, a.cu_q, a.kv_lens, a.total_q, a.window, a.n_sink, G, n_splits,
      a.split_min, a.part_o, a.part_lse, (int)unit0, row_halves, PagedKV{});
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_prefill_t(const PrefillArgs& a, cudaStream_t stream) {
  using C = PrefillCfg<D, false>;
  const int G = a.pack;
  const long long rows = (long long)a.Sq * G;
  const long long n_blocks_q = (rows + C::NQ * kPrefillTileM - 1) / (C::NQ * kPrefillTileM);
  const int n_splits = a.n_splits > 1 ? a.n_splits : 1;
  const long long units = n_blocks_q * (a.Hq / G) * a.B * n_splits;
  if (units <= 0) return cudaSuccess;
  if (2 * units > 0x7FFFFFFFLL || rows > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  if (a.halves) return launch_prefill_grid<D, true>(a, stream, 0, units, 0);
  // a causal fixed-length launch (one head per tile, no window or key splits) runs
  // on the persistent kernel, which overlaps each unit's Q load, first MMAs and O
  // epilogue with its neighbours (prefill_persist.cu)
  if (a.causal && a.window == 0 && n_splits == 1 && a.cu_q == nullptr && a.kv_lens == nullptr && G == 1)
    return launch_prefill_persistent(a, stream);
  // A non-causal fixed-length launch whose last wave is at most half full: that
  // wave's units run as two 128-row halves each, whose two query tiles take the
  // two halves of the keys (the key-halves kernel), in about half a unit's time.
  const bool plain = !a.causal && a.window == 0 && n_splits == 1 && a.cu_q == nullptr &&
                     a.kv_lens == nullptr && G == 1;
  const long long n_sm = sm_count();
  const long long tail = n_sm > 0 ? units % n_sm : 0;
  if (plain && units > n_sm && tail > 0 && 2 * tail <= n_sm) {
    cudaError_t e = launch_prefill_grid<D, false>(a, stream, 0, units - tail, 0);
    if (e != cudaSuccess) return e;
    return launch_prefill_grid<D, true>(a, stream, units - tail, 2 * tail, 1);
  }
  return launch_prefill_grid<D, false>(a, stream, 0, units, 0);
}

}  // namespace

cudaError_t launch_prefill(const PrefillArgs& a, cudaStream_t stream) {
  switch (a.d) {
    case 64: return launch_prefill_t<64>(a, stream);
    case 128: return launch_prefill_t<128>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_prefill_empty_kv(const PrefillArgs& a, cudaStream_t stream) {
  const size_t rows = a.cu_q ? (size_t)a.total_q : (size_t)a.B * a.Sq;
  const size_t n_o = rows * a.Hq * a.d;
  const size_t n_lse = rows * a.Hq;
  if (n_o == 0) return cudaSuccess;
  fill_empty_kernel<<<1024, 256, 0, stream>>>(a.o, a.lse, n_o, n_lse, a.o_bf16);
  return cudaGetLastError();
}

}  // namespace attn
