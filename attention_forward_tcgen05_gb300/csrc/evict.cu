// evict.cu -- eviction from a cache by accumulated attention weight.
//
// Per (sequence, KV head) with L keys and a budget of N: if L <= N every key stays; else
// the first n_sink, the last n_recent, and of the keys between them the
// N - n_sink - n_recent with the largest weights (equal weights: the lowest index).  The
// kept rows of K and V move to the front, in order.
//
// Two launches.  select: one CTA per (sequence, KV head) finds the weight of the last key
// that stays by a radix search over the weights' bits (11 + 11 + 10, three histograms in
// shared memory, integer counts: the order of the atomics does not show), then one scan
// numbers the kept keys.  Reads 4 bytes a key; latency of its passes bounds it.
// move: copies the rows, 16 bytes a thread; bound by HBM.  Into other pages the kept list
// is cut into ranges, one CTA each.  In place a row only ever moves towards the front and
// the list is ascending, so a CTA that owns a (sequence, KV head, column slice) and walks
// it front to back never overwrites a row it has yet to read; slices give the parallelism.
#include <cmath>

#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kBins = 2048;
constexpr int kStageKeys = 49152;  // weights kept in shared memory (192 KB); longer rows are re-read

// Order of weights as unsigned integers: -0 = +0, NaN above everything.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 -> +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive sum over the block (kSelThreads threads); *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // warp_sums of an earlier call are no longer read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  *total = warp_sums[31];
  return x - v + (warp ? warp_sums[warp - 1] : 0);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a, int staged) {
  extern __shared__ float sw[];
  __shared__ int hist[kBins];
  __shared__ int warp_sums[32];
  __shared__ int found[2];  // the digit of the threshold, keys still wanted at it
  const int b = blockIdx.x / a.Hkv;
  const int cap = a.src.max_pages * a.src.page_size;
  const int L = min(max(a.kv_lens[b], 0), cap);
  const int n = min(L, a.budget);
  const float* w = a.weights + (size_t)blockIdx.x * a.w_stride;
  int* kept = a.kept + (size_t)blockIdx.x * a.budget;
  for (int i = n + threadIdx.x; i < a.budget; i += kSelThreads) kept[i] = -1;
  const int c_lo = a.n_sink, c_hi = L - a.n_recent;  // the keys that compete
  const bool in_smem = L <= staged;
  if (in_smem) {
    for (int j = threadIdx.x; j < L; j += kSelThreads) sw[j] = w[j];
    __syncthreads();
  }
  const float* ws = in_smem ? sw : w;
  uint32_t prefix = 0;  // the threshold's bits so far
  int want = L > n ? n - a.n_sink - a.n_recent : 0;
  const bool search = want > 0;
  if (search) {
    int shift = 21, bits = 11;
    for (int pass = 0; pass < 3; ++pass) {
      for (int i = threadIdx.x; i < kBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      const uint32_t mask = (1u << bits) - 1u;
      for (int j = c_lo + threadIdx.x; j < c_hi; j += kSelThreads) {
        const uint32_t k = order_key(ws[j]);
        if (pass == 0 || (k >> (shift + bits)) == prefix) atomicAdd(&hist[(k >> shift) & mask], 1);
      }
      __syncthreads();
      // the digit at which the count from the top reaches `want`: thread t holds the
      // bins kBins - 1 - 2t and kBins - 2 - 2t
      const int h0 = hist[kBins - 1 - 2 * threadIdx.x], h1 = hist[kBins - 2 - 2 * threadIdx.x];
      int total;
      const int above = block_scan(h0 + h1, warp_sums, &total);
      if (above < want && want <= above + h0) {
        found[0] = kBins - 1 - 2 * (int)threadIdx.x;
        found[1] = want - above;
      } else if (above + h0 < want && want <= above + h0 + h1) {
        found[0] = kBins - 2 - 2 * (int)threadIdx.x;
        found[1] = want - above - h0;
      }
      __syncthreads();
      prefix = (prefix << bits) | (uint32_t)found[0];
      want = found[1];
      shift -= pass == 0 ? 11 : 10;
      bits = pass == 0 ? 11 : 10;
    }
  }
  // keys above the threshold stay, and the first `want` equal to it.  Thread t numbers a
  // run of consecutive keys (an odd count: no bank conflicts).
  const int per = ((L + kSelThreads - 1) / kSelThreads) | 1;
  const int j0 = min(L, (int)threadIdx.x * per), j1 = min(L, j0 + per);
  auto cls = [&](int j) -> int {  // 1: stays, 2: equal to the threshold
    if (L <= n || j < c_lo || j >= c_hi) return 1;
    if (!search) return 0;
    const uint32_t k = order_key(ws[j]);
    return k > prefix ? 1 : (k == prefix ? 2 : 0);
  };
  int sure = 0, ties = 0;
  for (int j = j0; j < j1; ++j) {
    const int c = cls(j);
    sure += c == 1;
    ties += c == 2;
  }
  int total;
  const int sure_before = block_scan(sure, warp_sums, &total);
  const int ties_before = block_scan(ties, warp_sums, &total);
  int at = sure_before + min(ties_before, want), tie = ties_before;
  for (int j = j0; j < j1; ++j) {
    const int c = cls(j);
    const bool take = c == 1 || (c == 2 && tie < want);
    tie += c == 2;
    if (take) kept[at++] = j;
  }
  __syncthreads();
  if (a.weights_out) {
    float* wo = a.weights_out + (size_t)blockIdx.x * a.w_stride;
    // in place: position i is written after every thread of the chunk has read, and later
    // chunks read at or past their own positions
    for (int i0 = 0; i0 < n; i0 += kSelThreads) {
      const int i = i0 + threadIdx.x;
      const float v = i < n ? ws[kept[i]] : 0.f;
      __syncthreads();
      if (i < n) wo[i] = v;
    }
    __syncthreads();
    for (int i = n + threadIdx.x; i < L; i += kSelThreads) wo[i] = 0.f;  // the freed keys' sums
  }
}

// grid (ranges of kept rows, B * Hkv); rows of K, then of V
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 64;

template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_copy_kernel(const EvictArgs a, int ranges) {
  constexpr int CPR = D / 8, RPP = kMoveThreads / CPR;  // lanes of a row, rows of a pass
  constexpr int NP = kMoveRows / RPP;
  const int bh = blockIdx.x / ranges, range = blockIdx.x % ranges;
  const int b = bh / a.Hkv, hk = bh % a.Hkv;
  const int cap = a.src.max_pages * a.src.page_size;
  const int n = min(min(max(a.kv_lens[b], 0), cap), a.budget);
  if (bh % a.Hkv == 0 && range == 0 && threadIdx.x == 0) a.new_lens[b] = n;
  const int lo = range * kMoveRows;
  if (lo >= n) return;
  const int c = threadIdx.x % CPR, r0 = threadIdx.x / CPR;
  const int* kept = a.kept + (size_t)bh * a.budget;
  uint4 x[2][NP];
  int dst[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int i = lo + p * RPP + r0;
    dst[p] = -1;
    x[0][p] = x[1][p] = make_uint4(0, 0, 0, 0);
    if (i < n) {
      const int s = paged_row(a.src, b, kept[i], a.err);
      dst[p] = paged_row(a.dst, b, i, a.err);
      if (s >= 0) {
        const size_t off = ((size_t)s * a.Hkv + hk) * D + c * 8;
        x[0][p] = *reinterpret_cast<const uint4*>(a.src.k + off);
        x[1][p] = *reinterpret_cast<const uint4*>(a.src.v + off);
      }
    }
  }
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    if (dst[p] >= 0) {
      const size_t off = ((size_t)dst[p] * a.Hkv + hk) * D + c * 8;
      *reinterpret_cast<uint4*>(a.dk + off) = x[0][p];
      *reinterpret_cast<uint4*>(a.dv + off) = x[1][p];
    }
  }
}

// In place: one CTA per (sequence, KV head, 64-byte column slice, K or V), front to back.
template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_compact_kernel(const EvictArgs a) {
  constexpr int kSlices = D / 32, RPP = kMoveThreads / 4, NP = 4;
  const int slice = blockIdx.x % kSlices, is_v = blockIdx.x / kSlices % 2, bh = blockIdx.x / (2 * kSlices);
  const int b = bh / a.Hkv, hk = bh % a.Hkv;
  const int cap = a.src.max_pages * a.src.page_size;
  const int L = min(max(a.kv_lens[b], 0), cap), n = min(L, a.budget);
  if (L <= n) return;  // nothing moves
  const int* kept = a.kept + (size_t)bh * a.budget;
  uint16_t* pool = is_v ? a.dv : a.dk;
  const int c = threadIdx.x % 4, r0 = threadIdx.x / 4;
  for (int lo = 0; lo < n; lo += RPP * NP) {
    uint4 x[NP];
    int dst[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int i = lo + p * RPP + r0;
      dst[p] = -1;
      if (i < n && kept[i] != i) {
        const int s = paged_row(a.src, b, kept[i], a.err);
        if (s >= 0) {
          dst[p] = paged_row(a.src, b, i, a.err);
          x[p] = *reinterpret_cast<const uint4*>(pool + ((size_t)s * a.Hkv + hk) * D + slice * 32 + c * 8);
        }
      }
    }
    __syncthreads();  // every row of this step is read before one is written
#pragma unroll
    for (int p = 0; p < NP; ++p)
      if (dst[p] >= 0)
        *reinterpret_cast<uint4*>(pool + ((size_t)dst[p] * a.Hkv + hk) * D + slice * 32 + c * 8) = x[p];
  }
}

// new_lens of the in-place form, after every CTA has read kv_lens (which it may alias)
__global__ void evict_lens_kernel(const int* kv_lens, int* new_lens, int B, int cap, int budget) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b < B) new_lens[b] = min(min(max(kv_lens[b], 0), cap), budget);
}

template <int D>
cudaError_t launch_move(const EvictArgs& a, cudaStream_t stream) {
  const int cap = a.src.max_pages * a.src.page_size;
  if (a.in_place) {
    const long long ctas = (long long)a.B * a.Hkv * 2 * (D / 32);
    if (ctas > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    evict_compact_kernel<D><<<(unsigned)ctas, kMoveThreads, 0, stream>>>(a);
    evict_lens_kernel<<<(a.B + 255) / 256, 256, 0, stream>>>(a.kv_lens, a.new_lens, a.B, cap, a.budget);
    return cudaGetLastError();
  }
  const int rows = a.budget < cap ? a.budget : cap;
  const int ranges = rows > 0 ? (rows + kMoveRows - 1) / kMoveRows : 1;
  const long long ctas = (long long)a.B * a.Hkv * ranges;
  if (ctas > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  evict_copy_kernel<D><<<(unsigned)ctas, kMoveThreads, 0, stream>>>(a, ranges);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
  const int cap = a.src.max_pages * a.src.page_size;
  const int staged = cap < kStageKeys ? cap : kStageKeys;
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kStageKeys * 4);
  if (e != cudaSuccess) return e;
  evict_select_kernel<<<(unsigned)(a.B * a.Hkv), kSelThreads, (size_t)staged * 4, stream>>>(a, staged);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  switch (a.d) {
    case 64: return launch_move<64>(a, stream);
    case 128: return launch_move<128>(a, stream);
    case 256: return launch_move<256>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
