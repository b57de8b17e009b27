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
// numbers the kept keys.  Reads 4 bytes a key; the instructions of its four passes bound it.
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

constexpr int kBins = 2048;
// keys whose weights are in shared memory at a time: 31 (an odd number) for each thread
constexpr int sel_block(int threads) { return 31 * threads; }

// Order of weights as unsigned integers: -0 = +0, NaN above everything.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 -> +0
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// Exclusive sum over the block of kSelWarps warps; *total gets the sum.
template <int kSelWarps>
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
    int s = lane < kSelWarps ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < kSelWarps; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, s, o);
      if (lane >= o) s += y;
    }
    if (lane < kSelWarps) warp_sums[lane] = s;
  }
  __syncthreads();
  *total = warp_sums[kSelWarps - 1];
  return x - v + (warp ? warp_sums[warp - 1] : 0);
}

template <int kSelThreads>
__global__ void __launch_bounds__(kSelThreads, kSelThreads == 1024 ? 1 : 4)
    evict_select_kernel(const EvictArgs a) {
  constexpr int kSelWarps = kSelThreads / 32, kBlock = sel_block(kSelThreads);
  extern __shared__ float sw[];  // a block of the row's weights
  __shared__ int hist[kBins];
  __shared__ int warp_sums[32];
  __shared__ int found[2];  // the digit of the threshold, keys still wanted at it
  const int b = blockIdx.x / a.Hkv;
  const int cap = a.src.max_pages * a.src.page_size;
  const int L = min(max(a.kv_lens[b], 0), cap);
  const int n = min(L, a.budget);
  const float* w = a.weights + (size_t)blockIdx.x * a.w_stride;
  float* wo = a.weights_out ? a.weights_out + (size_t)blockIdx.x * a.w_stride : nullptr;
  int* kept = a.kept + (size_t)blockIdx.x * a.budget;
  const int c_lo = a.n_sink, c_hi = L - a.n_recent;  // the keys that compete
  auto copy_in = [&](int j0) {
#pragma unroll 4
    for (int i = threadIdx.x; i < min(kBlock, L - j0); i += kSelThreads) sw[i] = w[j0 + i];
  };
  // a row of one block is read once
  auto stage = [&](int j0) {
    if (L <= kBlock) return;
    __syncthreads();  // the block before is no longer read
    copy_in(j0);
    __syncthreads();
  };
  // a thread's keys of the block at j0: a run of an odd number of them (no bank conflicts)
  auto run = [&](int j0, int& i0, int& i1) {
    const int m = min(kBlock, L - j0), per = ((m + kSelThreads - 1) / kSelThreads) | 1;
    i0 = min(m, (int)threadIdx.x * per);
    i1 = min(m, i0 + per);
  };
  if (L <= kBlock) copy_in(0);
  for (int i = n + threadIdx.x; i < a.budget; i += kSelThreads) kept[i] = -1;

  uint32_t prefix = 0;  // the threshold's bits so far
  int want = L > n ? n - a.n_sink - a.n_recent : 0;
  const bool search = want > 0;
  if (search) {
    int shift = 21, bits = 11;
    for (int pass = 0; pass < 3; ++pass) {
      for (int i = threadIdx.x; i < kBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      const uint32_t mask = (1u << bits) - 1u;
      for (int j0 = 0; j0 < L; j0 += kBlock) {
        stage(j0);
        int i0, i1;
        run(j0, i0, i1);
        i0 = max(i0, c_lo - j0);
        i1 = min(i1, c_hi - j0);
#pragma unroll 4
        for (int i = i0; i < i1; ++i) {
          const uint32_t key = order_key(sw[i]);
          if (pass == 0 || (key >> (shift + bits)) == prefix) atomicAdd(&hist[(key >> shift) & mask], 1);
        }
      }
      __syncthreads();
      // the digit at which the count from the top reaches `want`: thread t holds the
      // kPer bins from kBins - 1 - kPer t down
      constexpr int kPer = kBins / kSelThreads;
      int h[kPer], sum = 0;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        h[k] = hist[kBins - 1 - kPer * (int)threadIdx.x - k];
        sum += h[k];
      }
      int total;
      int above = block_scan<kSelWarps>(sum, warp_sums, &total);
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (above < want && want <= above + h[k]) {
          found[0] = kBins - 1 - kPer * (int)threadIdx.x - k;
          found[1] = want - above;
        }
        above += h[k];
      }
      __syncthreads();
      prefix = (prefix << bits) | (uint32_t)found[0];
      want = found[1];
      shift -= pass == 0 ? 11 : 10;
      bits = pass == 0 ? 11 : 10;
    }
  }
  // Keys above the threshold stay, and the first `want` equal to it (as floats: NaN counts
  // as above every number, and the zeros are equal).  A thread marks its run in two masks,
  // one scan numbers the runs.  A kept key's place is at or before its own, and everything up
  // to the end of a block is in shared memory when its places are written: weights_out may
  // be weights.
  const bool limit_nan = prefix == 0xFFFFFFFFu;
  const float limit = __uint_as_float((prefix & 0x80000000u) ? prefix & 0x7FFFFFFFu : ~prefix);
  int sure0 = 0, ties0 = 0;  // of the blocks before
  __syncthreads();
  for (int j0 = 0; j0 < L; j0 += kBlock) {
    stage(j0);
    int i0, i1;
    run(j0, i0, i1);
    uint32_t sure = 0, tie = 0;  // bit i - i0
    if (search) {
#pragma unroll 4
      for (int i = i0; i < i1; ++i) {
        const float v = sw[i];
        const bool in = j0 + i >= c_lo && j0 + i < c_hi;
        const uint32_t bit = 1u << (i - i0);
        if (!in || (!(v <= limit) && !limit_nan)) sure |= bit;
        if (in && (limit_nan ? v != v : v == limit)) tie |= bit;
      }
    } else {
      for (int i = i0; i < i1; ++i)
        if (L <= n || j0 + i < c_lo || j0 + i >= c_hi) sure |= 1u << (i - i0);
    }
    // (a block's counts fit 16 bits each)
    int total;
    const int before = block_scan<kSelWarps>(__popc(sure) << 16 | __popc(tie), warp_sums, &total);
    int ties = ties0 + (before & 0xFFFF);
    int at = sure0 + (before >> 16) + min(ties, want);
    for (uint32_t m = sure | tie; m; m &= m - 1) {
      const int k = __ffs(m) - 1;
      const bool is_tie = (tie >> k) & 1u;
      if (!is_tie || ties < want) {
        kept[at] = j0 + i0 + k;
        if (wo) wo[at] = sw[i0 + k];
        ++at;
      }
      ties += is_tie;
    }
    sure0 += total >> 16;
    ties0 += total & 0xFFFF;
  }
  __syncthreads();
  if (wo)
    for (int i = n + threadIdx.x; i < L; i += kSelThreads) wo[i] = 0.f;  // the freed keys' sums
}

// One CTA per (sequence, range of kept rows, KV head), heads innermost: CTAs that run
// together then write whole slots, and read near one another.
// The rows' places are found once, a thread each, and the copy then runs on them.
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 128;

template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_copy_kernel(const EvictArgs a, int ranges) {
  constexpr int CPR = D / 8, RPP = kMoveThreads / CPR;  // lanes of a row, rows of a pass
  constexpr int NP = 4;                                 // passes in flight (K and V)
  __shared__ int place[2][kMoveRows];                   // pool rows: from, to
  const int hk = blockIdx.x % a.Hkv, range = blockIdx.x / a.Hkv % ranges, b = blockIdx.x / a.Hkv / ranges;
  const int bh = b * a.Hkv + hk;
  const int cap = a.src.max_pages * a.src.page_size;
  const int n = min(min(max(a.kv_lens[b], 0), cap), a.budget);
  if (hk == 0 && range == 0 && threadIdx.x == 0) a.new_lens[b] = n;
  const int lo = range * kMoveRows;
  if (lo >= n) return;
  {
    static_assert(kMoveThreads == 2 * kMoveRows, "a thread per row and side");
    const int side = threadIdx.x / kMoveRows, i = lo + threadIdx.x % kMoveRows;
    int r = -1;
    if (i < n) r = side ? paged_row(a.dst, b, i, a.err) : paged_row(a.src, b, a.kept[(size_t)bh * a.budget + i], a.err);
    place[side][threadIdx.x % kMoveRows] = r;
  }
  __syncthreads();
  const int c = threadIdx.x % CPR, r0 = threadIdx.x / CPR;
  const size_t head = (size_t)hk * D + c * 8, stride = (size_t)a.Hkv * D;
#pragma unroll 1
  for (int p0 = 0; p0 < kMoveRows / RPP; p0 += NP) {
    uint4 x[2][NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int s = place[0][(p0 + p) * RPP + r0];
      x[0][p] = x[1][p] = make_uint4(0, 0, 0, 0);
      if (s >= 0) {
        x[0][p] = *reinterpret_cast<const uint4*>(a.src.k + s * stride + head);
        x[1][p] = *reinterpret_cast<const uint4*>(a.src.v + s * stride + head);
      }
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int d = place[1][(p0 + p) * RPP + r0];
      if (d >= 0) {
        *reinterpret_cast<uint4*>(a.dk + d * stride + head) = x[0][p];
        *reinterpret_cast<uint4*>(a.dv + d * stride + head) = x[1][p];
      }
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
  // where every row has an SM to itself, a row in one large CTA
  const bool few = (long long)a.B * a.Hkv <= 152;
  const int threads = few ? 1024 : 512, block = sel_block(threads);
  auto kern = few ? evict_select_kernel<1024> : evict_select_kernel<512>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, block * 4);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)(a.B * a.Hkv), threads, (size_t)(cap < block ? cap : block) * 4, stream>>>(a);
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
