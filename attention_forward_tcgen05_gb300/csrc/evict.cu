// evict.cu -- eviction from a cache by accumulated attention weight.
//
// Per (sequence, KV head) with L keys and a budget of N: if L <= N every key stays; else
// the first n_sink, the last n_recent, and of the keys between them the
// N - n_sink - n_recent with the largest weights (equal weights: the lowest index).  The
// kept rows of K and V move to the front, in order.
//
// Two launches.  select: one CTA per (sequence, KV head), or a cluster that shares a long row,
// finds the weight of the last key that stays by a radix search over the weights' bits (11 +
// 11 + 10, histograms in shared memory, integer counts: the order of the atomics does not
// show), which ends as soon as all keys of a digit stay: after two digits, as a rule.  One
// scan then numbers the kept keys.  Reads 4 bytes a key; the instructions of its passes bound
// it (512 rows of up to 8192 keys: 25 us).
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
// keys whose weights are in shared memory at a time
constexpr int sel_block(int threads) { return 31 * threads; }

// Order of weights as unsigned integers: -0 = +0, NaN above everything.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 -> +0
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

constexpr uint32_t kMinusInf = 0x007FFFFFu, kPlusInf = 0xFF800000u;  // of -inf and +inf

// The weight of such an integer.
__device__ __forceinline__ float order_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
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

// cs CTAs take equal slices of a row each (a cluster, if kCluster; else cs = 1).
template <int kSelThreads, bool kCluster>
__global__ void __launch_bounds__(kSelThreads, kSelThreads == 1024 ? 1 : (kCluster ? 2 : 4))
    evict_select_kernel(const EvictArgs a, int cs) {
  constexpr int kSelWarps = kSelThreads / 32, kBlock = sel_block(kSelThreads);
  extern __shared__ float sw[];  // a block of the row's weights
  __shared__ __align__(16) int hists[kCluster ? 2 : 1][kBins];
  __shared__ int warp_sums[32];
  __shared__ int found[3];  // the digit of the threshold, keys still wanted at it, keys that have it
  __shared__ uint32_t slice_count;
  const int bh = kCluster ? blockIdx.x / cs : blockIdx.x, rank = kCluster ? blockIdx.x % cs : 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cap = a.src.max_pages * a.src.page_size;
  const int L = min(max(a.kv_lens[bh / a.Hkv], 0), cap);
  const int n = min(L, a.budget);
  const int slice = kCluster ? ((L + cs - 1) / cs + 31) / 32 * 32 : L;  // (at most kBlock in a cluster)
  const int lo = min(L, rank * slice), hi = min(L, lo + slice);
  const float* w = a.weights + (size_t)bh * a.w_stride;
  float* wo = a.weights_out ? a.weights_out + (size_t)bh * a.w_stride : nullptr;
  int* kept = a.kept + (size_t)bh * a.budget;
  const int c_lo = a.n_sink, c_hi = L - a.n_recent;  // the keys that compete
  auto copy_in = [&](int j0) {
    const int m = min(kBlock, hi - j0);
#pragma unroll 8
    for (int i = threadIdx.x; i < m; i += kSelThreads) sw[i] = w[j0 + i];
  };
  // a slice of one block is read once
  auto stage = [&](int j0) {
    if (hi - lo <= kBlock) return;
    __syncthreads();  // the block before is no longer read
    copy_in(j0);
    __syncthreads();
  };
  if (hi - lo <= kBlock) copy_in(lo);
  // (unsigned: a step past a budget near 2^31 is no int)
  for (unsigned i = n + rank * kSelThreads + threadIdx.x; i < (unsigned)a.budget; i += cs * kSelThreads) kept[i] = -1;

  uint32_t prefix = 0;  // the threshold's bits so far
  int want = L > n ? n - a.n_sink - a.n_recent : 0;
  const bool search = want > 0;
  // Until the keys that share the threshold's bits so far all stay: `below` is then the
  // largest integer that does not.  Or to its last bit: `below` is the threshold, and the
  // first `want` keys that equal it stay (ties).
  bool ties_count = false;
  uint32_t below = 0;
  if (search) {
    int shift = 21, bits = 11;
    for (int pass = 0; pass < 3; ++pass) {
      int* hist = hists[kCluster ? pass & 1 : 0];
      if (!kCluster || pass == 0) {
        for (int i = threadIdx.x; i < (int)(sizeof(hists) / 4); i += kSelThreads) hists[0][i] = 0;
        __syncthreads();
      }
      const uint32_t mask = (1u << bits) - 1u;
      // the weights that share the threshold's bits so far, as floats: [v_lo, v_hi] and maybe
      // NaN (2 comparisons where the integer takes 6 instructions; -0 is not at 0x7FFFFFFF)
      const uint32_t low = pass == 0 ? 0u : prefix << (shift + bits);
      const uint32_t high = pass == 0 ? 0xFFFFFFFFu : low | ((1u << (shift + bits)) - 1u);
      const float v_lo = order_value(max(low, kMinusInf));
      const bool nan = high == 0xFFFFFFFFu;
      const float v_hi = order_value(high == 0x7FFFFFFFu ? high - 1 : min(high, kPlusInf));
      for (int j0 = lo; j0 < hi; j0 += kBlock) {
        stage(j0);
        const int i1 = min(min(kBlock, hi - j0), c_hi - j0);
#pragma unroll 8
        for (int i = max(0, c_lo - j0) + (int)threadIdx.x; i < i1; i += kSelThreads) {
          const float v = sw[i];
          if ((v >= v_lo && v <= v_hi) || (nan && v != v)) atomicAdd(&hist[(order_key(v) >> shift) & mask], 1);
        }
      }
      // the digit at which the count from the top reaches `want`: thread t holds the
      // kPer bins from kBins - 1 - kPer t down
      constexpr int kPer = kBins / kSelThreads;
      const int b0 = kBins - kPer * ((int)threadIdx.x + 1);
      int h[kPer], sum = 0;
      if constexpr (kCluster) {
        static_assert(kPer == 4, "a thread's bins are one load");
        __syncwarp();
        cluster_sync_all();  // every CTA's counts are there (and those of the pass before read)
#pragma unroll
        for (int k = 0; k < kPer; ++k) h[k] = 0;
        const uint32_t at = smem_u32(hist + b0);
        for (int r0 = 0; r0 < cs; r0 += 4) {  // (cs is a power of two)
          uint4 x[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            x[r] = make_uint4(0, 0, 0, 0);
            if (r0 + r < cs) x[r] = ld_cluster_v4(mapa_shared(at, (rank + r0 + r) & (cs - 1)));
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            h[3] += (int)x[r].x; h[2] += (int)x[r].y; h[1] += (int)x[r].z; h[0] += (int)x[r].w;
          }
        }
        if (pass == 1)  // the third pass's
          for (int i = threadIdx.x; i < kBins; i += kSelThreads) hists[0][i] = 0;
      } else {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kPer; ++k) h[k] = hist[b0 + kPer - 1 - k];
      }
#pragma unroll
      for (int k = 0; k < kPer; ++k) sum += h[k];
      int total;
      int above = block_scan<kSelWarps>(sum, warp_sums, &total);
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (above < want && want <= above + h[k]) {
          found[0] = b0 + kPer - 1 - k;
          found[1] = want - above;
          found[2] = h[k];
        }
        above += h[k];
      }
      __syncthreads();
      prefix = (prefix << bits) | (uint32_t)found[0];
      want = found[1];
      if (want == found[2]) {
        const uint32_t floor = prefix << shift;
        below = floor ? floor - 1 : 0;  // (0, a NaN's that no weight has, is below all)
        break;
      }
      if (pass == 2) {
        ties_count = true;
        below = prefix;
      }
      shift -= pass == 0 ? 11 : 10;
      bits = pass == 0 ? 11 : 10;
    }
  }
  // As floats (NaN counts as above every number, and the zeros are equal): v stays unless
  // v <= v_below.
  const bool below_nan = below == 0xFFFFFFFFu;
  const float v_below = order_value(below == 0x7FFFFFFFu ? below - 1 : min(below, kPlusInf));
  // A warp takes a span of the block in rows of 32 keys, a key a lane, and lane r keeps what
  // row r's ballot said.  From the warps' counts a lane learns where its row's keys go, and
  // the rows are written lanes side by side.  (With a run of keys to each thread, written one
  // after the other, the scattered stores took 8.4 of a 16384-key row's 21 us.)  A kept key's
  // place is at or before its own, and everything up to the end of a block is in shared memory
  // when its places are written: weights_out may be weights.
  int sure0 = 0, ties0 = 0;  // of the slices and blocks before
  __syncthreads();
  for (int j0 = lo; kCluster ? j0 == lo : j0 < hi; j0 += kBlock) {
    stage(j0);
    const int m = min(kBlock, hi - j0), rows = (m + kSelThreads - 1) / kSelThreads;  // at most 31
    const int i0 = min(m, warp * rows * 32), i1 = min(m, i0 + rows * 32);
    uint32_t stays = 0, tied = 0;
#pragma unroll 4
    for (int r = 0; r < rows; ++r) {
      const int i = i0 + r * 32 + lane, j = j0 + i;
      const float v = i < i1 ? sw[i] : 0.f;
      const bool in = L > n && j >= c_lo && j < c_hi;  // (it competes)
      const uint32_t s = __ballot_sync(0xFFFFFFFFu, i < i1 && (!in || (search && !(v <= v_below) && !below_nan)));
      if (lane == r) stays = s;
      if (ties_count) {
        const uint32_t t = __ballot_sync(0xFFFFFFFFu, i < i1 && in && (below_nan ? v != v : v == v_below));
        if (lane == r) tied = t;
      }
    }
    // (a block's counts fit 16 bits each)
    const uint32_t count = __reduce_add_sync(0xFFFFFFFFu, (uint32_t)(__popc(stays) << 16 | __popc(tied)));
    if (lane == 0) warp_sums[warp] = (int)count;
    __syncthreads();
    const uint32_t others = lane < kSelWarps ? (uint32_t)warp_sums[lane] : 0u;
    const uint32_t before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? others : 0u);
    const uint32_t total = __reduce_add_sync(0xFFFFFFFFu, others);
    if constexpr (kCluster) {
      if (threadIdx.x == 0) slice_count = total;
      __syncwarp();
      cluster_sync_all();
      const uint32_t x = lane < rank ? ld_cluster_u32(mapa_shared(smem_u32(&slice_count), lane)) : 0u;
      sure0 = (int)__reduce_add_sync(0xFFFFFFFFu, x >> 16);
      ties0 = (int)__reduce_add_sync(0xFFFFFFFFu, x & 0xFFFFu);
      cluster_arrive();  // this CTA reads no more of the others
    }
    int ties = ties0 + (int)(before & 0xFFFFu);
    int at = sure0 + (int)(before >> 16) + (ties_count ? min(ties, want) : 0);
    // exclusive sum over the warp's lanes
    auto scan = [&](int v) {
      int x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
      }
      return x - v;
    };
    if (ties_count) {  // the first of them stay
      const int left = max(want - ties - scan(__popc(tied)), 0);
      while (__popc(tied) > left) tied &= ~(0x80000000u >> __clz(tied));
      stays |= tied;
    }
    at += scan(__popc(stays));
#pragma unroll 4
    for (int r = 0; r < rows; ++r) {
      const uint32_t s = __shfl_sync(0xFFFFFFFFu, stays, r);
      const int to = __shfl_sync(0xFFFFFFFFu, at, r) + __popc(s & ((1u << lane) - 1u));
      if ((s >> lane) & 1u) {
        const int i = i0 + r * 32 + lane;
        kept[to] = j0 + i;
        if (wo) wo[to] = sw[i];
      }
    }
    sure0 += (int)(total >> 16);
    ties0 += (int)(total & 0xFFFFu);
  }
  __syncthreads();
  if (wo)  // the freed keys' sums
    for (int i = n + rank * kSelThreads + threadIdx.x; i < L; i += cs * kSelThreads) wo[i] = 0.f;
  __syncwarp();
  if constexpr (kCluster) cluster_wait();  // its counts are read until the others have arrived
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
      x[p] = make_uint4(0, 0, 0, 0);  // (a row of a bad page)
      if (i < n && kept[i] != i) {
        const int s = paged_row(a.src, b, kept[i], a.err);
        dst[p] = paged_row(a.src, b, i, a.err);
        if (s >= 0)
          x[p] = *reinterpret_cast<const uint4*>(pool + ((size_t)s * a.Hkv + hk) * D + slice * 32 + c * 8);
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


cudaError_t launch_select(const EvictArgs& a, cudaStream_t stream) {
  const int cap = a.src.max_pages * a.src.page_size;
  const long long rows = (long long)a.B * a.Hkv;
  constexpr int kThreads = 512, kBlock = sel_block(kThreads);
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  // Long rows that leave SMs idle are shared by up to four CTAs, by eight where only that keeps
  // a slice in one block (4 rows of 16384 / 30000 keys, call: 26 / 38 us alone, 17.3 / 19.9 with
  // two, 15.5 / 16.7 with four, 15.9 / 17.0 with eight; of 8192: 12.0, 11.5, 11.4, 12.5)
  int cs = 1;
  if (cap > 8192)
    while (rows * cs * 2 <= 152 && (cs < 4 || (cs < 8 && cap > cs * kBlock))) cs *= 2;
  if (cs > 1 && cap <= cs * kBlock) {
    auto kern = evict_select_kernel<kThreads, true>;
    const int slice = ((cap + cs - 1) / cs + 31) / 32 * 32;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kBlock * 4);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(rows * cs));
    cfg.dynamicSmemBytes = (size_t)slice * 4;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)cs;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a, cs);
  }
  auto kern = evict_select_kernel<kThreads, false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kBlock * 4);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)rows);
  cfg.dynamicSmemBytes = (size_t)(cap < kBlock ? cap : kBlock) * 4;
  return cudaLaunchKernelEx(&cfg, kern, a, 1);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
  cudaError_t e = launch_select(a, stream);
  if (e != cudaSuccess) return e;
  switch (a.d) {
    case 64: return launch_move<64>(a, stream);
    case 128: return launch_move<128>(a, stream);
    case 256: return launch_move<256>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
