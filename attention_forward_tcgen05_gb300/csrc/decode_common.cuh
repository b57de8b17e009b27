// decode_common.cuh -- what the one-token decode kernels share (decode.cu over a dense
// cache, decode_paged.cu over pages): the launch order of the split units and the
// LSE-weighted combine of their partials.
#pragma once
#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
  return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
  return v;
}

// ---- launch order of the split units ----
// Unit (b, s) holds clamp(L_b - s*chunk_b, 0, chunk_b) rows.  CTAs start in index
// order and an SM takes the next one when a slot frees, so a ragged batch ends
// soonest when the long units start first and the short ones fill the end (the
// longest-first list-scheduling rule).  Every unit of a sequence but its last
// non-empty one is full, so the order is: all full units, then the partial last
// units by size (kOrderBuckets buckets of chunk / kOrderBuckets rows, largest
// first, batch order within a bucket), then the empty units.  Each CTA derives
// its unit from kv_lens with two warp-wide passes over the batch.  Batches above
// kOrderMaxBatch take the batch-major order instead (the passes would cost more
// than the tail they save).
constexpr int kOrderBuckets = 16;
constexpr int kOrderMaxBatch = 1024;

struct SplitShape {
  int nf;  // full units (chunk rows each)
  int hp;  // 1 if a partial unit follows them
  int bk;  // size bucket of the partial unit, or -1
  int ne;  // empty units
};

// the split rule of the kernel: chunk = max(ceil(L / n_splits), min_rows, 1)
__device__ __forceinline__ SplitShape split_shape(int L, int max_kv, int n_splits, int min_rows) {
  L = L < 0 ? 0 : (L > max_kv ? max_kv : L);
  int chunk = L / n_splits + (L % n_splits != 0 ? 1 : 0);
  chunk = max(max(chunk, min_rows), 1);
  SplitShape r;
  r.nf = L / chunk;
  const int rem = L - r.nf * chunk;
  r.hp = rem > 0 ? 1 : 0;
  r.bk = r.hp ? (int)((long long)rem * kOrderBuckets / chunk) : -1;
  r.ne = n_splits - r.nf - r.hp;
  return r;
}

__device__ __forceinline__ int warp_incl_scan(int v, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int x = __shfl_up_sync(0xFFFFFFFFu, v, off);
    if (lane >= off) v += x;
  }
  return v;
}

// (b, s) of the unit at position p of the launch order, for every lane of the
// calling warp; (-1, -1) if p is past the last unit.
__device__ __noinline__ int2 unit_at(int p, const int* __restrict__ kv_lens, int B, int max_kv, int n_splits,
                                      int min_rows, int lane) {
  auto shape_of = [&](int b) {
    return b < B ? split_shape(kv_lens[b], max_kv, n_splits, min_rows) : SplitShape{0, 0, -1, 0};
  };
  int F = 0, P = 0;  // full and partial units of the batch
  for (int b0 = 0; b0 < B; b0 += 32) {
    const SplitShape sh = shape_of(b0 + lane);
    F += (int)__reduce_add_sync(0xFFFFFFFFu, (unsigned)sh.nf);
    P += __popc(__ballot_sync(0xFFFFFFFFu, sh.hp != 0));
  }
  if (p < F || p >= F + P) {
    // a full unit (the p-th, batch-major) or an empty one (the (p-F-P)-th)
    const bool full = p < F;
    const int q = full ? p : p - F - P;
    int carry = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
      const SplitShape sh = shape_of(b0 + lane);
      const int n = full ? sh.nf : sh.ne;
      const int incl = warp_incl_scan(n, lane) + carry, excl = incl - n;
      const unsigned hit = __ballot_sync(0xFFFFFFFFu, excl <= q && q < incl);
      if (hit) {
        const int src = __ffs(hit) - 1;
        const int first = full ? 0 : sh.nf + sh.hp;  // first unit of the class in the sequence
        const int s = __shfl_sync(0xFFFFFFFFu, first + q - excl, src);
        return make_int2(b0 + src, s);
      }
      carry = __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    return make_int2(-1, -1);
  }
  // a partial unit: count the buckets (lane k < kOrderBuckets holds bucket k)
  int cnt = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    const SplitShape sh = shape_of(b0 + lane);
#pragma unroll
    for (int k = 0; k < kOrderBuckets; ++k) {
      const int c = __popc(__ballot_sync(0xFFFFFFFFu, sh.bk == k));
      if (lane == k) cnt += c;
    }
  }
  int j = p - F, K = -1;
  for (int k = kOrderBuckets - 1; k >= 0; --k) {  // largest bucket first
    const int c = __shfl_sync(0xFFFFFFFFu, cnt, k);
    if (j < c) {
      K = k;
      break;
    }
    j -= c;
  }
  if (K < 0) return make_int2(-1, -1);
  for (int b0 = 0; b0 < B; b0 += 32) {  // the j-th sequence of bucket K, in batch order
    const SplitShape sh = shape_of(b0 + lane);
    const unsigned m = __ballot_sync(0xFFFFFFFFu, sh.bk == K);
    const int c = __popc(m);
    if (j < c) {
      const unsigned below = (1u << lane) - 1u;
      const unsigned hit = __ballot_sync(0xFFFFFFFFu, ((m >> lane) & 1u) && __popc(m & below) == j);
      const int src = __ffs(hit) - 1;
      return make_int2(b0 + src, __shfl_sync(0xFFFFFFFFu, sh.nf, src));
    }
    j -= c;
  }
  return make_int2(-1, -1);
}

// Non-empty splits whose partial rows a merge warp loads at once: eight covers
// the common split counts in one round trip (four took two on eight splits).
constexpr int kMergeBatch = 8;

// The LSE-weighted combine of the n_splits partials of one (sequence, query
// head) row, by one warp: lane = DPL consecutive dims.  The partials are read
// through L2 (ld.global.cg): in the fused decode other CTAs of the same launch
// wrote them, and this SM's L1 may not see those writes.
template <int D, int BATCH = kMergeBatch>
__device__ __noinline__ void merge_row(const float* __restrict__ part_o,
                                          const float* __restrict__ part_lse, void* o,
                                          float* __restrict__ lse, size_t row, size_t lse_row,
                                          int n_splits, int o_bf16, int lane) {
  constexpr int DPL = D / 32;
  const float* pl = part_lse + row * n_splits;
  const float* po = part_o + row * n_splits * D + lane * DPL;
  float M = -INFINITY;
  for (int s = lane; s < n_splits; s += 32) M = fmaxf(M, __ldcg(pl + s));
  M = warp_max(M);
  float acc[DPL];
#pragma unroll
  for (int e = 0; e < DPL; ++e) acc[e] = 0.f;
  float wsum = 0.f;
  if (M != -INFINITY) {
    for (int s0 = 0; s0 < n_splits; s0 += 32) {
      // lane j holds the weight of split s0 + j (0 for empty or missing splits)
      const int s = s0 + lane;
      const float ls = s < n_splits ? __ldcg(pl + s) : -INFINITY;
      const float w = ls == -INFINITY ? 0.f : ex2_approx((ls - M) * kLog2e);
      wsum += w;
      uint32_t live = __ballot_sync(0xFFFFFFFFu, w > 0.f);  // empty splits are never read
      while (live) {
        // up to BATCH non-empty splits per round: their loads are issued together
        int idx[BATCH];
        float wk[BATCH];
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
          idx[u] = live ? __ffs(live) - 1 : -1;
          if (live) live &= live - 1;
          wk[u] = __shfl_sync(0xFFFFFFFFu, w, idx[u] < 0 ? 0 : idx[u]);
        }
        float x[BATCH][DPL];
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
          if (idx[u] >= 0) {
            const float* src = po + (size_t)(s0 + idx[u]) * D;
#pragma unroll
            for (int e = 0; e < DPL; e += 2) {
              const float2 v2 = __ldcg(reinterpret_cast<const float2*>(src + e));
              x[u][e] = v2.x;
              x[u][e + 1] = v2.y;
            }
          }
        }
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
          if (idx[u] >= 0) {
#pragma unroll
            for (int e = 0; e < DPL; ++e) acc[e] = fmaf(wk[u], x[u][e], acc[e]);
          }
        }
      }
    }
    wsum = warp_sum(wsum);
  }
  const float inv = wsum > 0.f ? 1.f / wsum : 0.f;
  if (o_bf16) {
    uint16_t* dst = reinterpret_cast<uint16_t*>(o) + row * D + lane * DPL;
#pragma unroll
    for (int e = 0; e < DPL; e += 2) {
      *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    }
  } else {
    float* dst = reinterpret_cast<float*>(o) + row * D + lane * DPL;
#pragma unroll
    for (int e = 0; e < DPL; e += 2) {
      *reinterpret_cast<float2*>(dst + e) = make_float2(acc[e] * inv, acc[e + 1] * inv);
    }
  }
  if (lane == 0) lse[lse_row] = wsum > 0.f ? M + logf(wsum) : -INFINITY;
}

// The combine fused into the split launch ("66 . D2: explicit K+V register
// staging", section 5.2, without a launch of its own).  The n_splits CTAs that
// hold the same query heads of a sequence form a group with one completion
// counter, indexed by the group's first (sequence, query head) row.  Each CTA,
// once its partials are written, fences them and counts
// itself; the CTA that takes the count to n_splits merges the group's rows
// into o and lse and puts the counter back to zero, so the counters are zero
// again when the launch ends.  Called by the first NWARPS warps of the CTA
// together; `sync` is their barrier.
template <int D, int NWARPS, int BATCH = kMergeBatch, class Sync>
__device__ __forceinline__ void combine_if_last(unsigned* done, int n_splits,
                                                const float* part_o, const float* part_lse,
                                                void* o, float* lse, size_t row0, int G,
                                                int o_bf16, Sync sync) {
  __shared__ int last_sh;
  __threadfence();  // this thread's partials are visible device-wide before the count
  sync();
  if (threadIdx.x == 0) {
    const unsigned prev = atomicAdd(done, 1u);
    const int last = prev + 1u == (unsigned)n_splits;
    if (last) {
      __threadfence();      // the other CTAs' partials are read after their counts
      atomicExch(done, 0u);  // ready for the next launch
    }
    last_sh = last;
  }
  sync();
  if (!last_sh) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int g = warp; g < G; g += NWARPS)
    merge_row<D, BATCH>(part_o, part_lse, o, lse, row0 + g, row0 + g, n_splits, o_bf16, lane);
}

}  // namespace
}  // namespace attn
