// rope.cu -- rotary positions of a batch's new tokens and the append of their keys and
// values to the cache, in one pass over the projections' outputs.
//
// For token t with position p and rotated pair i (frequency f_i, radians per position):
//   (x1, x2) -> amp * (x1 cos(p f_i) - x2 sin(p f_i), x1 sin(p f_i) + x2 cos(p f_i)),
// pairs (i, i + rot/2) in the half layout, (2i, 2i + 1) in the interleaved one; the head's
// dims past rot_dim pass through.  Every 16-byte chunk is read once and written once, so
// HBM bounds long batches and the launch bounds short ones.
//
// Angles.  p f_i in fp32 is off by 0.06 radians at p = 10^6, so the angle is kept as a
// fraction of a turn in 64-bit fixed point: f_i / 2 pi is taken to 2^-64 turns once per
// CTA (in fp64: its relative error, below 2^-52, is multiplied by the position), and the
// product with the 32-bit position wraps modulo one turn by itself, exactly.  The top 32 bits
// go to sincospi as a signed half turn (2^-25 of it, 2^-26 of a turn, rounded away).  fp64 per token instead would
// cost the few fp64 lanes of this GPU about as long as the copy itself.
#include <cmath>

#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float lo_f(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_f(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

// rotates the pairs (a.e, b.e) of two 16-byte chunks (half layout: b is the partner chunk)
__device__ __forceinline__ void rotate_half(uint4& a, uint4& b, const float2* cs) {
  uint32_t* pa = reinterpret_cast<uint32_t*>(&a);
  uint32_t* pb = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 c0 = cs[2 * e], c1 = cs[2 * e + 1];
    const float x0 = lo_f(pa[e]), x1 = hi_f(pa[e]), y0 = lo_f(pb[e]), y1 = hi_f(pb[e]);
    pa[e] = pack_bf16x2(x0 * c0.x - y0 * c0.y, x1 * c1.x - y1 * c1.y);
    pb[e] = pack_bf16x2(x0 * c0.y + y0 * c0.x, x1 * c1.y + y1 * c1.x);
  }
}
// rotates the four pairs inside one chunk (interleaved layout)
__device__ __forceinline__ void rotate_inter(uint4& a, const float2* cs) {
  uint32_t* pa = reinterpret_cast<uint32_t*>(&a);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 c = cs[e];
    const float x = lo_f(pa[e]), y = hi_f(pa[e]);
    pa[e] = pack_bf16x2(x * c.x - y * c.y, x * c.y + y * c.x);
  }
}

// One CTA takes up to kTokens consecutive tokens: their places in the cache (a chain of
// dependent loads) and their angles are found side by side, and the copies of all of them
// follow without a barrier between.  A work item is two chunks of one head: the two partners
// of the half layout, or two neighbours.  rot = 0 copies.
template <bool INTER, int kTokens>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const RopeArgs a) {
  __shared__ unsigned long long turn[128];       // f_i / 2 pi, units of 2^-64 turns
  __shared__ float2 cs[kTokens * 128];           // (cos, sin) * amp of each token's pairs
  __shared__ int place[kTokens], at[kTokens];    // cache row (-1: none, -2: no sequence), position
  const int half = a.rot / 2, t0 = blockIdx.x * kTokens, nt = min(kTokens, a.total - t0);
  for (int i = threadIdx.x; i < half; i += kThreads) {
    const double x = a.inv_freq[i] * 0.15915494309189535, y = fabs(x);  // 1 / (2 pi)
    // the fraction of |x|, which is exact (that of a small negative x would be rounded to 2^-54)
    const unsigned long long f = (unsigned long long)((y - floor(y)) * 18446744073709551616.0);
    turn[i] = x < 0 ? 0ull - f : f;
  }
  if ((int)threadIdx.x >= kThreads - nt) {
    // (the last threads, whose warp has no frequency to convert up to d = 256)
    const int s = kThreads - 1 - (int)threadIdx.x, t = t0 + s;
    // the token's sequence: the last b with cu[b] <= t (cu is non-decreasing)
    int b = t, i = 0, n = 1;
    bool live = t < a.B;
    if (a.cu_q) {
      int lo = 0, hi = a.B;  // cu[lo] <= t < cu[hi] (or t behind the last sequence)
      live = t >= a.cu_q[0] && t < a.cu_q[a.B];
      while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;  // (lo + hi may pass an int)
        if (a.cu_q[mid] <= t) lo = mid; else hi = mid;
      }
      b = lo;
      const int c0 = max(a.cu_q[b], 0);  // (clamped to [0, total], as the attention calls do)
      i = t - c0;
      n = min(a.cu_q[b + 1], a.total) - c0;
    }
    int row = -2;  // behind the last sequence: the token's rows are left as they are
    if (live) {
      const long long cap = (long long)a.kv.max_pages * a.kv.page_size;
      const long long j = (long long)a.kv_lens[b] - n + i;  // key index
      if (j < 0 || j >= cap) {
        atomicCAS(a.err, kErrNone, kErrBadShape);
        row = -1;
      } else {
        row = paged_row(a.kv, b, (int)j, a.err);
      }
      at[s] = a.positions ? a.positions[t] : (int)j;
    }
    place[s] = row;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int s = kTokens == 1 ? 0 : i / half, m = i - s * half;
    const unsigned long long w = turn[m] * (unsigned long long)(long long)at[s];
    const float x = (float)(int)(w >> 32) * 4.656612873077393e-10f;  // half turns in [-1, 1): 2^-31
    float sn, c;
    sincospif(x, &sn, &c);
    cs[s * 128 + m] = make_float2(c * a.amp, sn * a.amp);
  }
  __syncthreads();
  const int cpr = a.d / 8, rc = a.rot / 8;  // chunks of a head, rotated ones (rot % 16 == 0)
  const int n_q = a.q ? a.Hq : 0;
  const int ipr = cpr / 2;  // items of a head
  const int items = (n_q + 2 * a.Hkv) * ipr;
#pragma unroll 2
  for (int it = threadIdx.x; it < nt * items; it += kThreads) {
    const int s = kTokens == 1 ? 0 : it / items, in = it - s * items, t = t0 + s;
    const int h = in / ipr, x = in - h * ipr;
    const int row = place[s];
    const bool is_q = h < n_q, is_k = !is_q && h < n_q + a.Hkv;
    const int hk = is_q ? 0 : (is_k ? h - n_q : h - n_q - a.Hkv);
    if (row == -2 || (!is_q && row < 0)) continue;  // no sequence, or no place in the cache
    const uint16_t* src = is_q ? a.q + (size_t)t * a.q_stride + (size_t)h * a.d
                               : (is_k ? a.k + (size_t)t * a.k_stride + (size_t)hk * a.d
                                       : a.v + (size_t)t * a.v_stride + (size_t)hk * a.d);
    uint16_t* dst = is_q ? a.q_out + ((size_t)t * a.Hq + h) * a.d
                         : (is_k ? a.kc : a.vc) + ((size_t)row * a.Hkv + hk) * a.d;
    // the item's chunks: rotated partners (c, c + rc/2) first, then the rest two by two
    int c0, c1;
    if (!INTER && x < rc / 2) { c0 = x; c1 = x + rc / 2; }
    else { c0 = 2 * x; c1 = 2 * x + 1; }
    uint4 u0 = *reinterpret_cast<const uint4*>(src + c0 * 8), u1 = *reinterpret_cast<const uint4*>(src + c1 * 8);
    if (is_q || is_k) {
      const float2* c = cs + s * 128;
      if (INTER) {
        if (c0 < rc) rotate_inter(u0, c + c0 * 4);
        if (c1 < rc) rotate_inter(u1, c + c1 * 4);
      } else if (x < rc / 2) {
        rotate_half(u0, u1, c + c0 * 8);
      }
    }
    *reinterpret_cast<uint4*>(dst + c0 * 8) = u0;
    *reinterpret_cast<uint4*>(dst + c1 * 8) = u1;
  }
}

template <int kTokens>
cudaError_t launch_t(const RopeArgs& a, cudaStream_t stream) {
  const unsigned grid = (unsigned)((a.total + kTokens - 1) / kTokens);
  if (a.interleaved) rope_append_kernel<true, kTokens><<<grid, kThreads, 0, stream>>>(a);
  else rope_append_kernel<false, kTokens><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs& a, cudaStream_t stream) {
  // one token a CTA while that leaves SMs idle, else eight
  return a.total >= 8 * 152 * 2 ? launch_t<8>(a, stream) : launch_t<1>(a, stream);
}

}  // namespace attn
