// prefill_backward.cuh -- gradients of the prefill attention (causal or not, sliding window
// with sinks, GQA, fixed-length or packed batches; d = 64, 128).
//
// With P_ij = exp(scale q_i.k_j - lse_i) (0 where the mask admits nothing), g = dL/do,
//   dP_ij = g_i . v_j        D_i = g_i . o_i - dL/dlse_i
//   dS_ij = P_ij (dP_ij - D_i)
//   dV_j = sum_i P_ij g_i    dK_j = scale sum_i dS_ij q_i    dQ_i = scale sum_j dS_ij k_j,
// dK and dV summed over the query heads of a KV head's group.  Nothing but lse and D is
// kept from the forward pass: P is computed again.
//
// Two passes over the tiles, one whose CTAs own key blocks (dK, dV: four products a tile) and
// one whose CTAs own query blocks (dQ: three), instead of one pass of five products that adds
// dQ into global memory: every sum has one owner and a fixed order, so the same inputs give
// the same bits, no fp32 copy of dQ is zeroed, added to by atomics and converted, and the
// accumulators, S and dP of a 128 x 128 tile fill TMEM (512 columns) in either pass at
// d = 128; a third accumulator would not fit beside them.  Both passes are one kernel: with
//   the fixed pair F1, F2 and the streamed pair Y1, Y2
//     dK/dV pass:  F = K, V    Y = Q, g
//     dQ pass:     F = Q, g    Y = K, V
//   S = F1 Y1^T,  dP = F2 Y2^T,  [acc0 += P Y2,]  acc1 += dS Y1,
// rows of F are TMEM lanes, P and dS stay in TMEM as the A operands of the second products,
// and a Y tile serves K-major in the first product and MN-major in the second.
// In the dK/dV pass lse and D belong to columns: they ride in the products as a further step
// of 16 columns (ones beside K and V, -lse / scale and -D in three bf16 terms each beside Q
// and g), since reading them from shared memory would cost as many wavefronts as the MMA's
// own operands.
//
// Work.  A unit is one F tile (of one head); its items are the Y tiles its rows admit (of all
// heads of the group in the dK/dV pass).  The units' items form one list, which the CTAs (one
// per SM) cut into equal slices: neither causal triangles, the few key blocks of the sinks
// that every row sees, nor groups of odd sizes leave SMs idle.  A unit cut between CTAs
// goes out as fp32 partials, which the one that finishes last sums in slice order.
//
// Warps: 0-7 softmax (thread = row of F, 64 columns of an item), 8 / 9 S and dP with their F tiles, 10
// the second products, 11 the rings of Y1 and Y2.
#pragma once
#include <algorithm>
#include <cmath>

#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kT = 128;           // rows of a tile
constexpr int kMaxCtas = kBackwardCtas;
// A run of a unit's items costs its start and end (the F tiles' copy, the sums' way out, the sum of a
// cut unit's parts) beside its items: units of few items would otherwise fill some slices with
// nothing but starts and ends.  In rows of Y: 640 in the dK/dV pass, 128 in the dQ pass (of 64 to
// 768 and 128 to 384; 3314 rows without a window: 227 us, 235 with 192 and 384; eight packed sequences:
// 224 and 229).
constexpr int run_cost(bool kv, int ty) { return (kv ? 640 : 128) / ty; }
constexpr int kMinCost = 8;  // of a slice
// Rows of Y that a run sums in TMEM.  The tensor core's fp32 sums round towards zero, by up to 2^-23 of the sum for
// every 16 terms (2^-24 on average), so that a sum of 4.2 million terms of one sign came out 1.6 % short; a unit's
// longer part of a slice is cut into runs, 2^-12 of each left out at most, whose sums are added to nearest.  (Two
// terms are two sums a step.)
constexpr int run_rows(bool fine) { return fine ? 16384 : 32768; }

// TN: rows of a Y tile, the columns of an item's S and dP.
//   128, halved between the softmax warpgroups.  P and dS go back over dP, two dP beside one S: of
//     an item's two products the one that waits for the second products two items back is then the
//     one that the softmax needs last, after its exponentials.
//   64 (dK/dV pass, d = 128, whose sums leave 256 columns): the warpgroups take an item each in turn;
//     one S, one dP and two of P and dS, so that the next S waits for the softmax's load only.  A
//     product of 64 columns re-reads as much of F for half of the work (49 cycles a step, bound by
//     shared memory, against 65 for 128 columns); elsewhere items of 64 were slower (d = 64, 2 x 16
//     heads of 4096, not causal: 494 us in the dK/dV pass alone so, against 434).
// FINE: P and dS as two bf16 terms each (2^-17 of them left out, not 2^-8), both multiplied by the same rows
// of Y, in sequences of few pairs (backward_two_terms).  Items of 64 columns, whose terms have columns of
// their own: one buffer of them where the dK/dV pass's sums leave no room for two.
template <int D, bool KV, bool FINE>
struct BwdCfg {
  static constexpr int TN = ((D == 128 && KV) || FINE) ? 64 : 128;
  static constexpr bool kSep = TN == 64;                   // P and dS in columns of their own, not over dP
  static constexpr int NS = 1;                             // S buffers
  static constexpr int ND = kSep ? 1 : 2;                  // dP buffers
  static constexpr int kArrive = TN == 64 ? 4 : 8;         // softmax warps of an item
  static constexpr int kPanels = D / 64;
  static constexpr int kFPanel = kT * 128;
  static constexpr int kFTile = kPanels * kFPanel;
  static constexpr int kYPanel = TN * 128;
  static constexpr int kYTile = kPanels * kYPanel;
  static constexpr int kSt1 = D == 64 ? 4 : (KV ? 5 : 3);  // ring of Y1
  static constexpr int kSt2 = D == 64 ? 4 : (KV ? 4 : 2);  // ring of Y2
  static constexpr int kY1Off = 2 * kFTile;
  static constexpr int kY2Off = kY1Off + kSt1 * kYTile;
  // columns beside the tiles, 16 bytes a row: lse beside Q, D beside g, ones beside K and V, and zeros,
  // the second eight columns of all of them.  In the dQ pass, whose rows are a thread's own, at d = 64
  // only, where the softmax warps' work is longest: an addition fewer a pair of columns, no loads of stat, against a step more a
  // product (2 x 16 heads of 4096, not causal: 429 us without, 417 so)
  static constexpr bool kRowExt = !KV && D == 64;
  static constexpr int kExt = KV ? TN * 16 : (kRowExt ? kT * 16 : 0);
  static constexpr int kExtSlots = KV ? 5 : 1;
  static constexpr int kOnes = KV || kRowExt ? kT * 16 : 0;
  static constexpr int kExt1Off = kY2Off + kSt2 * kYTile;
  static constexpr int kExt2Off = kExt1Off + kExtSlots * kExt;
  static constexpr int kOnesOff = kExt2Off + kExtSlots * kExt;
  static constexpr int kZeroOff = kOnesOff + kOnes;
  static constexpr int kBarOff = kZeroOff + kOnes;
  static constexpr int kNumBars = 2 * kSt1 + 2 * kSt2 + 4 + 2 + NS + 2 + ND + 4 + 5;
  static constexpr int kSmem = kBarOff + kNumBars * 8 + 16 + 1024;  // (16: TMEM address, abort and last flags)
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static constexpr uint32_t kAcc1 = KV ? D : 0;  // TMEM columns; acc0 at 0
  static constexpr uint32_t kS = kAcc1 + D;
  static constexpr uint32_t kDP = kS + NS * TN;
  // P and dS of an item (two buffers): kP + buffer * kPStep
  static constexpr uint32_t kP = kSep ? kDP + ND * TN : kDP;
  static constexpr uint32_t kPCols = FINE ? 2 * TN : TN;  // FINE: the second terms behind the first ones
  static constexpr bool kOneP = FINE && KV && D == 128;
  static constexpr uint32_t kPStep = kOneP ? 0 : kPCols;
  static_assert(kP + kPStep + kPCols <= 512 && kDP + ND * TN <= 512, "TMEM budget");
  static constexpr int kThreads = 384;
};

// Extent of a unit: which Y tiles its F tile meets.  SEL: none for sequences of the other form (FINE or not).
struct Unit {
  int Sq, Skv, qbase, kbase;  // rows and keys of the sequence, first row of q, first row of k
  long long off;              // key index of row i: i + off
  int nt, t0;                 // Y tiles, dK/dV pass: from t0 on; dQ pass: by the tile list
  TileList tl;
};
template <int TN, bool KV, bool FINE, bool SEL>
__device__ __forceinline__ Unit unit_of(const BackwardArgs& a, int b, int x) {
  Unit u;
  const SeqExtent e = seq_extent(b, a.Sq, a.Skv, a.cu_q, a.kv_lens, a.total_q);
  u.Sq = e.Sq; u.Skv = e.Skv;
  u.qbase = a.cu_q ? e.qbase : b * a.Sq;
  u.kbase = b * a.Skv;
  u.off = (long long)u.Skv - u.Sq;
  u.nt = 0; u.t0 = 0;
  u.tl = TileList{0x7FFFFFFF, 0};
  // (a fixed-length call has sequences, and lists, of one form only)
  if (SEL && a.cu_q && backward_two_terms(u.Sq, u.Skv, a.causal, a.window, a.n_sink) != FINE) return u;
  const int f0 = x * kT;
  if constexpr (KV) {
    if (f0 >= u.Skv) return u;
    const int last = min(u.Skv, f0 + kT) - 1;
    const long long lo = a.causal ? max(0LL, f0 - u.off) : 0LL;
    long long hi = u.Sq;
    if (a.window > 0 && f0 >= a.n_sink) hi = min(hi, last + (long long)a.window - u.off);
    if (hi <= lo) return u;
    u.t0 = (int)(lo / TN);
    u.nt = (int)((hi + TN - 1) / TN) - u.t0;
  } else {
    if (f0 >= u.Sq) return u;
    const int last = min(u.Sq, f0 + kT) - 1;
    const long long hi = a.causal ? min((long long)u.Skv, max(0LL, last + u.off + 1)) : u.Skv;
    const int n = (int)((hi + TN - 1) / TN);
    u.tl = tile_list(f0 + u.off, n, a.window, a.n_sink, u.Skv, TN);
    u.nt = tile_list_len(u.tl, n);
  }
  return u;
}
template <bool KV>
__device__ __forceinline__ int unit_items(const BackwardArgs& a, const Unit& u) {
  return KV ? u.nt * (a.Hq / a.Hkv) : u.nt;
}
template <int TN, bool KV>
__device__ __forceinline__ int unit_cost(int items) {
  return items > 0 ? items + run_cost(KV, TN) : 0;
}
// Groups (sequence, F tile) of the pass: each holds a unit per head.
__host__ __device__ __forceinline__ int f_tiles(const BackwardArgs& a, bool kv) {
  return ((kv ? a.Skv : a.Sq) + kT - 1) / kT;
}
// The slices' share of the units' costs.
__device__ __forceinline__ int slice_cost(int total, int ctas) { return max((total + ctas - 1) / ctas, kMinCost); }

// ------------------------------------------------------------------ rows' lse and D, the item list
constexpr int kPrepThreads = 256;

__device__ __forceinline__ float dot8(uint4 a, uint4 b) {
  float s0 = 0.f, s1 = 0.f;
  fma_bf16x2_f32(a.x, b.x, s0, s1);
  fma_bf16x2_f32(a.y, b.y, s0, s1);
  fma_bf16x2_f32(a.z, b.z, s0, s1);
  fma_bf16x2_f32(a.w, b.w, s0, s1);
  return s0 + s1;
}
__device__ __forceinline__ float dot8(uint4 a, float4 b0, float4 b1) {
  auto lo = [](uint32_t x) { return __uint_as_float(x << 16); };
  auto hi = [](uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); };
  float s0 = lo(a.x) * b0.x, s1 = hi(a.x) * b0.y;
  s0 = fmaf(lo(a.y), b0.z, s0); s1 = fmaf(hi(a.y), b0.w, s1);
  s0 = fmaf(lo(a.z), b1.x, s0); s1 = fmaf(hi(a.z), b1.y, s1);
  s0 = fmaf(lo(a.w), b1.z, s0); s1 = fmaf(hi(a.w), b1.w, s1);
  return s0 + s1;
}
// x as three bf16 terms (2^-24 of it left out)
__device__ __forceinline__ void split3(float x, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = pack_bf16x2(x, 0.f) & 0xFFFFu;
  const float r1 = x - __uint_as_float(hi << 16);
  mid = pack_bf16x2(r1, 0.f) & 0xFFFFu;
  lo = pack_bf16x2(r1 - __uint_as_float(mid << 16), 0.f) & 0xFFFFu;
}

// Exclusive prefix of the groups' costs (all heads of a group) by one CTA; pre[n] the total.
template <int TN, bool KV, bool FINE>
__device__ void scan_costs(const BackwardArgs& a, int* pre) {
  __shared__ int sums[kPrepThreads / 32];
  const int nx = f_tiles(a, KV), n = a.B * nx, H = KV ? a.Hkv : a.Hq;
  const int per = (n + kPrepThreads - 1) / kPrepThreads;
  const int lo = min(n, (int)threadIdx.x * per), hi = min(n, lo + per);
  int s = 0;
  auto cost = [&](int g) { return unit_cost<TN, KV>(unit_items<KV>(a, unit_of<TN, KV, FINE, true>(a, g / nx, g % nx))) * H; };
  for (int g = lo; g < hi; ++g) s += cost(g);
  int incl = s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int at = incl - s;
  for (int w = 0; w < warp; ++w) at += sums[w];
  for (int g = lo; g < hi; ++g) {
    pre[g] = at;
    at += cost(g);
  }
  if (hi == n && lo < n) pre[n] = at;
  if (n == 0 && threadIdx.x == 0) pre[0] = 0;
}

// Zeros for the gradients of units without items: keys that no row sees, rows that see no key and,
// with `fill`, rows of no sequence and slots behind a sequence's keys.  CTA c of n.
template <int D, bool KV>
__device__ void zero_units(const BackwardArgs& a, int c, int n) {
  const int nx = f_tiles(a, KV), n_groups = a.B * nx, H = KV ? a.Hkv : a.Hq;
  constexpr int kRows = 16;  // of a CTA's turn
  for (int gc = c; gc < n_groups * (kT / kRows); gc += n) {
    const int g = gc / (kT / kRows), b = g / nx, x = g - b * nx;
    const Unit u = unit_of<kT, KV, false, false>(a, b, x);
    if (unit_items<KV>(a, u) > 0) continue;
    const int f0 = x * kT + gc % (kT / kRows) * kRows;
    const int rows = min(kRows, (KV ? (a.fill ? a.Skv : u.Skv) : u.Sq) - f0);
    const size_t at = ((size_t)(KV ? u.kbase : u.qbase) + f0) * H * D;
    const long long w = (long long)H * (D / 8);
    for (long long i = threadIdx.x; i < rows * w; i += kPrepThreads) {
      if (KV) {
        reinterpret_cast<uint4*>(a.dk + at)[i] = make_uint4(0, 0, 0, 0);
        reinterpret_cast<uint4*>(a.dv + at)[i] = make_uint4(0, 0, 0, 0);
      } else {
        reinterpret_cast<uint4*>(a.dq + at)[i] = make_uint4(0, 0, 0, 0);
      }
    }
  }
  if (!KV && a.cu_q && a.fill) {
    const long long w = (long long)a.Hq * (D / 8), step = (long long)n * kPrepThreads;
    const int c0 = min(max(a.cu_q[0], 0), a.total_q), c1 = min(max(a.cu_q[a.B], c0), a.total_q);
    for (long long i = (long long)c * kPrepThreads + threadIdx.x; i < (c0 + (long long)a.total_q - c1) * w; i += step)
      reinterpret_cast<uint4*>(a.dq)[i < c0 * w ? i : i + (c1 - c0) * w] = make_uint4(0, 0, 0, 0);
  }
}
constexpr int kZeroCtas = 304;
// The item lists: dK/dV and dQ of the sequences of two terms, then of those of one.
constexpr int kLists = 4;
constexpr int list_of(bool kv, bool fine) { return (fine ? 0 : 2) + (kv ? 0 : 1); }

// D / 8 lanes to a row of a head, kPrepRows consecutive rows of it in flight: a row is 128 or 256 bytes, so
// that nothing is lost by reading a head's rows and what is written, by head, lies side by side.
constexpr int kPrepRows = 4;
constexpr int prep_rows(int d) { return kPrepThreads / (d / 8) * kPrepRows; }  // of a CTA
template <int D, bool OBF16>
__global__ void __launch_bounds__(kPrepThreads) backward_prep_kernel(const __grid_constant__ BackwardArgs a) {
  if (blockIdx.x < kLists) {
    const int i = (int)blockIdx.x;  // list_of
    // a sequence above max_sq is reported, as the positions of its first rows would be taken for the last ones
    if (i == 0 && a.cu_q)
      for (int b = threadIdx.x; b < a.B; b += kPrepThreads) {
        const int c0 = min(max(a.cu_q[b], 0), a.total_q), c1 = min(a.cu_q[b + 1], a.total_q);
        if (c1 - c0 > a.Sq) atomicCAS(a.err, kErrNone, kErrBadShape);
      }
    if (!(a.forms & (i < 2 ? kTwoTerms : kOneTerm))) return;
    if (i == 0) scan_costs<BwdCfg<D, true, true>::TN, true, true>(a, a.pre[0]);
    else if (i == 1) scan_costs<BwdCfg<D, false, true>::TN, false, true>(a, a.pre[1]);
    else if (i == 2) scan_costs<BwdCfg<D, true, false>::TN, true, false>(a, a.pre[2]);
    else scan_costs<BwdCfg<D, false, false>::TN, false, false>(a, a.pre[3]);
    for (int c = threadIdx.x; c < kMaxCtas; c += kPrepThreads) a.joined[i * kMaxCtas + c] = 0;
    return;
  }
  if (blockIdx.x < kLists + kZeroCtas) {
    zero_units<D, true>(a, (int)blockIdx.x - kLists, kZeroCtas);
    zero_units<D, false>(a, (int)blockIdx.x - kLists, kZeroCtas);
    return;
  }
  constexpr int L = D / 8;
  const int h = ((int)blockIdx.x - kLists - kZeroCtas) % a.Hq;
  const int row0 = ((int)blockIdx.x - kLists - kZeroCtas) / a.Hq * prep_rows(D) + (int)threadIdx.x / L * kPrepRows;
  const int c = threadIdx.x % L;
  float s[kPrepRows];
#pragma unroll
  for (int k = 0; k < kPrepRows; ++k) {
    // (every lane takes part in the sums)
    const size_t at = ((size_t)min(row0 + k, a.total_q - 1) * a.Hq + h) * D + c * 8;
    const uint4 g = __ldg(reinterpret_cast<const uint4*>(a.dout + at));
    if constexpr (OBF16) {
      s[k] = dot8(g, __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.o) + at)));
    } else {
      const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.o) + at);
      s[k] = dot8(g, __ldg(p), __ldg(p + 1));
    }
  }
#pragma unroll
  for (int k = 0; k < kPrepRows; ++k) {
#pragma unroll
    for (int o = 1; o < L; o <<= 1) s[k] += __shfl_xor_sync(0xFFFFFFFFu, s[k], o);
  }
  // lane k of a row's lanes writes the k-th row's
  float D_i = s[0];
#pragma unroll
  for (int k = 1; k < kPrepRows; ++k) D_i = c == k ? s[k] : D_i;
  const int row = row0 + c;
  if (c >= kPrepRows || row >= a.total_q) return;
  // [B][Hq][Sq], or packed [Hq][total_q]
  const size_t i = a.cu_q ? (size_t)h * a.total_q + row
                          : ((size_t)(row / a.Sq) * a.Hq + h) * a.Sq + row % a.Sq;
  const float lse = a.lse[i];
  if (a.dlse) D_i -= a.dlse[i];
  // a row that saw no key (lse = -inf) takes no part
  a.stat[i] = make_float2(lse == -INFINITY ? INFINITY : lse * kLog2e, D_i);
  float x = -lse / a.scale;
  if (x > 1e38f || x < -1e38f) x = -1e38f;
  uint32_t l0, l1, l2, d0, d1, d2;
  split3(x, l0, l1, l2);
  split3(-D_i, d0, d1, d2);
  a.ext1[i] = make_uint4(l0 | l1 << 16, l2, 0u, 0u);
  a.ext2[i] = make_uint4(d0 | d1 << 16, d2, 0u, 0u);
}

// ------------------------------------------------------------------ the two passes
// The last group of [lo, hi) that starts at or before pos (pre[lo] <= pos < pre[hi]): those without items start
// where the next does.  By a whole warp, first `step` groups apart.
__device__ __forceinline__ int group_at(const int* pre, int lo, int hi, int pos, int lane, int step) {
  while (hi - lo > 1) {
    const int p = min(lo + (lane + 1) * step, hi);
    const unsigned over = __ballot_sync(0xFFFFFFFFu, p >= hi || pre[p] > pos);
    const int k = over ? __ffs(over) - 1 : 32;  // probes at or before pos
    hi = k < 32 ? min(lo + (k + 1) * step, hi) : hi;
    lo = lo + k * step;
    step = max(1, (hi - lo) / 32);
  }
  return lo;
}
// A run: items [i0, i0 + n) of the unit of head h in group (b, x), at most run_rows of Y; n = 0: none.
struct Run {
  Unit u;
  int b, x, h, i0, n, cnt, first;  // cnt: items of the unit, first: the place of its first one
};
// The items of a slice in order, run by run of one unit.
template <int TN, bool KV, bool FINE, bool SEL>
struct Walk {
  const BackwardArgs& a;
  int per, pos, end;  // a slice's share of the list of costs, place in it, end of the slice
  int g, g0;     // group, its place
  Run at;        // of the group: u, b, x, cnt
  __device__ __forceinline__ const int* pre() const { return a.pre[list_of(KV, FINE)]; }
  __device__ __forceinline__ Walk(const BackwardArgs& a_, int cta, int ctas, int lane) : a(a_) {
    const int n_groups = a.B * f_tiles(a, KV);
    const int total = pre()[n_groups];
    per = slice_cost(total, ctas);
    pos = (int)min((long long)total, (long long)cta * per);
    end = min(total, pos + per);
    g = g0 = 0;
    if (pos >= end) return;
    g = group_at(pre(), 0, n_groups, pos, lane, max(1, n_groups / 32));
    enter();
  }
  __device__ __forceinline__ void enter() {
    const int nx = f_tiles(a, KV);
    at.b = g / nx;
    at.x = g - at.b * nx;
    at.u = unit_of<TN, KV, FINE, SEL>(a, at.b, at.x);
    at.cnt = unit_items<KV>(a, at.u);
    g0 = pre()[g];
  }
  // The next run.  Roles take it while they still work on the one before: a new group costs
  // dependent loads and divisions.
  __device__ __forceinline__ Run next() {
    const int H = KV ? a.Hkv : a.Hq;
    at.n = 0;
    while (pos < end) {
      while (pos >= g0 + unit_cost<TN, KV>(at.cnt) * H) {
        ++g;
        enter();
        if (at.cnt > 0) continue;
        // groups without items, of which there may be many: tiles behind short sequences' ends, sequences of the
        // other form (one by one, 4000 sequences of 8 rows between two of 2000 took 40 ms)
        g = group_at(pre(), g, a.B * f_tiles(a, KV), pos, (int)threadIdx.x & 31, 1);
        enter();
      }
      const int cost = unit_cost<TN, KV>(at.cnt);
      at.h = (pos - g0) / cost;
      const int from = pos - g0 - at.h * cost;  // of the unit's cost
      at.first = g0 + at.h * cost + run_cost(KV, TN);
      at.i0 = max(0, from - run_cost(KV, TN));
      const int to = min(min(cost, from + end - pos), at.i0 + run_rows(FINE) / TN + run_cost(KV, TN));
      pos += to - from;
      at.n = max(0, to - run_cost(KV, TN)) - at.i0;
      if (at.n > 0) break;
    }
    return at;
  }
};

// Y tile of an item of a run: its first row (query rows of head h, or keys), and the head.
template <int TN, bool KV>
struct ItemWalk {
  int h, t, row0;
  __device__ __forceinline__ ItemWalk(const BackwardArgs& a, const Run& r) : h(0), t(0), row0(0) {
    if (r.n == 0) return;
    const int G = a.Hq / a.Hkv;
    if constexpr (KV) {
      const int q = r.i0 / r.u.nt;
      h = r.h * G + q;
      t = r.i0 - q * r.u.nt;
      row0 = (r.u.t0 + t) * TN;
    } else {
      h = r.h / G;
      t = r.i0;
      row0 = tile_list_key(r.u.tl, t) * TN;
    }
  }
  __device__ __forceinline__ void step(const Unit& u) {
    ++t;
    if constexpr (KV) {
      if (t == u.nt) {
        t = 0;
        ++h;
      }
      row0 = (u.t0 + t) * TN;
    } else {
      row0 = tile_list_key(u.tl, t) * TN;
    }
  }
};

// the lowest n of 32 bits, n clamped to [0, 32]
__device__ __forceinline__ uint32_t bits_below(int n) { return n >= 32 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << n) - 1u); }
// bf16 pairs: element i stays where bit i is set, else becomes 0
template <int N>
__device__ __forceinline__ void keep_bits(uint32_t* t, uint32_t in) {
#pragma unroll
  for (int c = 0; c < N; ++c) {
    t[c] = (in & (1u << (2 * c))) ? t[c] : t[c] & 0xFFFF0000u;
    t[c] = (in & (2u << (2 * c))) ? t[c] : t[c] & 0x0000FFFFu;
  }
}

// what their rounding to a pair of bf16 left of x0 and x1
__device__ __forceinline__ uint32_t rest_bf16x2(uint32_t t, float x0, float x1) {
  return pack_bf16x2(x0 - __uint_as_float(t << 16), x1 - __uint_as_float(t & 0xFFFF0000u));
}
// 8 columns of 4 rows, one row a lane (unit c: columns 8 c ..), to one column unit a lane: lane i of
// four gets unit i of each row.
__device__ __forceinline__ void transpose4(uint4 (&u)[4], int lane) {
#pragma unroll
  for (int k = 1; k <= 2; ++k) {
    const bool up = lane & k;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c & k) continue;
      uint4 &lo = u[c], &hi = u[c | k];
      uint4 x = up ? lo : hi;  // what goes to the lane k away
      x.x = __shfl_xor_sync(0xFFFFFFFFu, x.x, k);
      x.y = __shfl_xor_sync(0xFFFFFFFFu, x.y, k);
      x.z = __shfl_xor_sync(0xFFFFFFFFu, x.z, k);
      x.w = __shfl_xor_sync(0xFFFFFFFFu, x.w, k);
      if (up) lo = x;
      else hi = x;
    }
  }
}

// The items whose tiles (or lse / D columns) a warp still has to bring.
template <int TN, bool KV, bool FINE, bool SEL>
struct Stream {
  Walk<TN, KV, FINE, SEL> w;
  Run r;
  ItemWalk<TN, KV> y;
  int m, it;
  __device__ __forceinline__ Stream(const BackwardArgs& a, const Walk<TN, KV, FINE, SEL>& w_)
      : w(w_), r(w.next()), y(a, r), m(0), it(0) {}
  __device__ __forceinline__ void step(const BackwardArgs& a) {
    ++it;
    if (++m < r.n) {
      y.step(r.u);
      return;
    }
    m = 0;
    r = w.next();
    y = ItemWalk<TN, KV>(a, r);
  }
};

// One CTA's slice of a pass: `cta` of `ctas`, whose partials start at slot `slot0`.  PK: a packed batch.
template <int D, bool KV, bool PK, bool FINE>
__device__ __forceinline__ void backward_pass(const BackwardArgs& a, int cta, int ctas, int slot0) {
  using C = BwdCfg<D, KV, FINE>;
  using W = Walk<C::TN, KV, FINE, PK>;
  using S = Stream<C::TN, KV, FINE, PK>;
  constexpr int NS = C::NS, ND = C::ND, TN = C::TN;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full1 = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* empty1 = full1 + C::kSt1;
  uint64_t* full2 = empty1 + C::kSt1;
  uint64_t* empty2 = full2 + C::kSt2;
  uint64_t* fullF = empty2 + C::kSt2;  // [2] F tiles
  uint64_t* emptyF = fullF + 2;
  // S and dP computed: two each whatever the buffers, as a warpgroup may wait for every other item
  uint64_t* bar_S = emptyF + 2;
  uint64_t* bar_Sr = bar_S + 2;        // [NS] S read
  uint64_t* bar_dP = bar_Sr + NS;
  uint64_t* bar_dPr = bar_dP + 2;      // [ND] dP read (where P and dS lie over it: they are used up)
  uint64_t* bar_P = bar_dPr + ND;      // [2] P and dS stored
  uint64_t* bar_Pr = bar_P + 2;        // [2] P and dS used up
  uint64_t* bar_acc = bar_Pr + 2;      // a run's sums complete
  uint64_t* bar_accr = bar_acc + 1;    // they are read
  uint64_t* bar_out = bar_accr + 1;    // a partial is written
  uint64_t* bar_last = bar_out + 1;    // last_flag is set
  uint64_t* bar_go = bar_last + 1;     // a run's last second product is issued
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_go + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* last_flag = abort_flag + 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kSt1; ++s) { mbar_init(&full1[s], 1); mbar_init(&empty1[s], 1); }
    for (int s = 0; s < C::kSt2; ++s) { mbar_init(&full2[s], 1); mbar_init(&empty2[s], 1); }
    for (int s = 0; s < 2; ++s) { mbar_init(&fullF[s], 1); mbar_init(&emptyF[s], 1); }
    for (int s = 0; s < NS; ++s) mbar_init(&bar_Sr[s], C::kArrive);
    for (int s = 0; s < ND; ++s) mbar_init(&bar_dPr[s], C::kSep ? C::kArrive : 1);
    for (int s = 0; s < 2; ++s) { mbar_init(&bar_S[s], 1); mbar_init(&bar_dP[s], 1); }
    for (int s = 0; s < 2; ++s) { mbar_init(&bar_P[s], C::kArrive); mbar_init(&bar_Pr[s], 1); }
    mbar_init(bar_acc, 1);
    mbar_init(bar_accr, 8);
    mbar_init(bar_out, 8);
    mbar_init(bar_last, 1);
    mbar_init(bar_go, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if constexpr (KV || C::kRowExt) {
    for (int i = threadIdx.x; i < kT; i += C::kThreads) {
      *reinterpret_cast<uint4*>(smem + C::kOnesOff + i * 16) = make_uint4(0x3F803F80u, 0x00003F80u, 0, 0);
      *reinterpret_cast<uint4*>(smem + C::kZeroOff + i * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const W start(a, cta, ctas, lane);  // (a chain of dependent loads: made once)
  W w = start;
  Run run = w.next();
  if (warp == 8 || warp == 9) {
    // ---- first products: S = F1 Y1^T (warp 8), dP = F2 Y2^T (warp 9), and their F tiles ----
    constexpr uint32_t idesc = idesc_bf16_f32(128, TN, 0, 0);
    const bool first = warp == 8;
    const CUtensorMap* map = KV ? (first ? &a.tm_k : &a.tm_v) : (first ? &a.tm_q : &a.tm_do);
    uint8_t* sF = smem + (first ? 0 : C::kFTile);
    uint64_t *fF = fullF + (first ? 0 : 1), *eF = emptyF + (first ? 0 : 1);
    uint64_t* full = first ? full1 : full2;
    uint64_t *done = first ? bar_S : bar_dP, *freed = first ? bar_Sr : bar_dPr;
    const int stages = first ? C::kSt1 : C::kSt2, bufs = first ? NS : ND;
    const uint64_t df = smem_desc(smem_u32(sF), 16, 1024, kSwizzle128B);
    const uint64_t dy = smem_desc(smem_u32(smem + (first ? C::kY1Off : C::kY2Off)), 16, 1024, kSwizzle128B);
    const uint32_t out = tmem + (first ? C::kS : C::kDP);
    const uint32_t ext = smem_u32(smem + (first ? C::kExt1Off : C::kExt2Off)), zero = smem_u32(smem + C::kZeroOff);
    const uint64_t d1 = smem_desc(smem_u32(smem + C::kOnesOff), C::kOnes, 128, kSwizzleNone);
    if (lane == 0) tma_prefetch_desc(map);
    // the lse / D columns of an item (a tensor or bulk copy of them would take the copy engine as long
    // as a tile: 300 to 400 cycles whatever its size)
    S ex(a, start);
    auto load_ext = [&] {
      if constexpr (KV) {
        if (ex.r.n > 0) {
          const size_t i = PK ? (size_t)ex.y.h * a.total_q + ex.r.u.qbase + ex.y.row0
                                  : ((size_t)ex.r.b * a.Hq + ex.y.h) * a.Sq + ex.y.row0;
          const uint4* src = (first ? a.ext1 : a.ext2) + i;
          const uint32_t dst = ext + ex.it % C::kExtSlots * C::kExt;
#pragma unroll
          for (int k = 0; k < TN; k += 32) cp_async16(dst + (k + lane) * 16, src + k + lane, 16);
          ex.step(a);
        }
        cp_async_commit();
      }
    };
    // The next item's columns are whole for the tensor core, those three items on are on their way: after
    // item `it` is issued, into the slot of it - 2, whose product is done, as `it` waited for a buffer
    // (with two of them for that of it - 2, else for it - 1).
    auto next_ext = [&] {
      if constexpr (KV) {
        load_ext();
        cp_async_wait<2>();
        fence_proxy_async_smem();
        __syncwarp();
      }
    };
    load_ext();
    load_ext();
    next_ext();
    int it = 0, n_run = 0;
    bool ok = true;
    while (ok && run.n > 0) {
      if (!mbar_wait_warp(eF, ((uint32_t)n_run & 1u) ^ 1u, a.err, abort_flag)) break;
      constexpr bool packed = !KV && PK;
      mbar_arrive_expect_tx_e(fF, C::kFTile);
      tma_load_5d_e(sF, map, fF, 0, packed ? run.u.qbase + run.x * kT : run.x * kT, 0, run.h, packed ? 0 : run.b);
      if constexpr (C::kRowExt) {
        // (its rows past the sequence's, anything, belong to rows that are not written)
        const size_t i = PK ? (size_t)run.h * a.total_q + run.u.qbase + run.x * kT
                            : ((size_t)run.b * a.Hq + run.h) * a.Sq + run.x * kT;
        const uint4* src = (first ? a.ext1 : a.ext2) + i;
#pragma unroll
        for (int k = 0; k < kT; k += 32) cp_async16(ext + (k + lane) * 16, src + k + lane, 16);
        cp_async_commit();
      }
      const int n = run.n;
      run = w.next();
      if constexpr (C::kRowExt) {
        cp_async_wait<0>();
        fence_proxy_async_smem();
        __syncwarp();
      }
      ok = mbar_wait_warp(fF, (uint32_t)n_run & 1u, a.err, abort_flag);
      // behind the run before: its sums go out under these products, not after them
      if (ok && n_run > 0) ok = mbar_wait_warp(bar_go, (uint32_t)(n_run - 1) & 1u, a.err, abort_flag);
      for (int m = 0; ok && m < n; ++m, ++it) {
        const int s = it % stages, buf = it % bufs;
        const uint32_t ph_f = (uint32_t)(it / stages) & 1u, ph_b = ((uint32_t)(it / bufs) & 1u) ^ 1u;
        // both at once, one by one only where they are not ready
        const bool r0 = mbar_test(&full[s], ph_f), r1 = mbar_test(&freed[buf], ph_b);
        if (!__all_sync(0xFFFFFFFFu, r0 & r1)) {
          ok = mbar_wait_warp(&freed[buf], ph_b, a.err, abort_flag) &&
               mbar_wait_warp(&full[s], ph_f, a.err, abort_flag);
          if (!ok) break;
        }
        tc_fence_after();
        const uint64_t y = dy + (uint64_t)((s * C::kYTile) >> 4);
        const uint32_t d = out + buf * TN;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss_e(d, df + (uint64_t)(((kk >> 2) * C::kFPanel + (kk & 3) * 32) >> 4),
                   y + (uint64_t)(((kk >> 2) * C::kYPanel + (kk & 3) * 32) >> 4), idesc, kk > 0 ? 1u : 0u);
        if constexpr (KV) {
          const uint32_t e = ext + it % C::kExtSlots * C::kExt;
          mma_ss_e(d, d1, smem_desc(e, zero - e, 128, kSwizzleNone), idesc, 1u);
        } else if constexpr (C::kRowExt) {
          mma_ss_e(d, smem_desc(ext, zero - ext, 128, kSwizzleNone), d1, idesc, 1u);
        }
        mma_commit_e(&done[it & 1]);
        if (!KV && !first) mma_commit_e(&empty2[s]);
        if (m == n - 1) mma_commit_e(eF);
        next_ext();  // (of item it + 1, off the way from one product to the next)
      }
      ++n_run;
    }
    cp_async_wait<0>();
    // (aborted: the last copy lands before shared memory is released)
    if (!ok && n_run > 0) mbar_wait(fF, (uint32_t)(n_run - 1) & 1u, nullptr, nullptr, 100000000ull);
  } else if (warp == 10) {
    // ---- second products: acc0 += P Y2 (dV), acc1 += dS Y1 ----
    constexpr uint32_t idesc = idesc_bf16_f32(128, D, 0, 1);
    const uint64_t my1 = smem_desc(smem_u32(smem + C::kY1Off), C::kYPanel, 1024, kSwizzle128B);
    const uint64_t my2 = smem_desc(smem_u32(smem + C::kY2Off), C::kYPanel, 1024, kSwizzle128B);
    // A in TMEM, 16 rows of Y at a time (8 columns; of each half of dP's where it lies over dP); Y
    // MN-major
    auto issue = [&](uint32_t acc, uint32_t p, uint64_t y, bool fresh) {
#pragma unroll
      for (int kk = 0; kk < TN / 16; ++kk)
        mma_ts_e(tmem + acc, p + (kk >> 2) * 64 + (kk & 3) * 8, y + (uint64_t)(kk * (2048 >> 4)), idesc,
                 (!fresh || kk > 0) ? 1u : 0u);
    };
    int it = 0, n_run = 0;
    bool ok = true;
    while (ok && run.n > 0) {
      const int n = run.n;
      run = w.next();
      if (n_run > 0) ok = mbar_wait_warp(bar_accr, (uint32_t)(n_run - 1) & 1u, a.err, abort_flag);
      for (int m = 0; ok && m < n; ++m, ++it) {
        const int s1 = it % C::kSt1, s2 = it % C::kSt2, buf = it & 1;
        const uint32_t p = tmem + C::kP + buf * C::kPStep;
        // (dP is done where dS is stored, so g's tile is whole)
        ok = mbar_wait_warp(&bar_P[buf], (uint32_t)(it >> 1) & 1u, a.err, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if constexpr (KV) {
          issue(0, p, my2 + (uint64_t)((s2 * C::kYTile) >> 4), m == 0);
          if constexpr (FINE) issue(0, p + TN, my2 + (uint64_t)((s2 * C::kYTile) >> 4), false);
          mma_commit_e(&empty2[s2]);
        }
        issue(C::kAcc1, p + (KV ? 32 : 0), my1 + (uint64_t)((s1 * C::kYTile) >> 4), m == 0);
        if constexpr (FINE) issue(C::kAcc1, p + TN + (KV ? 32 : 0), my1 + (uint64_t)((s1 * C::kYTile) >> 4), false);
        mma_commit_e(C::kSep ? &bar_Pr[buf] : &bar_dPr[buf]);
        mma_commit_e(&empty1[s1]);
        if (m == n - 1) {
          mma_commit_e(bar_acc);
          if (lane == 0) mbar_arrive(bar_go);
        }
      }
      ++n_run;
    }
  } else if (warp == 11) {
    // ---- the rings of Y1 and Y2, each slot filled as soon as it is free ----
    const CUtensorMap* my1 = KV ? (TN == 64 ? &a.tm_q64 : &a.tm_q) : (TN == 64 ? &a.tm_k64 : &a.tm_k);
    const CUtensorMap* my2 = KV ? (TN == 64 ? &a.tm_do64 : &a.tm_do) : (TN == 64 ? &a.tm_v64 : &a.tm_v);
    S st[2] = {S(a, start), S(a, start)};
    if (lane == 0) {
      tma_prefetch_desc(my1);
      tma_prefetch_desc(my2);
    }
    bool ok = true;
    long long t0 = clock64();
    uint32_t idle = 0;
    while (ok && (st[0].r.n > 0 || st[1].r.n > 0)) {
      bool moved = false;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        S& t = st[k];
        if (t.r.n == 0) continue;
        const int stages = k == 0 ? C::kSt1 : C::kSt2, s = t.it % stages;
        uint64_t *full = k == 0 ? full1 : full2, *empty = k == 0 ? empty1 : empty2;
        if (!mbar_test_warp(&empty[s], ((uint32_t)(t.it / stages) & 1u) ^ 1u)) continue;
        moved = true;
        const Unit& u = t.r.u;
        const CUtensorMap* map = k == 0 ? my1 : my2;
        uint8_t* dst = smem + (k == 0 ? C::kY1Off : C::kY2Off) + s * C::kYTile;
        mbar_arrive_expect_tx_e(&full[s], C::kYTile);
        if (KV && PK) tma_load_5d_e(dst, map, &full[s], 0, u.qbase + t.y.row0, 0, t.y.h, 0);
        else tma_load_5d_e(dst, map, &full[s], 0, t.y.row0, 0, t.y.h, t.r.b);
        t.step(a);
      }
      if (moved) {
        idle = 0;
        t0 = clock64();
        continue;
      }
      __nanosleep(100);  // (the softmax warps beside it want the issue slots)
      if ((++idle & 63u) == 0) {  // bounded, as every wait here
        bool out = *abort_flag != 0;
        if (!out && clock64() - t0 > (long long)(ATTN_WAIT_LIMIT_NS * kMaxSmClockGHz)) {
          atomicCAS(a.err, kErrNone, kErrWaitTimeout);
          *abort_flag = 1;
          out = true;
        }
        ok = !__any_sync(0xFFFFFFFFu, out);
      }
    }
    if (!ok) {  // aborted: the copies in flight land before shared memory is released
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int stages = k == 0 ? C::kSt1 : C::kSt2;
        for (int v = max(0, st[k].it - stages); v < st[k].it; ++v)
          mbar_wait(&(k == 0 ? full1 : full2)[v % stages], (uint32_t)(v / stages) & 1u, nullptr, nullptr, 100000000ull);
      }
    }
  } else {
    // ---- softmax: P and dS ----
    const int wg = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float sl2 = a.scale * kLog2e;
    const uint64_t sl2x2 = f2pack(sl2, sl2);
    const int c0 = TN == 128 ? wg * 64 : 0;  // this thread's columns of an item: c0 .. c0 + 63
    // lse and D of this thread's row (dQ pass, d = 128; elsewhere they are in the products)
    auto row_stat = [&](const Run& q) {
      float2 v = make_float2(INFINITY, 0.f);
      if (!KV && !C::kRowExt && q.n > 0 && q.x * kT + r < q.u.Sq) {
        const size_t i = PK ? (size_t)q.h * a.total_q + q.u.qbase + q.x * kT + r
                                : ((size_t)q.b * a.Hq + q.h) * a.Sq + q.x * kT + r;
        v = a.stat[i];
      }
      return v;
    };
    // Rows of Y that this thread's row admits: [lo, hi) and (dQ pass) those below `sink`; tiles inside
    // [full_lo, full_hi) are admitted whole by every row of the F tile.
    struct Limits {
      int lo, hi, sink, full_lo, full_hi;
    };
    auto limits_of = [&](const Run& q) {
      Limits l{0, 0, 0, 0, 0};
      const Unit& u = q.u;
      const int f0 = q.x * kT;
      auto cl = [](long long x) { return (int)max(-(1LL << 30), min(x, 1LL << 30)); };
      const long long first = KV ? f0 - u.off : f0 + u.off, own = first + r;  // of the tile, of this row
      if constexpr (KV) {
        l.hi = l.full_hi = u.Sq;
        if (a.causal) {
          l.lo = cl(own);
          l.full_lo = cl(first + kT - 1);
        }
        if (a.window > 0) {
          if (f0 + r >= a.n_sink) l.hi = min(l.hi, cl(own + a.window));
          l.full_hi = min(l.full_hi, cl(first + a.window));
        }
      } else {
        l.hi = l.full_hi = u.Skv;
        if (a.causal) {
          l.hi = min(l.hi, cl(own + 1));
          l.full_hi = min(l.full_hi, cl(first + 1));
        }
        if (a.window > 0) {
          l.lo = cl(own - a.window + 1);
          l.full_lo = cl(first + kT - a.window);
          l.sink = min(a.n_sink, l.hi);
        }
      }
      return l;
    };
    Limits lim = limits_of(run);
    float2 stat = row_stat(run);
    ItemWalk<TN, KV> y(a, run);
    int it = 0, n_run = 0, n_part = 0;
    bool ok = true;
    while (ok && run.n > 0) {
      const int f0 = run.x * kT;
      const Unit& u = run.u;
      const uint64_t nlse2 = f2pack(-stat.x, -stat.x), ndd = f2pack(-stat.y, -stat.y);
      for (int m = 0; m < run.n; ++m, ++it) {
        if (m > 0) y.step(u);
        if (TN == 64 && (it & 1) != wg) continue;  // the other warpgroup's
        const int row0 = y.row0;
        const bool mask = row0 < lim.full_lo || row0 + TN > lim.full_hi;
        const int bs = it % NS, bd = it % ND, bp = it & 1;
        const uint32_t sc = lanes + C::kS + bs * TN + c0, dc = lanes + C::kDP + bd * TN + c0;
        const uint32_t pc = lanes + C::kP + bp * C::kPStep + c0;
        uint32_t s[64], p[64];
        ok = mbar_wait_warp(&bar_S[bp], (uint32_t)(it >> 1) & 1u, a.err, abort_flag);
        if (!ok) break;
        tc_fence_after();
        tmem_ld32(sc, s);
        tmem_ld32(sc + 32, s + 32);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_Sr[bs]);  // (the next S need not wait for this dP)
        // At d = 128 the exponentials before dP is waited for, under its product (after it: 172 and 233 us for
        // 3314 rows with and without a window, so 167 and 227); at d = 64, whose products are short, after
        // it, beside the rest of the chain's instructions (2 x 16 heads of 4096, not causal: 427 us, before it 434).
        auto exponentials = [&] {
#pragma unroll
          for (int c = 0; c < 64; c += 2) {
            const uint64_t x = f2pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
            float e0, e1;
            f2unpack(KV || C::kRowExt ? mul2(x, sl2x2) : fma2(x, sl2x2, nlse2), e0, e1);
            s[c] = __float_as_uint(ex2_approx(e0));
            s[c + 1] = __float_as_uint(ex2_approx(e1));
          }
        };
        if constexpr (D == 128) exponentials();
        ok = mbar_wait_warp(&bar_dP[bp], (uint32_t)(it >> 1) & 1u, a.err, abort_flag);
        if (!ok) break;
        tc_fence_after();
        tmem_ld32(dc, p);
        tmem_ld32(dc + 32, p + 32);
        tmem_wait_ld();
        if constexpr (C::kSep) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_dPr[bd]);
        }
        if constexpr (D == 64) exponentials();
        if constexpr (C::kSep) {
          // (of the item before the last, or of the last where there is one buffer)
          if constexpr (C::kOneP) ok = it == 0 || mbar_wait_warp(&bar_Pr[bp ^ 1], (uint32_t)((it - 1) >> 1) & 1u, a.err, abort_flag);
          else ok = mbar_wait_warp(&bar_Pr[bp], ((uint32_t)(it >> 1) & 1u) ^ 1u, a.err, abort_flag);
          if (!ok) break;
          tc_fence_after();
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t t[16], tp[16], tl[16], tpl[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const int k = q * 32 + 2 * c;
            uint64_t g = f2pack(__uint_as_float(p[k]), __uint_as_float(p[k + 1]));
            const float e0 = __uint_as_float(s[k]), e1 = __uint_as_float(s[k + 1]);
            float x0, x1;
            if constexpr (KV) tp[c] = pack_bf16x2(e0, e1);
            else if constexpr (!C::kRowExt) g = add2(g, ndd);
            f2unpack(mul2(g, f2pack(e0, e1)), x0, x1);
            t[c] = pack_bf16x2(x0, x1);
            if constexpr (FINE) {
              tl[c] = rest_bf16x2(t[c], x0, x1);
              if constexpr (KV) tpl[c] = rest_bf16x2(tp[c], e0, e1);
            }
          }
          if (mask) {
            // (a weight out of the row's columns may be inf, dP of a column that is no row anything:
            // both operands are cleared after their rounding)
            const int c1 = row0 + c0 + q * 32;
            const uint32_t in = (bits_below(lim.hi - c1) & ~bits_below(lim.lo - c1)) | bits_below(lim.sink - c1);
            if constexpr (KV) keep_bits<16>(tp, in);
            keep_bits<16>(t, in);
            if constexpr (FINE && KV) keep_bits<16>(tpl, in);
            if constexpr (FINE) keep_bits<16>(tl, in);
          }
          if constexpr (KV) tmem_st16(pc + q * 16, tp);
          tmem_st16(pc + (KV ? 32 : 0) + q * 16, t);
          if constexpr (FINE && KV) tmem_st16(pc + TN + q * 16, tpl);
          if constexpr (FINE) tmem_st16(pc + TN + (KV ? 32 : 0) + q * 16, tl);
        }
        if (PK && mask) {
          // rows of other sequences, or of none, behind this one's last: zeros for the second products, as
          // a weight of zero times what lies there could be NaN (the first ones have read the tile; gathered
          // instead of copied, such tiles held up the rings: eight packed sequences 249 us, so 231)
          const int from = max(0, (KV ? u.Sq : u.Skv) - row0);
          uint8_t* y1 = smem + C::kY1Off + it % C::kSt1 * C::kYTile;
          uint8_t* y2 = smem + C::kY2Off + it % C::kSt2 * C::kYTile;
#pragma unroll 1
          for (int i = from * 8 + (TN == 128 ? (int)threadIdx.x : r); i < TN * 8; i += TN == 128 ? 256 : 128) {
#pragma unroll
            for (int c = 0; c < C::kPanels; ++c) {
              *reinterpret_cast<uint4*>(y1 + c * C::kYPanel + i * 16) = make_uint4(0, 0, 0, 0);
              if (KV) *reinterpret_cast<uint4*>(y2 + c * C::kYPanel + i * 16) = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async_smem();
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_P[bp]);
      }
      if (!ok) break;
      // ---- the run's sums: rows of the output, or fp32 partials ----
      // (what the next run needs, while this one's last products end)
      const Run next = w.next();
      stat = row_stat(next);
      lim = limits_of(next);
      y = ItemWalk<TN, KV>(a, next);
      const bool part = run.n != run.cnt;
      // Of the unit's part in this slice, which starts at item s0 (or with the unit): whether there were runs
      // before this one, and whether there are more.
      const int s0 = cta * w.per - run.first;
      const bool more = run.i0 > max(0, s0), ends = run.i0 + run.n == min(run.cnt, s0 + w.per);
      // KV: warpgroup 0 dV, 1 dK; else a half of dQ's columns each
      constexpr int kCols = KV ? D : D / 2;
      const uint32_t col0 = KV ? (wg == 0 ? 0 : C::kAcc1) : C::kAcc1 + wg * kCols;
      const float f = (KV && wg == 0) ? 1.f : a.scale;
      // rows [0, live) are the sequence's, [live, wrote) written as zeros
      const int live = min(kT, (KV ? u.Skv : u.Sq) - f0);
      const int wrote = KV && a.fill ? min(kT, a.Skv - f0) : live;
      uint16_t* out;
      size_t row_w;  // elements from row to row
      if constexpr (KV) {
        out = (wg == 0 ? a.dv : a.dk) + (((size_t)run.b * a.Skv + f0) * a.Hkv + run.h) * D;
        row_w = (size_t)a.Hkv * D;
      } else {
        out = a.dq + ((size_t)(u.qbase + f0) * a.Hq + run.h) * D + wg * kCols;
        row_w = (size_t)a.Hq * D;
      }
      // 32 columns of the thread's row from `col` on; four lanes write 64 bytes of a row side by side (a
      // row a lane made each store 32 lines)
      auto put_rows = [&](uint4 (&q)[4], int col) {
        transpose4(q, lane);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = (r & ~3) + e;
          if (row < wrote)
            *reinterpret_cast<uint4*>(out + (size_t)row * row_w + col + (lane & 3) * 8) =
                row < live ? q[e] : make_uint4(0, 0, 0, 0);
        }
      };
      constexpr int kSlot = kT * D * (KV ? 2 : 1) / 4;  // float4s of a partial: [column / 4][row]
      float4* const parts = reinterpret_cast<float4*>(KV ? a.part_k : a.part_q) + (size_t)slot0 * kSlot +
                            (size_t)wg * (kCols / 4) * kT + r;
      float4* pp = parts + ((size_t)cta * 2 + (s0 > 0 ? 0 : 1)) * kSlot;
      ok = mbar_wait_warp(bar_acc, (uint32_t)n_run & 1u, a.err, abort_flag);
      if (!ok) break;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < kCols; c += 32) {
        uint32_t x[32];
        tmem_ld32(lanes + col0 + c, x);
        tmem_wait_ld();
        if (c + 32 == kCols) {  // the next run's sums may start
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_accr);
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
        if (part) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float4 v = make_float4(__uint_as_float(x[e]), __uint_as_float(x[e + 1]), __uint_as_float(x[e + 2]),
                                   __uint_as_float(x[e + 3]));
            float4* const to = pp + (size_t)((c + e) / 4) * kT;
            if (more) {  // (this thread's own, of the run before)
              const float4 u = *to;
              v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
            }
            *to = v;
          }
        } else {
          uint4 q[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t* y = x + 8 * e;
            q[e] = make_uint4(pack_bf16x2(__uint_as_float(y[0]), __uint_as_float(y[1])),
                              pack_bf16x2(__uint_as_float(y[2]), __uint_as_float(y[3])),
                              pack_bf16x2(__uint_as_float(y[4]), __uint_as_float(y[5])),
                              pack_bf16x2(__uint_as_float(y[6]), __uint_as_float(y[7])));
          }
          put_rows(q, c);
        }
      }
      if (part && ends) {
        // The slice that finishes a cut unit last sums its parts, in slice order whoever it is.
        const int c0 = run.first / w.per, c1 = (run.first + run.cnt - 1) / w.per;  // the unit's slices
        bool sum = c0 == c1;  // (a whole one of several runs is this slice's alone, and the counters are not its)
        __threadfence();
        if (!sum) {
          // (mbarriers, whose waits end, in place of a barrier that a warp after a failed wait would miss)
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_out);
          if (warp == 0) {
            ok = mbar_wait_warp(bar_out, (uint32_t)n_part & 1u, a.err, abort_flag);
            if (!ok) break;
            if (lane == 0) {
              __threadfence();
              *last_flag = atomicAdd(a.joined + list_of(KV, FINE) * kMaxCtas + c0, 1) == c1 - c0;
              mbar_arrive(bar_last);
            }
            __syncwarp();
          }
          ok = mbar_wait_warp(bar_last, (uint32_t)n_part & 1u, a.err, abort_flag);
          if (!ok) break;
          ++n_part;
          sum = *last_flag;
          __threadfence();
        }
        if (sum) {
          // (32 columns of two parts in flight: one 8-column group at a time took 20 us a unit)
#pragma unroll 1
          for (int c = 0; c < kCols; c += 32) {
            float4 x[8], y[8];
            const float4* p = parts + (size_t)(c / 4) * kT;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = __ldcg(p + ((size_t)c0 * 2 + 1) * kSlot + (size_t)e * kT);
#pragma unroll 1
            for (int k = c0 + 1; k <= c1; ++k) {
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] = __ldcg(p + (size_t)k * 2 * kSlot + (size_t)e * kT);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                x[e].x += y[e].x; x[e].y += y[e].y; x[e].z += y[e].z; x[e].w += y[e].w;
              }
            }
            uint4 q[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 u = x[2 * e], v = x[2 * e + 1];
              q[e] = make_uint4(pack_bf16x2(u.x, u.y), pack_bf16x2(u.z, u.w), pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
            }
            put_rows(q, c);
          }
        }
      }
      run = next;
      ++n_run;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

// Both passes: dQ's CTAs start as dK/dV's end.  A pass of a packed batch (PK) may have sequences of both forms,
// which then share its CTAs by their lists' costs.
constexpr int kThreads = 384;
// CTAs of a pass that take the sequences of two terms, whose tiles cost about 1.7 times as much a row.
template <int D, bool KV>
__device__ __forceinline__ int two_term_ctas(const BackwardArgs& a) {
  const int n = a.B * f_tiles(a, KV);
  const float two = a.forms & kTwoTerms ? a.pre[list_of(KV, true)][n] * (1.7f * BwdCfg<D, KV, true>::TN) : 0.f;
  const float one = a.forms & kOneTerm ? a.pre[list_of(KV, false)][n] * (1.f * BwdCfg<D, KV, false>::TN) : 0.f;
  if (two == 0.f || one == 0.f) return two == 0.f ? 0 : a.ctas;
  // (rounded up, as a few CTAs' share too large shows and a few too small does not: 64 sequences of 100 to 1990
  // rows, four heads of 64, 332 us with it rounded to nearest)
  return min(max((int)(a.ctas * (two / (two + one)) + 0.9f), 1), a.ctas - 1);
}
template <int D, bool KV, bool PK, bool ONE, bool TWO>
__device__ __forceinline__ void backward_forms(const BackwardArgs& a, int cta) {
  int n = 0;
  if constexpr (TWO) n = ONE ? two_term_ctas<D, KV>(a) : a.ctas;
  // (one term first: behind two, eight packed sequences of 1000 rows, 32 heads of 128, took 4 us more of 290)
  if constexpr (ONE) {
    if (!TWO || cta >= n) return backward_pass<D, KV, PK, false>(a, cta - n, a.ctas - n, 2 * n);
  }
  if constexpr (TWO) backward_pass<D, KV, PK, true>(a, cta, n, 0);
}
template <int D, bool PK, bool ONE, bool TWO>
__global__ void __launch_bounds__(kThreads, 1) backward_kernel(const __grid_constant__ BackwardArgs a) {
  static_assert(BwdCfg<D, true, ONE>::kThreads == kThreads && BwdCfg<D, false, TWO>::kThreads == kThreads);
  if ((int)blockIdx.x < a.ctas) backward_forms<D, true, PK, ONE, TWO>(a, (int)blockIdx.x);
  else backward_forms<D, false, PK, ONE, TWO>(a, (int)blockIdx.x - a.ctas);
}

template <int D>
cudaError_t launch_prep(const BackwardArgs& a, bool any, cudaStream_t stream) {
  const long long blocks = any ? (a.total_q + prep_rows(D) - 1LL) / prep_rows(D) * a.Hq : 0;
  const unsigned grid = kLists + kZeroCtas + (unsigned)blocks;
  if (a.o_bf16) backward_prep_kernel<D, true><<<grid, kPrepThreads, 0, stream>>>(a);
  else backward_prep_kernel<D, false><<<grid, kPrepThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int D, bool PK, bool ONE, bool TWO>
cudaError_t launch_d(const BackwardArgs& a, cudaStream_t stream) {
  constexpr int one = ONE ? std::max(BwdCfg<D, true, false>::kSmem, BwdCfg<D, false, false>::kSmem) : 0;
  constexpr int two = TWO ? std::max(BwdCfg<D, true, true>::kSmem, BwdCfg<D, false, true>::kSmem) : 0;
  constexpr int kSmem = std::max(one, two);
  auto kern = backward_kernel<D, PK, ONE, TWO>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  kern<<<2 * a.ctas, kThreads, kSmem, stream>>>(a);
  return cudaGetLastError();
}
template <bool PK, bool ONE, bool TWO>
cudaError_t launch_all(const BackwardArgs& a, cudaStream_t stream) {
  switch (a.d) {
    case 64: return launch_d<64, PK, ONE, TWO>(a, stream);
    case 128: return launch_d<128, PK, ONE, TWO>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace
}  // namespace attn
