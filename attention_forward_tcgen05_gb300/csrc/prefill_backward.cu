// prefill_backward.cu -- gradients of the prefill attention (causal or not, sliding window
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
// d = 128; a third accumulator would not fit.  Both passes are one kernel: with
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
// goes out as fp32 partials, which a last launch sums in slice order.
//
// Warps: 0-7 softmax (thread = row of F, 64 columns of an item), 8 / 9 S and dP with their F tiles, 10
// the second products, 11 the rings of Y1 and Y2.
#include <algorithm>
#include <cmath>

#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kT = 128;           // rows of a tile
// A run of a unit's items costs its start and end (the F tiles' copy, the sums' way out) beside its
// items, about as much as kRunCost of them: units of few items would otherwise fill some slices
// with nothing but starts and ends.
constexpr int kRunCost = 3;
constexpr int kMinCost = 2 + kRunCost;  // of a slice

// Columns of S and dP per item.  128, halved between the softmax warpgroups, where TMEM holds
// two S and one dP beside the sums; the dK/dV pass at d = 128 has 256 columns for both: 64, two
// buffers of each, an item for each warpgroup in turn.
template <int D, bool KV>
struct BwdCfg {
  static constexpr int TN = (KV && D == 128) ? 64 : 128;  // rows of a Y tile
  static constexpr int NS = 2;                            // S buffers
  static constexpr int ND = TN == 64 ? 2 : 1;             // dP buffers
  static constexpr int kArrive = TN == 64 ? 4 : 8;        // softmax warps of an item
  static constexpr int kPanels = D / 64;
  static constexpr int kFPanel = kT * 128;
  static constexpr int kFTile = kPanels * kFPanel;
  static constexpr int kYPanel = TN * 128;
  static constexpr int kYTile = kPanels * kYPanel;
  static constexpr int kSt1 = (D == 128 && !KV) ? 3 : 4;  // ring of Y1
  static constexpr int kSt2 = (D == 128 && !KV) ? 2 : 4;  // ring of Y2
  static constexpr int kY1Off = 2 * kFTile;
  static constexpr int kY2Off = kY1Off + kSt1 * kYTile;
  // columns beside the dK/dV pass's tiles, 16 bytes a row: lse beside Q, D beside g, ones beside K
  // and V, and zeros, the second eight columns of all of them
  static constexpr int kExt = KV ? TN * 16 : 0;
  static constexpr int kOnes = KV ? kT * 16 : 0;
  static constexpr int kExt1Off = kY2Off + kSt2 * kYTile;
  static constexpr int kExt2Off = kExt1Off + kSt1 * kExt;
  static constexpr int kOnesOff = kExt2Off + kSt2 * kExt;
  static constexpr int kZeroOff = kOnesOff + kOnes;
  static constexpr int kBarOff = kZeroOff + kOnes;
  static constexpr int kNumBars = 2 * kSt1 + 2 * kSt2 + 4 + 4 * NS + 2 * ND + 2;
  static constexpr int kSmem = kBarOff + kNumBars * 8 + 16 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static constexpr uint32_t kAcc1 = KV ? D : 0;  // TMEM columns; acc0 at 0
  static constexpr uint32_t kS = kAcc1 + D;
  static constexpr uint32_t kDP = kS + NS * TN;
  static_assert(kDP + ND * TN <= 512, "TMEM budget");
  static constexpr int kThreads = 384;
};

// Extent of a unit: which Y tiles its F tile meets.
struct Unit {
  int Sq, Skv, qbase, kbase;  // rows and keys of the sequence, first row of q, first row of k
  long long off;              // key index of row i: i + off
  int nt, t0;                 // Y tiles, dK/dV pass: from t0 on; dQ pass: by the tile list
  TileList tl;
};
template <bool KV>
__device__ __forceinline__ Unit unit_of(const BackwardArgs& a, int b, int x) {
  Unit u;
  const SeqExtent e = seq_extent(b, a.Sq, a.Skv, a.cu_q, a.kv_lens, a.total_q);
  u.Sq = e.Sq; u.Skv = e.Skv;
  u.qbase = a.cu_q ? e.qbase : b * a.Sq;
  u.kbase = b * a.Skv;
  u.off = (long long)u.Skv - u.Sq;
  u.nt = 0; u.t0 = 0;
  u.tl = TileList{0x7FFFFFFF, 0};
  const int f0 = x * kT;
  if constexpr (KV) {
    if (f0 >= u.Skv) return u;
    const int last = min(u.Skv, f0 + kT) - 1;
    const long long lo = a.causal ? max(0LL, f0 - u.off) : 0LL;
    long long hi = u.Sq;
    if (a.window > 0 && f0 >= a.n_sink) hi = min(hi, last + (long long)a.window - u.off);
    if (hi <= lo) return u;
    u.t0 = (int)(lo / a.tn_k);
    u.nt = (int)((hi + a.tn_k - 1) / a.tn_k) - u.t0;
  } else {
    if (f0 >= u.Sq) return u;
    const int last = min(u.Sq, f0 + kT) - 1;
    const long long hi = a.causal ? min((long long)u.Skv, max(0LL, last + u.off + 1)) : u.Skv;
    const int n = (int)((hi + kT - 1) / kT);
    u.tl = tile_list(f0 + u.off, n, a.window, a.n_sink, u.Skv, kT);
    u.nt = tile_list_len(u.tl, n);
  }
  return u;
}
template <bool KV>
__device__ __forceinline__ int unit_items(const BackwardArgs& a, const Unit& u) {
  return KV ? u.nt * (a.Hq / a.Hkv) : u.nt;
}
__device__ __forceinline__ int unit_cost(int items) { return items > 0 ? items + kRunCost : 0; }
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
template <bool KV>
__device__ void scan_costs(const BackwardArgs& a, int* pre) {
  __shared__ int sums[kPrepThreads / 32];
  const int nx = f_tiles(a, KV), n = a.B * nx, H = KV ? a.Hkv : a.Hq;
  const int per = (n + kPrepThreads - 1) / kPrepThreads;
  const int lo = min(n, (int)threadIdx.x * per), hi = min(n, lo + per);
  int s = 0;
  // a sequence above max_sq is reported, as the positions of its first rows would be taken for the last ones
  if (KV && a.cu_q)
    for (int b = threadIdx.x; b < a.B; b += kPrepThreads) {
      const int c0 = min(max(a.cu_q[b], 0), a.total_q), c1 = min(a.cu_q[b + 1], a.total_q);
      if (c1 - c0 > a.Sq) atomicCAS(a.err, kErrNone, kErrBadShape);
    }
  for (int g = lo; g < hi; ++g) s += unit_cost(unit_items<KV>(a, unit_of<KV>(a, g / nx, g % nx))) * H;
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
    at += unit_cost(unit_items<KV>(a, unit_of<KV>(a, g / nx, g % nx))) * H;
  }
  if (hi == n && lo < n) pre[n] = at;
  if (n == 0 && threadIdx.x == 0) pre[0] = 0;
}

// D / 8 lanes to a (row, head), rows in memory order of o: [rows][Hq][D].
template <int D, bool OBF16>
__global__ void __launch_bounds__(kPrepThreads) backward_prep_kernel(const __grid_constant__ BackwardArgs a) {
  if (blockIdx.x < 2) {
    if (blockIdx.x == 0) scan_costs<true>(a, a.pre_k);
    else scan_costs<false>(a, a.pre_q);
    return;
  }
  constexpr int L = D / 8;
  const long long n = (long long)a.total_q * a.Hq;
  const long long at = ((long long)(blockIdx.x - 2) * kPrepThreads + threadIdx.x) / L;
  const int c = threadIdx.x % L;
  const long long rh = min(at, n - 1);  // (every lane takes part in the sums)
  const uint4 g = *reinterpret_cast<const uint4*>(a.dout + rh * D + c * 8);
  float s;
  if constexpr (OBF16) {
    s = dot8(g, *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.o) + rh * D + c * 8));
  } else {
    const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.o) + rh * D + c * 8);
    s = dot8(g, p[0], p[1]);
  }
#pragma unroll
  for (int o = 1; o < L; o <<= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if (c != 0 || at >= n) return;
  const int row = (int)(rh / a.Hq), h = (int)(rh % a.Hq);
  // [B][Hq][Sq], or packed [Hq][total_q]
  const size_t i = a.cu_q ? (size_t)h * a.total_q + row
                          : ((size_t)(row / a.Sq) * a.Hq + h) * a.Sq + row % a.Sq;
  const float lse = a.lse[i];
  if (a.dlse) s -= a.dlse[i];
  // a row that saw no key (lse = -inf) takes no part
  a.stat[i] = make_float2(lse == -INFINITY ? INFINITY : lse * kLog2e, s);
  float x = -lse / a.scale;
  if (x > 1e38f || x < -1e38f) x = -1e38f;
  uint32_t l0, l1, l2, d0, d1, d2;
  split3(x, l0, l1, l2);
  split3(-s, d0, d1, d2);
  a.ext1[i] = make_uint4(l0 | l1 << 16, l2, 0u, 0u);
  a.ext2[i] = make_uint4(d0 | d1 << 16, d2, 0u, 0u);
}

// ------------------------------------------------------------------ the two passes
// The items of a slice in order, run by run of one unit.
template <bool KV>
struct Walk {
  const BackwardArgs& a;
  const int* pre;
  int nx, n_groups, H, pos, end;  // place in the list of costs, end of the slice
  int g, g0, cnt;                 // group, its place, items of one of its units
  Unit u;
  int b, x;
  __device__ __forceinline__ Walk(const BackwardArgs& a_, int lane)
      : a(a_), pre(KV ? a_.pre_k : a_.pre_q), H(KV ? a_.Hkv : a_.Hq) {
    nx = f_tiles(a, KV);
    n_groups = a.B * nx;
    const int total = pre[n_groups], per = slice_cost(total, (int)gridDim.x);
    pos = (int)min((long long)total, (long long)blockIdx.x * per);
    end = min(total, pos + per);
    g = 0; g0 = 0; cnt = 0; b = x = 0;
    if (pos >= end) return;
    // the last group that starts at or before pos (those without items start where the next does)
    int lo = 0, hi = n_groups;  // pre[lo] <= pos < pre[hi]
    while (hi - lo > 1) {
      const int step = max(1, (hi - lo) / 32);
      const int p = min(lo + (lane + 1) * step, hi);
      const unsigned over = __ballot_sync(0xFFFFFFFFu, p >= hi || pre[p] > pos);
      const int k = over ? __ffs(over) - 1 : 32;  // probes at or before pos
      hi = k < 32 ? min(lo + (k + 1) * step, hi) : hi;
      lo = lo + k * step;
    }
    g = lo;
    enter();
  }
  __device__ __forceinline__ void enter() {
    b = g / nx;
    x = g % nx;
    u = unit_of<KV>(a, b, x);
    cnt = unit_items<KV>(a, u);
    g0 = pre[g];
  }
  // the next run: head h, its items [i0, i0 + n); false at the end of the slice
  __device__ __forceinline__ bool next(int& h, int& i0, int& n) {
    while (pos < end) {
      while (pos >= g0 + unit_cost(cnt) * H) {
        ++g;
        enter();
      }
      const int cost = unit_cost(cnt);
      h = (pos - g0) / cost;
      const int at = pos - g0 - h * cost, to = min(cost, at + end - pos);  // of the unit's cost
      pos += to - at;
      i0 = max(0, at - kRunCost);
      n = max(0, to - kRunCost) - i0;
      if (n > 0) return true;
    }
    return false;
  }
};

// Y tile of item i of a unit: its first row (query rows of head h, or keys), and the head.
template <bool KV>
struct ItemWalk {
  int h, t, row0;
  __device__ __forceinline__ ItemWalk() : h(0), t(0), row0(0) {}
  __device__ __forceinline__ ItemWalk(const BackwardArgs& a, const Unit& u, int unit_head, int i) {
    if constexpr (KV) {
      const int q = i / u.nt;
      h = unit_head * (a.Hq / a.Hkv) + q;
      t = i - q * u.nt;
      row0 = (u.t0 + t) * a.tn_k;
    } else {
      h = unit_head / (a.Hq / a.Hkv);
      t = i;
      row0 = tile_list_key(u.tl, t) * kT;
    }
  }
  __device__ __forceinline__ void step(const BackwardArgs& a, const Unit& u) {
    ++t;
    if constexpr (KV) {
      if (t == u.nt) {
        t = 0;
        ++h;
      }
      row0 = (u.t0 + t) * a.tn_k;
    } else {
      row0 = tile_list_key(u.tl, t) * kT;
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

// A ring of Y tiles and the items it still has to bring.
template <bool KV>
struct Stream {
  Walk<KV> w;
  ItemWalk<KV> y;
  int h, i0, n, m, it;
  bool live;
  __device__ __forceinline__ Stream(const BackwardArgs& a, const Walk<KV>& w_) : w(w_), y(), m(0), it(0) {
    live = w.next(h, i0, n);
    if (live) y = ItemWalk<KV>(a, w.u, h, i0);
  }
  __device__ __forceinline__ void step(const BackwardArgs& a) {
    ++it;
    if (++m < n) {
      y.step(a, w.u);
      return;
    }
    m = 0;
    live = w.next(h, i0, n);
    if (live) y = ItemWalk<KV>(a, w.u, h, i0);
  }
};

template <int D, bool KV>
__global__ void __launch_bounds__(BwdCfg<D, KV>::kThreads, 1)
    backward_kernel(const __grid_constant__ BackwardArgs a) {
  using C = BwdCfg<D, KV>;
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
  uint64_t* bar_S = emptyF + 2;        // [NS] S computed
  uint64_t* bar_Sr = bar_S + NS;       // [NS] its P and dS used up
  uint64_t* bar_P = bar_Sr + NS;       // [NS] P stored
  uint64_t* bar_dS = bar_P + NS;       // [NS] dS stored
  uint64_t* bar_dP = bar_dS + NS;      // [ND] dP computed
  uint64_t* bar_dPr = bar_dP + ND;     // [ND] dP read
  uint64_t* bar_acc = bar_dPr + ND;    // a run's sums complete
  uint64_t* bar_accr = bar_acc + 1;    // they are read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_accr + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kSt1; ++s) { mbar_init(&full1[s], 1); mbar_init(&empty1[s], 1); }
    for (int s = 0; s < C::kSt2; ++s) { mbar_init(&full2[s], 1); mbar_init(&empty2[s], KV ? 2 : 1); }
    for (int s = 0; s < 2; ++s) { mbar_init(&fullF[s], 1); mbar_init(&emptyF[s], 1); }
    for (int s = 0; s < NS; ++s) {
      mbar_init(&bar_S[s], 1);
      mbar_init(&bar_Sr[s], 1);
      mbar_init(&bar_P[s], C::kArrive);
      mbar_init(&bar_dS[s], C::kArrive);
    }
    for (int s = 0; s < ND; ++s) { mbar_init(&bar_dP[s], 1); mbar_init(&bar_dPr[s], C::kArrive); }
    mbar_init(bar_acc, 1);
    mbar_init(bar_accr, 8);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if constexpr (KV) {
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

  Walk<KV> w(a, lane);
  int h, i0, n;
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
    int it = 0, run = 0;
    bool ok = true;
    while (ok && w.next(h, i0, n)) {
      if (!mbar_wait_warp(eF, ((uint32_t)run & 1u) ^ 1u, a.err, abort_flag)) break;
      const bool packed = !KV && a.cu_q != nullptr;
      mbar_arrive_expect_tx_e(fF, C::kFTile);
      tma_load_5d_e(sF, map, fF, 0, packed ? w.u.qbase + w.x * kT : w.x * kT, 0, h, packed ? 0 : w.b);
      ok = mbar_wait_warp(fF, (uint32_t)run & 1u, a.err, abort_flag);
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
          const uint32_t e = ext + s * C::kExt;
          mma_ss_e(d, d1, smem_desc(e, zero - e, 128, kSwizzleNone), idesc, 1u);
        }
        mma_commit_e(&done[buf]);
        if (!first) mma_commit_e(&empty2[s]);
        if (m == n - 1) mma_commit_e(eF);
      }
      ++run;
    }
    // (aborted: the last copy lands before shared memory is released)
    if (!ok && run > 0) mbar_wait(fF, (uint32_t)(run - 1) & 1u, nullptr, nullptr, 100000000ull);
  } else if (warp == 10) {
    // ---- second products: acc0 += P Y2 (dV), acc1 += dS Y1 ----
    constexpr uint32_t idesc = idesc_bf16_f32(128, D, 0, 1);
    const uint64_t my1 = smem_desc(smem_u32(smem + C::kY1Off), C::kYPanel, 1024, kSwizzle128B);
    const uint64_t my2 = smem_desc(smem_u32(smem + C::kY2Off), C::kYPanel, 1024, kSwizzle128B);
    // A in TMEM: 32 columns of bf16 pairs for each 64 columns of S; Y MN-major
    auto issue = [&](uint32_t acc, uint32_t p, uint64_t y, bool fresh) {
#pragma unroll
      for (int kk = 0; kk < TN / 16; ++kk)
        mma_ts_e(tmem + acc, p + (kk >> 2) * 64 + (kk & 3) * 8, y + (uint64_t)(kk * (2048 >> 4)), idesc,
                 (!fresh || kk > 0) ? 1u : 0u);
    };
    int it = 0, run = 0;
    bool ok = true;
    while (ok && w.next(h, i0, n)) {
      if (run > 0) ok = mbar_wait_warp(bar_accr, (uint32_t)(run - 1) & 1u, a.err, abort_flag);
      for (int m = 0; ok && m < n; ++m, ++it) {
        const int buf = it % NS, s1 = it % C::kSt1, s2 = it % C::kSt2;
        const uint32_t sb = tmem + C::kS + buf * TN, ph = (uint32_t)(it / NS) & 1u;
        if constexpr (KV) {
          // (g's tile is whole where its dP is waited for: the softmax stores P before)
          ok = mbar_wait_warp(&full2[s2], (uint32_t)(it / C::kSt2) & 1u, a.err, abort_flag) &&
               mbar_wait_warp(&bar_P[buf], ph, a.err, abort_flag);
          if (!ok) break;
          tc_fence_after();
          issue(0, sb, my2 + (uint64_t)((s2 * C::kYTile) >> 4), m == 0);
          mma_commit_e(&empty2[s2]);
        }
        ok = mbar_wait_warp(&bar_dS[buf], ph, a.err, abort_flag);
        if (!ok) break;
        tc_fence_after();
        issue(C::kAcc1, sb + (KV ? 32 : 0), my1 + (uint64_t)((s1 * C::kYTile) >> 4), m == 0);
        mma_commit_e(&bar_Sr[buf]);
        mma_commit_e(&empty1[s1]);
        if (m == n - 1) mma_commit_e(bar_acc);
      }
      ++run;
    }
  } else if (warp == 11) {
    // ---- the rings of Y1 and Y2, each slot filled as soon as it is free ----
    Stream<KV> st[2] = {Stream<KV>(a, w), Stream<KV>(a, w)};
    if (lane == 0) {
      tma_prefetch_desc(KV ? &a.tm_qy : &a.tm_k);
      tma_prefetch_desc(KV ? &a.tm_doy : &a.tm_v);
    }
    bool ok = true;
    long long t0 = clock64();
    uint32_t idle = 0;
    while (ok && (st[0].live || st[1].live)) {
      bool moved = false;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        Stream<KV>& t = st[k];
        if (!t.live) continue;
        const int stages = k == 0 ? C::kSt1 : C::kSt2, s = t.it % stages;
        uint64_t *full = k == 0 ? full1 : full2, *empty = k == 0 ? empty1 : empty2;
        if (!mbar_test_warp(&empty[s], ((uint32_t)(t.it / stages) & 1u) ^ 1u)) continue;
        moved = true;
        const Unit& u = t.w.u;
        const CUtensorMap* map = KV ? (k == 0 ? &a.tm_qy : &a.tm_doy) : (k == 0 ? &a.tm_k : &a.tm_v);
        uint8_t* dst = smem + (k == 0 ? C::kY1Off : C::kY2Off) + s * C::kYTile;
        const int rows = KV ? u.Sq : u.Skv;  // Y rows of the sequence
        const int row_base = KV ? u.qbase : u.kbase;
        // a packed batch: other rows follow a sequence's own
        const bool whole = a.cu_q == nullptr || t.y.row0 + TN <= rows;
        uint32_t bytes = KV ? C::kExt : 0;
        if (whole) {
          bytes += C::kYTile;
        } else {
          // its last rows are gathered, so that the rows behind them arrive as zeros (a weight of
          // zero times what lies there could be NaN)
          const uint16_t* base = KV ? (k == 0 ? a.q : a.dout) : (k == 0 ? a.k : a.v);
          int ri[TN / 32];
#pragma unroll
          for (int e = 0; e < TN / 32; ++e) {
            const int r = t.y.row0 + e * 32 + lane;
            ri[e] = r < rows ? row_base + r : -1;
          }
          paged_gather<D, TN / 32>(smem_u32(dst), C::kYPanel, base, KV ? a.Hq : a.Hkv, t.y.h, lane, ri);
          cp_async_commit();
          cp_async_wait<0>();
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (bytes) mbar_arrive_expect_tx_e(&full[s], bytes);
        else if (lane == 0) mbar_arrive(&full[s]);
        if (whole) {
          if (KV && a.cu_q) tma_load_5d_e(dst, map, &full[s], 0, row_base + t.y.row0, 0, t.y.h, 0);
          else tma_load_5d_e(dst, map, &full[s], 0, t.y.row0, 0, t.y.h, t.w.b);
        }
        if constexpr (KV) {
          const size_t i = a.cu_q ? (size_t)t.y.h * a.total_q + row_base + t.y.row0
                                  : ((size_t)t.w.b * a.Hq + t.y.h) * a.Sq + t.y.row0;
          bulk_load_e(smem + (k == 0 ? C::kExt1Off : C::kExt2Off) + s * C::kExt, (k == 0 ? a.ext1 : a.ext2) + i,
                      C::kExt, &full[s]);
        }
        t.step(a);
      }
      if (moved) {
        idle = 0;
        t0 = clock64();
      } else if ((++idle & 63u) == 0) {  // bounded, as every wait here
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
    int it = 0, run = 0;
    bool ok = true;
    while (ok && w.next(h, i0, n)) {
      const int f0 = w.x * kT;
      float lse2 = INFINITY, dd = 0.f;
      if constexpr (!KV) {
        if (f0 + r < w.u.Sq) {
          const size_t i = a.cu_q ? (size_t)h * a.total_q + w.u.qbase + f0 + r
                                  : ((size_t)w.b * a.Hq + h) * a.Sq + f0 + r;
          const float2 st = a.stat[i];
          lse2 = st.x;
          dd = st.y;
        }
      }
      const uint64_t nlse2 = f2pack(-lse2, -lse2), ndd = f2pack(-dd, -dd);
      ItemWalk<KV> y(a, w.u, h, i0);
      for (int m = 0; m < n; ++m, ++it, y.step(a, w.u)) {
        if (TN == 64 && (it & 1) != wg) continue;  // the other warpgroup's
        const int buf = it % NS, bd = it % ND;
        const uint32_t sc = lanes + C::kS + buf * TN + c0, dc = lanes + C::kDP + bd * TN + c0;
        ok = mbar_wait_warp(&bar_S[buf], (uint32_t)(it / NS) & 1u, a.err, abort_flag);
        if (!ok) break;
        tc_fence_after();
        uint32_t s[64];
        tmem_ld32(sc, s);
        tmem_ld32(sc + 32, s + 32);
        // columns of this thread's row: [lo, hi) and, dQ pass, those before `sink`
        int lo = 0, hi = TN, sink = 0;
        bool mask;
        if constexpr (KV) {
          const long long d0 = w.u.off + y.row0;  // key index of the tile's first row
          const int j = f0 + r;
          mask = y.row0 + TN > w.u.Sq;
          hi = min(TN, w.u.Sq - y.row0);
          if (a.causal) {
            mask = mask || f0 + kT - 1 > d0;
            lo = (int)min((long long)TN, max(0LL, j - d0));
          }
          if (a.window > 0) {
            mask = mask || f0 + (long long)a.window < d0 + TN;
            if (j >= a.n_sink) hi = (int)min((long long)hi, max(0LL, j + (long long)a.window - d0));
          }
        } else {
          const long long pos = f0 + r + w.u.off;  // key index of this row
          const long long p0 = f0 + w.u.off;
          mask = y.row0 + TN > w.u.Skv;
          hi = min(TN, w.u.Skv - y.row0);
          if (a.causal) {
            mask = mask || y.row0 + TN - 1 > p0;
            hi = (int)min((long long)hi, max(0LL, pos + 1 - y.row0));
          }
          if (a.window > 0) {
            mask = mask || y.row0 <= p0 + kT - 1 - a.window;
            lo = (int)min((long long)TN, max(0LL, pos - a.window + 1 - y.row0));
            sink = min(TN, max(0, a.n_sink - y.row0));
          }
        }
        // as bits (a weight out of them may be inf, dP of a column that is no row anything: both
        // products' operands are cleared after their rounding)
        uint32_t in[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
        if (mask) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int c1 = c0 + q * 32;
            in[q] = (bits_below(hi - c1) & ~bits_below(lo - c1)) | bits_below(min(sink, hi) - c1);
          }
        }
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          const uint64_t x = f2pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
          float e0, e1;
          f2unpack(KV ? mul2(x, sl2x2) : fma2(x, sl2x2, nlse2), e0, e1);
          s[c] = __float_as_uint(ex2_approx(e0));
          s[c + 1] = __float_as_uint(ex2_approx(e1));
        }
        if constexpr (KV) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t t[16];
#pragma unroll
            for (int c = 0; c < 16; ++c)
              t[c] = pack_bf16x2(__uint_as_float(s[q * 32 + 2 * c]), __uint_as_float(s[q * 32 + 2 * c + 1]));
            if (mask) keep_bits<16>(t, in[q]);
            tmem_st16(sc + q * 16, t);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_P[buf]);
        }
        ok = mbar_wait_warp(&bar_dP[bd], (uint32_t)(it / ND) & 1u, a.err, abort_flag);
        if (!ok) break;
        tc_fence_after();
        uint32_t p[64];
        tmem_ld32(dc, p);
        tmem_ld32(dc + 32, p + 32);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_dPr[bd]);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t t[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const int k = q * 32 + 2 * c;
            uint64_t g = f2pack(__uint_as_float(p[k]), __uint_as_float(p[k + 1]));
            if constexpr (!KV) g = add2(g, ndd);
            float x0, x1;
            f2unpack(mul2(g, f2pack(__uint_as_float(s[k]), __uint_as_float(s[k + 1]))), x0, x1);
            t[c] = pack_bf16x2(x0, x1);
          }
          if (mask) keep_bits<16>(t, in[q]);
          tmem_st16(sc + (KV ? 32 : 0) + q * 16, t);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_dS[buf]);
      }
      if (!ok) break;
      // ---- the run's sums: rows of the output, or fp32 partials ----
      ok = mbar_wait_warp(bar_acc, (uint32_t)run & 1u, a.err, abort_flag);
      if (!ok) break;
      tc_fence_after();
      const bool part = n != w.cnt;
      // KV: warpgroup 0 dV, 1 dK; else a half of dQ's columns each
      constexpr int kCols = KV ? D : D / 2;
      const uint32_t col0 = KV ? (wg == 0 ? 0 : C::kAcc1) : C::kAcc1 + wg * kCols;
      const float f = (KV && wg == 0) ? 1.f : a.scale;
      // rows [0, live) are the sequence's, [live, wrote) written as zeros
      const int live = min(kT, (KV ? w.u.Skv : w.u.Sq) - f0);
      const int wrote = KV && a.fill ? min(kT, a.Skv - f0) : live;
      uint16_t* out;
      size_t row_w;  // elements from row to row
      if constexpr (KV) {
        out = (wg == 0 ? a.dv : a.dk) + (((size_t)w.b * a.Skv + f0) * a.Hkv + h) * D;
        row_w = (size_t)a.Hkv * D;
      } else {
        out = a.dq + ((size_t)(w.u.qbase + f0) * a.Hq + h) * D + wg * kCols;
        row_w = (size_t)a.Hq * D;
      }
      float4* pp = reinterpret_cast<float4*>(KV ? a.part_k : a.part_q) +
                   ((size_t)blockIdx.x * 2 + (i0 > 0 ? 0 : 1)) * (kT * D * (KV ? 2 : 1) / 4) +
                   (size_t)wg * (kCols / 4) * kT + r;
#pragma unroll
      for (int c = 0; c < kCols; c += 32) {
        uint32_t v[32];
        tmem_ld32(lanes + col0 + c, v);
        tmem_wait_ld();
        if (part) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            pp[(size_t)((c + e) / 4) * kT] = make_float4(__uint_as_float(v[e]) * f, __uint_as_float(v[e + 1]) * f,
                                                         __uint_as_float(v[e + 2]) * f, __uint_as_float(v[e + 3]) * f);
        } else {
          // four lanes write 64 bytes of a row side by side: a row a lane made each store 32 lines
          uint4 q[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t* x = v + e * 8;
            q[e] = make_uint4(pack_bf16x2(__uint_as_float(x[0]) * f, __uint_as_float(x[1]) * f),
                              pack_bf16x2(__uint_as_float(x[2]) * f, __uint_as_float(x[3]) * f),
                              pack_bf16x2(__uint_as_float(x[4]) * f, __uint_as_float(x[5]) * f),
                              pack_bf16x2(__uint_as_float(x[6]) * f, __uint_as_float(x[7]) * f));
          }
          transpose4(q, lane);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = (r & ~3) + e;
            if (row < wrote)
              *reinterpret_cast<uint4*>(out + (size_t)row * row_w + c + (lane & 3) * 8) =
                  row < live ? q[e] : make_uint4(0, 0, 0, 0);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_accr);
      ++run;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ cut units, units without items
constexpr int kJoinThreads = 256;

// CTA c > 0 of the first `ctas`: the unit cut at the start of slice c, if no earlier slice cuts it
// too; the further CTAs: zeros for units without items.
template <int D, bool KV>
__device__ void join(const BackwardArgs& a, int c, int ctas, int zero_cta, int zero_ctas) {
  constexpr int kAccs = KV ? 2 : 1;
  const int* pre = KV ? a.pre_k : a.pre_q;
  const int nx = f_tiles(a, KV), n_groups = a.B * nx, H = KV ? a.Hkv : a.Hq;
  const int total = pre[n_groups];
  const int lane = threadIdx.x & 31;
  // a unit's rows: [b][f0 + r], dK/dV or dQ
  auto row_ptr = [&](const Unit& u, int b, int f0, int h, int r, int acc) -> uint16_t* {
    const int row = f0 + r;
    if constexpr (KV) {
      if (row >= (a.fill ? a.Skv : u.Skv)) return nullptr;
      return (acc == 0 ? a.dv : a.dk) + (((size_t)b * a.Skv + row) * a.Hkv + h) * D;
    } else {
      if (row >= u.Sq) return nullptr;
      return a.dq + ((size_t)(u.qbase + row) * a.Hq + h) * D;
    }
  };
  if (zero_cta >= 0) {
    for (int g = zero_cta; g < n_groups; g += zero_ctas) {
      if (pre[g + 1] != pre[g]) continue;
      const int b = g / nx, f0 = g % nx * kT;
      const Unit u = unit_of<KV>(a, b, g % nx);
      for (int i = threadIdx.x; i < kAccs * H * kT * (D / 8); i += kJoinThreads) {
        const int e = i % (D / 8), h = i / (D / 8) % H, r = i / (D / 8) / H % kT, acc = i / (D / 8) / H / kT;
        uint16_t* out = row_ptr(u, b, f0, h, r, acc);
        if (out) *reinterpret_cast<uint4*>(out + e * 8) = make_uint4(0, 0, 0, 0);
      }
    }
    if (!KV && a.cu_q && a.fill) {  // rows of no sequence
      const long long w = (long long)a.Hq * (D / 8), step = (long long)zero_ctas * kJoinThreads;
      const int c0 = min(max(a.cu_q[0], 0), a.total_q), c1 = min(max(a.cu_q[a.B], c0), a.total_q);
      for (long long i = (long long)zero_cta * kJoinThreads + threadIdx.x; i < (c0 + (long long)a.total_q - c1) * w; i += step)
        reinterpret_cast<uint4*>(a.dq)[i < c0 * w ? i : i + (c1 - c0) * w] = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const int per = slice_cost(total, ctas);
  const long long at = (long long)c * per;
  if (c == 0 || at >= total) return;
  int lo = 0, hi = n_groups;
  while (hi - lo > 1) {
    const int step = max(1, (hi - lo) / 32);
    const int p = min(lo + (lane + 1) * step, hi);
    const unsigned over = __ballot_sync(0xFFFFFFFFu, p >= hi || pre[p] > at);
    const int k = over ? __ffs(over) - 1 : 32;
    hi = k < 32 ? min(lo + (k + 1) * step, hi) : hi;
    lo = lo + k * step;
  }
  const int b = lo / nx, f0 = lo % nx * kT;
  const Unit u = unit_of<KV>(a, b, lo % nx);
  const int cnt = unit_items<KV>(a, u);
  const int cost = unit_cost(cnt), h = (int)(at - pre[lo]) / cost;
  const int u0 = pre[lo] + h * cost + kRunCost, u1 = u0 + cnt;  // the places of the unit's items
  const int c0 = u0 / per, c1 = (u1 - 1) / per;                 // its slices
  if (at <= u0 || c != c0 + 1) return;
  const float4* part = reinterpret_cast<const float4*>(KV ? a.part_k : a.part_q);
  constexpr int kSlot = kT * D * kAccs / 4;
  // 8 columns of a row at a time
  for (int i = (int)blockIdx.y * kJoinThreads + threadIdx.x; i < kAccs * (D / 8) * kT; i += kJoinThreads * gridDim.y) {
    const int r = i % kT, e = i / kT % (D / 8), acc = i / kT / (D / 8);
    const size_t off = ((size_t)acc * (D / 4) + 2 * e) * kT + r;
    const float4* p = part + ((size_t)c0 * 2 + 1) * kSlot + off;
    float4 x = __ldcg(p), y = __ldcg(p + kT);
    for (int k = c0 + 1; k <= c1; ++k) {
      p = part + (size_t)k * 2 * kSlot + off;
      const float4 x2 = __ldcg(p), y2 = __ldcg(p + kT);
      x.x += x2.x; x.y += x2.y; x.z += x2.z; x.w += x2.w;
      y.x += y2.x; y.y += y2.y; y.z += y2.z; y.w += y2.w;
    }
    uint16_t* out = row_ptr(u, b, f0, h, r, acc);
    if (out == nullptr) continue;
    const bool live = !KV || f0 + r < u.Skv;
    *reinterpret_cast<uint4*>(out + e * 8) =
        live ? make_uint4(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w), pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w))
             : make_uint4(0, 0, 0, 0);
  }
}

constexpr int kZeroCtas = 16;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) backward_join_kernel(const __grid_constant__ BackwardArgs a, int ck, int cq) {
  // dK/dV slices, dQ slices, then the units without items
  const int x = (int)blockIdx.x;
  if (x < ck) join<D, true>(a, x, ck, -1, 0);
  else if (x < ck + cq) join<D, false>(a, x - ck, cq, -1, 0);
  else {
    const int z = (x - ck - cq) * (int)gridDim.y + (int)blockIdx.y, nz = kZeroCtas * (int)gridDim.y;
    join<D, true>(a, 0, ck, z, nz);
    join<D, false>(a, 0, cq, z, nz);
  }
}

template <int D, bool KV>
cudaError_t launch_pass(const BackwardArgs& a, int ctas, cudaStream_t stream) {
  using C = BwdCfg<D, KV>;
  auto kern = backward_kernel<D, KV>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  kern<<<ctas, C::kThreads, C::kSmem, stream>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const BackwardArgs& a, cudaStream_t stream) {
  const bool any = a.total_q > 0 && a.Sq > 0 && a.Skv > 0;  // else the gradients are zeros
  const long long threads = any ? (long long)a.total_q * a.Hq * (D / 8) : 0;
  const unsigned grid = 2 + (unsigned)((threads + kPrepThreads - 1) / kPrepThreads);
  if (a.o_bf16) backward_prep_kernel<D, true><<<grid, kPrepThreads, 0, stream>>>(a);
  else backward_prep_kernel<D, false><<<grid, kPrepThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (any && e == cudaSuccess) e = launch_pass<D, true>(a, a.ctas_k, stream);
  if (any && e == cudaSuccess) e = launch_pass<D, false>(a, a.ctas_q, stream);
  if (e != cudaSuccess) return e;
  backward_join_kernel<D><<<dim3(a.ctas_k + a.ctas_q + kZeroCtas, 4), kJoinThreads, 0, stream>>>(a, a.ctas_k, a.ctas_q);
  return cudaGetLastError();
}

}  // namespace

int backward_tile_rows(int d) { return d == 64 ? BwdCfg<64, true>::TN : BwdCfg<128, true>::TN; }

cudaError_t launch_backward(const BackwardArgs& a, cudaStream_t stream) {
  switch (a.d) {
    case 64: return launch_d<64>(a, stream);
    case 128: return launch_d<128>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
