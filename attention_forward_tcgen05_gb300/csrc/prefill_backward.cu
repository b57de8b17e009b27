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
// Warps: 0-7 softmax (thread = row of F; warpgroup w takes 64 of the tile's 128 columns),
// 8 MMA issue, 9 / 10 the rings of Y1 and Y2, 11 the F tiles.
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
constexpr int kRunCost = 2;
constexpr int kMinCost = 2 + kRunCost;  // of a slice

template <int D, bool KV>
struct BwdCfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kPanel = kT * 128;
  static constexpr int kTile = kPanels * kPanel;
  static constexpr int NS = (KV && D == 128) ? 1 : 2;                    // S buffers
  static constexpr int kSt1 = D == 64 ? 4 : (KV ? 2 : 3);                // ring of Y1
  static constexpr int kSt2 = D == 64 ? 4 : 2;                           // ring of Y2
  static constexpr int kY1Off = 2 * kTile;
  static constexpr int kY2Off = kY1Off + kSt1 * kTile;
  // lse and D columns of a Q tile (16 bytes a row), the ones beside K, beside V, and zeros:
  // the second eight columns of all of them
  static constexpr int kExt = KV ? kT * 16 : 0;
  static constexpr int kExtOff = kY2Off + kSt2 * kTile;
  static constexpr int kOnesLOff = kExtOff + kSt1 * kExt;
  static constexpr int kOnesDOff = kOnesLOff + kExt;
  static constexpr int kZeroOff = kOnesDOff + kExt;
  static constexpr int kBarOff = kZeroOff + kExt;
  static constexpr int kNumBars = 2 * kSt1 + 2 * kSt2 + 2 + NS + 2 + 2 * NS + 2;
  static constexpr int kSmem = kBarOff + kNumBars * 8 + 16 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static constexpr uint32_t kAcc1 = KV ? D : 0;  // TMEM columns; acc0 at 0
  static constexpr uint32_t kS = kAcc1 + D;
  static constexpr uint32_t kDP = kS + NS * 128;
  static_assert(kDP + 128 <= 512, "TMEM budget");
  static constexpr int kThreads = 384;
  static constexpr int kSoftRegs = 208, kCtlRegs = 80;  // as in the forward kernels: 63488 <= 384 * 168
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
    u.t0 = (int)(lo / kT);
    u.nt = (int)((hi + kT - 1) / kT) - u.t0;
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
  a.ext[i] = make_uint4(l0 | l1 << 16, l2 | d0 << 16, d1 | d2 << 16, 0u);
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
  __device__ __forceinline__ ItemWalk(const BackwardArgs& a, const Unit& u, int unit_head, int i) {
    if constexpr (KV) {
      const int q = i / u.nt;
      h = unit_head * (a.Hq / a.Hkv) + q;
      t = i - q * u.nt;
      row0 = (u.t0 + t) * kT;
    } else {
      h = unit_head / (a.Hq / a.Hkv);
      t = i;
      row0 = tile_list_key(u.tl, t) * kT;
    }
  }
  __device__ __forceinline__ void step(const Unit& u) {
    ++t;
    if constexpr (KV) {
      if (t == u.nt) {
        t = 0;
        ++h;
      }
      row0 = (u.t0 + t) * kT;
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

template <int D, bool KV>
__global__ void __launch_bounds__(BwdCfg<D, KV>::kThreads, 1)
    backward_kernel(const __grid_constant__ BackwardArgs a) {
  using C = BwdCfg<D, KV>;
  constexpr int NS = C::NS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const CUtensorMap &tm_f1 = KV ? a.tm_k : a.tm_q, &tm_f2 = KV ? a.tm_v : a.tm_do;
  const CUtensorMap &tm_y1 = KV ? a.tm_q : a.tm_k, &tm_y2 = KV ? a.tm_do : a.tm_v;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full1 = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* empty1 = full1 + C::kSt1;
  uint64_t* full2 = empty1 + C::kSt1;
  uint64_t* empty2 = full2 + C::kSt2;
  uint64_t* fullF = empty2 + C::kSt2;
  uint64_t* emptyF = fullF + 1;
  uint64_t* bar_S = emptyF + 1;        // [NS] S computed
  uint64_t* bar_dP = bar_S + NS;       // dP computed
  uint64_t* bar_dPr = bar_dP + 1;      // dP read
  uint64_t* bar_P = bar_dPr + 1;       // [NS] P stored
  uint64_t* bar_dS = bar_P + NS;       // [NS] dS stored
  uint64_t* bar_acc = bar_dS + NS;     // a run's sums complete
  uint64_t* bar_accr = bar_acc + 1;    // they are read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_accr + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kSt1; ++s) { mbar_init(&full1[s], 1); mbar_init(&empty1[s], 1); }
    for (int s = 0; s < C::kSt2; ++s) { mbar_init(&full2[s], 1); mbar_init(&empty2[s], 1); }
    mbar_init(fullF, 1);
    mbar_init(emptyF, 1);
    for (int s = 0; s < NS; ++s) { mbar_init(&bar_S[s], 1); mbar_init(&bar_P[s], 8); mbar_init(&bar_dS[s], 8); }
    mbar_init(bar_dP, 1);
    mbar_init(bar_dPr, 8);
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
    for (int i = threadIdx.x; i < kT; i += C::kThreads) {  // row i: columns 0-2, 3-5, none
      *reinterpret_cast<uint4*>(smem + C::kOnesLOff + i * 16) = make_uint4(0x3F803F80u, 0x00003F80u, 0, 0);
      *reinterpret_cast<uint4*>(smem + C::kOnesDOff + i * 16) = make_uint4(0, 0x3F800000u, 0x3F803F80u, 0);
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
  if (warp >= 8) {
    setmaxnreg_dec<C::kCtlRegs>();
    if (warp == 9 || warp == 10) {
      // ---- rings of Y1 (warp 9, with the lse and D columns) and Y2 (warp 10) ----
      const bool first = warp == 9;
      const CUtensorMap* map = first ? &tm_y1 : &tm_y2;
      uint64_t* full = first ? full1 : full2;
      uint64_t* empty = first ? empty1 : empty2;
      const int stages = first ? C::kSt1 : C::kSt2;
      uint8_t* ring = smem + (first ? C::kY1Off : C::kY2Off);
      const uint16_t* base = KV ? (first ? a.q : a.dout) : (first ? a.k : a.v);
      const int Hy = KV ? a.Hq : a.Hkv;
      if (lane == 0) tma_prefetch_desc(map);
      int it = 0;
      bool ok = true;
      while (ok && w.next(h, i0, n)) {
        ItemWalk<KV> y(a, w.u, h, i0);
        const int rows = KV ? w.u.Sq : w.u.Skv;        // Y rows of the sequence
        const bool slab = KV ? a.cu_q != nullptr : a.kv_lens != nullptr;  // other rows may follow them
        const int row_base = KV ? w.u.qbase : w.u.kbase;
        for (int m = 0; m < n; ++m, ++it, y.step(w.u)) {
          const int s = it % stages;
          ok = mbar_wait_warp(&empty[s], ((uint32_t)(it / stages) & 1u) ^ 1u, a.err, abort_flag);
          if (!ok) break;
          uint8_t* dst = ring + s * C::kTile;
          uint32_t bytes = 0;
          const bool whole = !slab || y.row0 + kT <= rows;
          if (!whole) {
            // a sequence's last rows: gathered, so that the rows behind them arrive as zeros
            // (a weight of zero times what lies there could be NaN)
            int ri[kT / 32];
#pragma unroll
            for (int k = 0; k < kT / 32; ++k) {
              const int r = y.row0 + k * 32 + lane;
              ri[k] = r < rows ? row_base + r : -1;
            }
            paged_gather<D, kT / 32>(smem_u32(dst), C::kPanel, base, Hy, y.h, lane, ri);
            cp_async_commit();
            cp_async_wait<0>();
            fence_proxy_async_smem();
            __syncwarp();
          } else {
            bytes = C::kTile;
          }
          if (KV && first) bytes += C::kExt;
          if (bytes) mbar_arrive_expect_tx_e(&full[s], bytes);
          else if (lane == 0) mbar_arrive(&full[s]);
          if (whole) {
#pragma unroll
            for (int p = 0; p < C::kPanels; ++p) {
              if (slab && KV) tma_load_4d_e(dst + p * C::kPanel, map, &full[s], p * 64, y.h, row_base + y.row0, 0);
              else tma_load_4d_e(dst + p * C::kPanel, map, &full[s], p * 64, y.h, y.row0, w.b);
            }
          }
          if (KV && first) {
            const size_t i = a.cu_q ? (size_t)y.h * a.total_q + row_base + y.row0
                                    : ((size_t)w.b * a.Hq + y.h) * a.Sq + y.row0;
            bulk_load_e(smem + C::kExtOff + s * C::kExt, a.ext + i, C::kExt, &full[s]);
          }
        }
      }
      if (!ok)  // aborted: the copies in flight land before shared memory is released
        for (int v = max(0, it - stages); v < it; ++v)
          mbar_wait(&full[v % stages], (uint32_t)(v / stages) & 1u, nullptr, nullptr, 100000000ull);
    } else if (warp == 11) {
      // ---- F tiles of the runs ----
      if (lane == 0) {
        tma_prefetch_desc(&tm_f1);
        tma_prefetch_desc(&tm_f2);
      }
      int run = 0;
      bool ok = true;
      while (ok && w.next(h, i0, n)) {
        ok = mbar_wait_warp(emptyF, ((uint32_t)run & 1u) ^ 1u, a.err, abort_flag);
        if (!ok) break;
        mbar_arrive_expect_tx_e(fullF, 2 * C::kTile);
        const bool packed = !KV && a.cu_q != nullptr;
        const int row = packed ? w.u.qbase + w.x * kT : w.x * kT, bb = packed ? 0 : w.b;
#pragma unroll
        for (int p = 0; p < C::kPanels; ++p) {
          tma_load_4d_e(smem + p * C::kPanel, &tm_f1, fullF, p * 64, h, row, bb);
          tma_load_4d_e(smem + C::kTile + p * C::kPanel, &tm_f2, fullF, p * 64, h, row, bb);
        }
        ++run;
      }
      if (!ok && run > 0) mbar_wait(fullF, (uint32_t)(run - 1) & 1u, nullptr, nullptr, 100000000ull);
    } else {
      // ---- MMA issue ----
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, kT, 0, 0);
      constexpr uint32_t idesc_a = idesc_bf16_f32(128, D, 0, 1);
      const uint64_t df1 = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
      const uint64_t df2 = smem_desc(smem_u32(smem + C::kTile), 16, 1024, kSwizzle128B);
      const uint64_t dy1 = smem_desc(smem_u32(smem + C::kY1Off), 16, 1024, kSwizzle128B);
      const uint64_t dy2 = smem_desc(smem_u32(smem + C::kY2Off), 16, 1024, kSwizzle128B);
      const uint64_t my1 = smem_desc(smem_u32(smem + C::kY1Off), C::kPanel, 1024, kSwizzle128B);
      const uint64_t my2 = smem_desc(smem_u32(smem + C::kY2Off), C::kPanel, 1024, kSwizzle128B);
      // the two products' first halves run one item ahead of the second ones: `ahead` walks
      // the slice in front of w
      Walk<KV> ahead = w;
      int ah, ai0, an = 0, am = 0, arun = -1, ait = 0;  // item ait, the am-th of its run's an
      bool ok = true, more = true;
      auto advance = [&] {  // to the next item of `ahead`
        ++am;
        if (am >= an) {
          more = ahead.next(ah, ai0, an);
          am = 0;
          ++arun;
        }
      };
      auto issue_s = [&]() -> bool {  // S of item ait
        const int s = ait % C::kSt1;
        if (am == 0 && !mbar_wait_warp(fullF, (uint32_t)arun & 1u, a.err, abort_flag)) return false;
        if (!mbar_wait_warp(&full1[s], (uint32_t)(ait / C::kSt1) & 1u, a.err, abort_flag)) return false;
        tc_fence_after();
        const uint64_t y = dy1 + (uint64_t)((s * C::kTile) >> 4);
        const uint32_t d = tmem + C::kS + (ait % NS) * 128;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t o = (uint64_t)(((kk >> 2) * C::kPanel + (kk & 3) * 32) >> 4);
          mma_ss_e(d, df1 + o, y + o, idesc_s, kk > 0 ? 1u : 0u);
        }
        if constexpr (KV) {
          const uint32_t e = smem_u32(smem + C::kExtOff + s * C::kExt);
          const uint32_t z = smem_u32(smem + C::kZeroOff), l = smem_u32(smem + C::kOnesLOff);
          mma_ss_e(d, smem_desc(l, z - l, 128, kSwizzleNone), smem_desc(e, z - e, 128, kSwizzleNone), idesc_s, 1u);
        }
        mma_commit_e(&bar_S[ait % NS]);
        return true;
      };
      auto issue_dp = [&]() -> bool {  // dP of item ait (its F tiles and, KV, its Y1 slot have been waited for)
        const int s = ait % C::kSt2, s1 = ait % C::kSt1;
        if (KV && NS == 1) {  // here dP runs ahead of S
          if (am == 0 && !mbar_wait_warp(fullF, (uint32_t)arun & 1u, a.err, abort_flag)) return false;
          if (!mbar_wait_warp(&full1[s1], (uint32_t)(ait / C::kSt1) & 1u, a.err, abort_flag)) return false;
        }
        if (!mbar_wait_warp(&full2[s], (uint32_t)(ait / C::kSt2) & 1u, a.err, abort_flag)) return false;
        if (ait > 0 && !mbar_wait_warp(bar_dPr, (uint32_t)(ait - 1) & 1u, a.err, abort_flag)) return false;
        tc_fence_after();
        const uint64_t y = dy2 + (uint64_t)((s * C::kTile) >> 4);
        const uint32_t d = tmem + C::kDP;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t o = (uint64_t)(((kk >> 2) * C::kPanel + (kk & 3) * 32) >> 4);
          mma_ss_e(d, df2 + o, y + o, idesc_s, kk > 0 ? 1u : 0u);
        }
        if constexpr (KV) {
          const uint32_t e = smem_u32(smem + C::kExtOff + s1 * C::kExt);
          const uint32_t z = smem_u32(smem + C::kZeroOff), l = smem_u32(smem + C::kOnesDOff);
          mma_ss_e(d, smem_desc(l, z - l, 128, kSwizzleNone), smem_desc(e, z - e, 128, kSwizzleNone), idesc_s, 1u);
        }
        mma_commit_e(bar_dP);
        if constexpr (!KV) mma_commit_e(&empty2[s]);
        return true;
      };
      // acc (+)= A (TMEM, 64 columns of bf16 pairs in two halves) * Y (MN-major)
      auto issue_acc = [&](uint32_t acc, uint32_t p, uint64_t y, bool fresh) {
#pragma unroll
        for (int kk = 0; kk < kT / 16; ++kk)
          mma_ts_e(tmem + acc, p + (kk >> 2) * 64 + (kk & 3) * 8, y + (uint64_t)(kk * (2048 >> 4)), idesc_a,
                   (!fresh || kk > 0) ? 1u : 0u);
      };
      am = an = 0;
      more = ahead.next(ah, ai0, an);
      arun = 0;
      if (more) {
        ok = issue_s() && issue_dp();
        if (ok && am == an - 1) mma_commit_e(emptyF);
      }
      int it = 0, run = 0;
      while (ok && w.next(h, i0, n)) {
        for (int m = 0; ok && m < n; ++m, ++it) {
          const int buf = it % NS, s1 = it % C::kSt1, s2 = it % C::kSt2;
          const uint32_t sb = tmem + C::kS + buf * 128, ph = (uint32_t)(it / NS) & 1u;
          advance();
          ++ait;
          // the next item's first products, under this one's softmax; those of another unit
          // (whose F tiles are still on their way) after this one's second products
          const bool early = more && am > 0;
          if (early) {
            if (NS > 1) ok = issue_s();
            if (ok) ok = issue_dp();
            if (NS > 1 && ok && am == an - 1) mma_commit_e(emptyF);
          }
          if (ok && m == 0 && run > 0) ok = mbar_wait_warp(bar_accr, (uint32_t)(run - 1) & 1u, a.err, abort_flag);
          if constexpr (KV) {
            ok = ok && mbar_wait_warp(&bar_P[buf], ph, a.err, abort_flag);
            if (!ok) break;
            tc_fence_after();
            issue_acc(0, sb, my2 + (uint64_t)((s2 * C::kTile) >> 4), m == 0);
            mma_commit_e(&empty2[s2]);
          }
          ok = ok && mbar_wait_warp(&bar_dS[buf], ph, a.err, abort_flag);
          if (!ok) break;
          tc_fence_after();
          issue_acc(C::kAcc1, sb + (KV ? 32 : 0), my1 + (uint64_t)((s1 * C::kTile) >> 4), m == 0);
          mma_commit_e(&empty1[s1]);
          if (m == n - 1) mma_commit_e(bar_acc);
          if (early ? NS == 1 : more) {
            ok = issue_s();
            if (ok && !early) ok = issue_dp();
            if (ok && am == an - 1) mma_commit_e(emptyF);
          }
        }
        ++run;
      }
    }
  } else {
    setmaxnreg_inc<C::kSoftRegs>();
    // ---- softmax: P and dS ----
    const int wg = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float sl2 = a.scale * kLog2e;
    const uint64_t sl2x2 = f2pack(sl2, sl2);
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
      for (int m = 0; m < n; ++m, ++it, y.step(w.u)) {
        const int buf = it % NS;
        const uint32_t sc = lanes + C::kS + buf * 128 + wg * 64;
        ok = mbar_wait_warp(&bar_S[buf], (uint32_t)(it / NS) & 1u, a.err, abort_flag);
        if (!ok) break;
        tc_fence_after();
        uint32_t s[64], p[64];
        tmem_ld32(sc, s);
        tmem_ld32(sc + 32, s + 32);
        ok = mbar_wait_warp(bar_dP, (uint32_t)it & 1u, a.err, abort_flag);
        if (!ok) {
          tmem_wait_ld();
          break;
        }
        tc_fence_after();
        tmem_ld32(lanes + C::kDP + wg * 64, p);
        tmem_ld32(lanes + C::kDP + wg * 64 + 32, p + 32);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_dPr);
        // columns of this thread's row: [lo, hi) and, dQ pass, those before `sink`
        int lo = 0, hi = kT, sink = 0;
        bool mask;
        const int c0 = wg * 64;
        if constexpr (KV) {
          const long long d0 = w.u.off + y.row0;  // key index of the tile's first row
          const int j = f0 + r;
          mask = y.row0 + kT > w.u.Sq;
          hi = min(kT, w.u.Sq - y.row0);
          if (a.causal) {
            mask = mask || f0 + kT - 1 > d0;
            lo = (int)min((long long)kT, max(0LL, j - d0));
          }
          if (a.window > 0) {
            mask = mask || f0 + (long long)a.window < d0 + kT;
            if (j >= a.n_sink) hi = (int)min((long long)hi, max(0LL, j + (long long)a.window - d0));
          }
        } else {
          const long long pos = f0 + r + w.u.off;  // key index of this row
          const long long p0 = f0 + w.u.off;
          mask = y.row0 + kT > w.u.Skv;
          hi = min(kT, w.u.Skv - y.row0);
          if (a.causal) {
            mask = mask || y.row0 + kT - 1 > p0;
            hi = (int)min((long long)hi, max(0LL, pos + 1 - y.row0));
          }
          if (a.window > 0) {
            mask = mask || y.row0 <= p0 + kT - 1 - a.window;
            lo = (int)min((long long)kT, max(0LL, pos - a.window + 1 - y.row0));
            sink = min(kT, max(0, a.n_sink - y.row0));
          }
        }
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          const uint64_t x = f2pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
          float e0, e1;
          f2unpack(KV ? mul2(x, sl2x2) : fma2(x, sl2x2, nlse2), e0, e1);
          e0 = ex2_approx(e0);
          e1 = ex2_approx(e1);
          s[c] = __float_as_uint(e0);
          s[c + 1] = __float_as_uint(e1);
        }
        // this thread's columns as bits (a weight out of them may be inf, dP of a column that is no
        // row anything: both products' operands are cleared after their rounding)
        uint32_t in[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
        if (mask) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int c1 = c0 + q * 32;
            in[q] = (bits_below(hi - c1) & ~bits_below(lo - c1)) | bits_below(min(sink, hi) - c1);
          }
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
        uint32_t t[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          uint64_t g = f2pack(__uint_as_float(p[2 * c]), __uint_as_float(p[2 * c + 1]));
          if constexpr (!KV) g = add2(g, ndd);
          float x0, x1;
          f2unpack(mul2(g, f2pack(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1]))), x0, x1);
          t[c] = pack_bf16x2(x0, x1);
        }
        if (mask) {
          keep_bits<16>(t, in[0]);
          keep_bits<16>(t + 16, in[1]);
        }
        tmem_st32(sc + (KV ? 32 : 0), t);
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
      const int row = f0 + r;
      uint16_t* out = nullptr;
      bool live = true;
      if constexpr (KV) {
        if (row < (a.fill ? a.Skv : w.u.Skv)) out = (wg == 0 ? a.dv : a.dk) + (((size_t)w.b * a.Skv + row) * a.Hkv + h) * D;
        live = row < w.u.Skv;
      } else if (row < w.u.Sq) {
        out = a.dq + ((size_t)(w.u.qbase + row) * a.Hq + h) * D + wg * kCols;
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
        } else if (out) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t q[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              q[k] = live ? pack_bf16x2(__uint_as_float(v[e + 2 * k]) * f, __uint_as_float(v[e + 2 * k + 1]) * f) : 0u;
            *reinterpret_cast<uint4*>(out + c + e) = make_uint4(q[0], q[1], q[2], q[3]);
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

cudaError_t launch_backward(const BackwardArgs& a, cudaStream_t stream) {
  switch (a.d) {
    case 64: return launch_d<64>(a, stream);
    case 128: return launch_d<128>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
