// key_weights.cu -- accumulated attention weight of every cached key.
//
//   W[b,hk,j] (+)= sum over the new rows i of sequence b and the G heads h of KV head hk of
//                  exp(scale * q[i,h] . k[j,hk] - lse[i,h]),   admissible (i, j) only,
// the column sums of the softmax whose row sums the attention call left in lse.  A key's
// sum has one owner, which adds its terms in a fixed order: no atomics, the same bits
// each time.  Two kernels, by how many query rows a KV head has in a sequence:
//   * up to kRowsMax (a decode step): the keys are streamed from HBM once and nothing else
//     matters; warp-level mma on rows gathered by each warp for itself;
//   * more: S^T = K Q^T on the tensor cores, so a key is a TMEM lane and a thread sums its
//     own row; one ex2 per pair (32 a cycle per SM) and the MMA (512 cycles per 128 x 128
//     tile at d = 128) take equally long.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "internal.h"
#include "mma.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void put_weight(const KeyWeightArgs& a, int b, int hk, int j, float w) {
  float* dst = a.weights + ((size_t)b * a.Hkv + hk) * a.w_stride + j;
  *dst = a.accumulate ? *dst + w : w;
}

// Rows of sequence b, which the launch was sized for, are at most max_sq: more are reported,
// as the positions of the first max_sq would be taken for the last ones.
__device__ __forceinline__ void check_rows(const KeyWeightArgs& a, int b) {
  if (a.cu_q == nullptr || threadIdx.x != 0) return;
  const int c0 = min(max(a.cu_q[b], 0), a.total_q), c1 = min(a.cu_q[b + 1], a.total_q);
  if (c1 - c0 > a.max_sq) atomicCAS(a.err, kErrNone, kErrBadShape);
}

// ------------------------------------------------------------------ few rows
constexpr int kRowsMax = 16;
constexpr int kRowWarps = 4;

template <int D>
struct RowCfg {
  static constexpr int kPanel = 16 * 128;
  static constexpr int kStage = 16 * D * 2;                          // K of 16 keys
  // a warp's ring: 6, 8, 16 KB.  A step is mostly a warp waiting on its own instructions, so
  // four CTAs an SM (three at d = 256) beat two of deeper rings: 64 sequences of up to 8192
  // keys 99 us against 110, 4 units of 117000 keys 23 against 33; a fifth and sixth add nothing
  static constexpr int kStages = D == 64 ? 3 : 2;
  static constexpr int kSmem = kRowWarps * kStages * kStage + 1024;
};

// One CTA per (sequence, KV head, range of `chunk` keys).  As in decode_paged.cu a warp
// gathers 16 keys at a time into its own ring and multiplies them with the resident query
// rows (up to 8 NB); a key's terms then lie in four lanes.
template <int D, int NB>
__global__ void __launch_bounds__(kRowWarps * 32, 4) key_weights_rows_kernel(const KeyWeightArgs a, int chunk) {
  using C = RowCfg<D>;
  constexpr int ST = C::kStages;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_bh = a.B * a.Hkv;
  const int bh = (int)(blockIdx.x % n_bh), hk = bh % a.Hkv, b = bh / a.Hkv;
  const int cap = a.kv.max_pages * a.kv.page_size;
  const SeqExtent e = seq_extent(b, a.cu_q ? a.max_sq : 1, cap, a.cu_q, a.kv_lens, a.total_q);
  const int base = a.cu_q ? e.qbase : b;
  const int lo = (int)(blockIdx.x / n_bh) * chunk, hi = min(e.Skv, lo + chunk);
  if (lo == 0 && hk == 0) check_rows(a, b);
  if (lo >= hi) return;
  const int G = a.Hq / a.Hkv, R = e.Sq * G;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + warp * ST * C::kStage;

  const int runs = (hi - lo + 31) / 32;
  const int n = 2 * (runs > warp ? (runs - warp + kRowWarps - 1) / kRowWarps : 0);
  auto key0 = [&](int i) { return lo + ((i >> 1) * kRowWarps + warp) * 32 + (i & 1) * 16; };
  int ri[1] = {-1}, rn[1];
  paged_rows<1>(a.kv, b, key0(0), hi, lane, a.err, rn);
  auto issue = [&](int i) {
    if (i < n) {
      if ((i & 1) == 0) {
        ri[0] = rn[0];
        if (i + 2 < n) paged_rows<1>(a.kv, b, key0(i + 2), hi, lane, a.err, rn);
      }
      paged_gather_rows<D, 16>(smem_u32(ring + (i % ST) * C::kStage), C::kPanel, a.kv.k, a.Hkv, hk, lane, ri[0],
                               (i & 1) * 16);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < ST - 1; ++i) issue(i);

  // row r: position r / G, head r % G.  This lane's columns: rows 8 nb + 2 (lane % 4) + {0, 1},
  // each with -lse log2 e and the keys it admits (j <= last, and j >= first or j < n_sink)
  const long long off = (long long)e.Skv - e.Sq;
  uint32_t qf[NB][D / 16][2];
  float nl[NB][2];
  int last[NB][2], first[NB][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int row = nb * 8 + (lane >> 2);
    load_q_frags<D>(qf[nb], [&](int r) { return a.q + ((size_t)(base + r / G) * a.Hq + hk * G + r % G) * D; }, row,
                    row < R, lane);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int r = nb * 8 + (lane & 3) * 2 + k;
      nl[nb][k] = 0.f;
      last[nb][k] = -1;  // admits nothing
      first[nb][k] = 0;
      if (r < R) {
        const int pos = r / G, h = hk * G + r % G;
        const float v = a.lse[(size_t)h * a.lse_hs + (size_t)(base + pos) * a.lse_ts];
        const long long p = (long long)pos + off;
        nl[nb][k] = -kLog2e * v;
        if (v != -INFINITY) last[nb][k] = a.causal ? (int)max(-1LL, p) : 0x7FFFFFFF;
        if (a.window > 0) first[nb][k] = (int)max(0LL, p - a.window + 1);
      }
    }
  }
  const int sink = a.window > 0 ? a.n_sink : 0;
  const float sl2 = a.scale * kLog2e;
  for (int i = 0; i < n; ++i) {
    issue(i + ST - 1);
    cp_async_wait<ST - 1>();
    __syncwarp();
    const uint32_t kt = smem_u32(ring + (i % ST) * C::kStage);
    float s[NB][4], s2[NB][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[nb][k] = s2[nb][k] = 0.f;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      uint32_t f[4];
      ldmatrix_x4(frag_keys<C::kPanel>(kt, kk, lane), f);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) mma_16816((kk & 1) ? s2[nb] : s[nb], f, qf[nb][kk][0], qf[nb][kk][1]);
    }
    float w[2] = {0.f, 0.f};  // keys j and j + 8
    const int j = key0(i) + (lane >> 2);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = k & 1, jj = j + (k >> 1) * 8;
        const float p = ex2_approx(fmaf(s[nb][k] + s2[nb][k], sl2, nl[nb][c]));
        if (jj <= last[nb][c] && (jj >= first[nb][c] || jj < sink)) w[k >> 1] += p;
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      w[0] += __shfl_xor_sync(0xFFFFFFFFu, w[0], o);
      w[1] += __shfl_xor_sync(0xFFFFFFFFu, w[1], o);
    }
    if ((lane & 3) == 0) {
      if (j < hi) put_weight(a, b, hk, j, w[0]);
      if (j + 8 < hi) put_weight(a, b, hk, j + 8, w[1]);
    }
    __syncwarp();  // every lane has read the stage before it is refilled
  }
  cp_async_wait<0>();
}

// ------------------------------------------------------------------ many rows
// CTA: 256 keys (two M = 128 tiles) of one (sequence, KV head), resident in shared memory;
// the query rows of the group's heads stream past in tiles of QN rows (whole positions).
// Two key tiles per query tile halve the query traffic from L2 (64 bytes a cycle per SM
// otherwise).  Sixteen warps sum (thread = key): a warpgroup for each key tile and parity of
// the query tile, each with a TMEM buffer of its own, read in two halves.  With eight warps
// and one wait for all of S^T a query tile took 1.4 us, its warps mostly waiting together
// for the buffers, barriers and loads; sixteen take 0.86 us, of which the exponentials are
// 0.54.  Warps 16, 19: MMA issue, one key tile each (a single warp's waits between the
// products left the tensor pipe idle for a third of the time); warp 17: query tiles by TMA;
// warp 18: their lse, by plain loads into sixteen further columns of the product,
// K' = (K, 1, 1, 1), Q' = (Q, -lse / scale in three bf16 terms), so that S^T comes out as
// q . k - lse / scale: read from shared memory under the exponentials instead, a value a
// column cost as many wavefronts as the MMA's operands.  The CTAs of a cluster share the
// keys and take every cs-th query tile; their sums meet in rank 0, in rank order.
template <int D>
struct TileCfg {
  static constexpr int QN = D == 256 ? 64 : 128;  // query rows of a tile
  static constexpr int kKeys = 256;
  static constexpr int kStages = D == 64 ? 6 : (D == 128 ? 4 : 2);  // ring of query tiles
  static constexpr int kLse = 4;                                    // ring of their lse columns
  static constexpr int kPanels = D / 64;
  static constexpr int kKPanel = 128 * 128;               // one panel of a 128-key tile
  static constexpr int kKTile = kPanels * kKPanel;
  static constexpr int kQPanel = QN * 128;
  static constexpr int kQTile = kPanels * kQPanel;
  static constexpr int kQOff = 2 * kKTile;
  // sixteen more columns of the product, without swizzle: three of ones beside the keys, and
  // -lse / scale beside the queries
  static constexpr int kOnesOff = kQOff + kStages * kQTile;  // [128 rows][16]
  static constexpr int kExtTile = QN * 32;
  static constexpr int kLseOff = kOnesOff + 128 * 32;        // [slot][QN rows][16]
  static constexpr int kSumOff = kQOff;                      // [parity][256] floats, at the end
  static constexpr int kBarOff = kLseOff + kLse * kExtTile;
  static constexpr int kNumBars = 2 * kStages + 2 * kLse + 2 * 2 * 2;  // full, empty, of each ring; S, free [tile][buf]
  static constexpr int kSmem = kBarOff + kNumBars * 8 + 16 + 1024;
  static constexpr int kSumWarps = 16;
  static constexpr int kThreads = (kSumWarps + 4) * 32;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
};

template <int D>
__global__ void __launch_bounds__(TileCfg<D>::kThreads, 1)
    key_weights_tiles_kernel(const __grid_constant__ CUtensorMap tm_q, const KeyWeightArgs a, int pack, int cs) {
  using C = TileCfg<D>;
  constexpr int QN = C::QN;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)blockIdx.x % cs;
  const int u = (int)blockIdx.x / cs, n_bh = a.B * a.Hkv;
  const int kb = u / n_bh;  // key block: under a causal mask the first ones see the most rows and start first
  const int hk = u % n_bh % a.Hkv, b = u % n_bh / a.Hkv;
  const int cap = a.kv.max_pages * a.kv.page_size;
  const SeqExtent e = seq_extent(b, a.cu_q ? a.max_sq : 1, cap, a.cu_q, a.kv_lens, a.total_q);
  const int base = a.cu_q ? e.qbase : b;
  const int k0 = kb * C::kKeys;
  if (kb == 0 && hk == 0 && rank == 0) check_rows(a, b);
  if (k0 >= e.Skv) return;  // the whole cluster: nothing of it waits on a peer
  const int Gall = a.Hq / a.Hkv, G = pack, n_hu = Gall / G;  // head groups of the KV head
  const int PT = QN / G;                  // positions of a query tile
  const long long off = (long long)e.Skv - e.Sq;  // key index of row i: i + off
  // positions [i0, i1) that admit a key of this block
  long long i0 = 0, i1 = e.Sq;
  const int k_last = min(e.Skv, k0 + C::kKeys) - 1;
  if (a.causal) i0 = max(0LL, (long long)k0 - off);
  if (a.window > 0 && k0 >= a.n_sink) i1 = min(i1, (long long)k_last + a.window - off);
  const int t0 = (int)(i0 / PT);
  const int tiles = i1 > i0 ? (int)((i1 + PT - 1) / PT) - t0 : 0;
  const int total_tiles = tiles * n_hu;
  const int n = total_tiles > rank ? (total_tiles - rank + cs - 1) / cs : 0;  // this CTA's tiles
  // i-th of them: tile index x = rank + i * cs; head group x % n_hu, positions from (t0 + x / n_hu) * PT

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem;
  uint8_t* sQ = smem + C::kQOff;
  uint8_t* sL = smem + C::kLseOff;
  float* sSum = reinterpret_cast<float*>(smem + C::kSumOff);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* empty = full + C::kStages;
  uint64_t* fullL = empty + C::kStages;
  uint64_t* emptyL = fullL + C::kLse;
  uint64_t* bar_S = emptyL + C::kLse;    // [tile][buf] S^T computed
  uint64_t* bar_F = bar_S + 4;           // [tile][buf] S^T read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_F + 4);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 2);  // both key tiles' products
    }
    for (int s = 0; s < C::kLse; ++s) {
      mbar_init(&fullL[s], 1);
      mbar_init(&emptyL[s], 2);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar_S[i], 1);
      mbar_init(&bar_F[i], 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::kSumWarps) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp < 8) {  // the block's keys: warp w gathers rows 32 w ..
    int ri[1];
    paged_rows<1>(a.kv, b, k0 + warp * 32, e.Skv, lane, a.err, ri);
    paged_gather<D, 1>(smem_u32(sK + (warp >> 2) * C::kKTile + (warp & 3) * 32 * 128), C::kKPanel, a.kv.k, a.Hkv,
                       hk, lane, ri);
    cp_async_commit();
    // rows of a query tile past its whole positions: no copy ever writes them, and as
    // zeros (with lse terms of -inf) they add nothing
    const int used = PT * G, pad = (QN - used) * 8;  // 16-byte chunks of one panel
    for (int i = threadIdx.x; i < pad * C::kPanels * C::kStages; i += 256)
      *reinterpret_cast<uint4*>(sQ + (i / pad) * C::kQPanel + used * 128 + (i % pad) * 16) = make_uint4(0, 0, 0, 0);
    // 8-row blocks of 16 bytes: columns 0-7 of row r at (r / 8) * 256 + (r % 8) * 16, then 8-15
    for (int i = threadIdx.x; i < 128 * 2; i += 256)  // ones in columns 0, 1, 2
      *reinterpret_cast<uint4*>(smem + C::kOnesOff + i * 16) =
          (i & 8) ? make_uint4(0, 0, 0, 0) : make_uint4(0x3F803F80u, 0x00003F80u, 0, 0);
    for (int i = threadIdx.x; i < C::kLse * C::kExtTile / 16; i += 256)
      *reinterpret_cast<uint4*>(sL + i * 16) = make_uint4(0, 0, 0, 0);
    cp_async_wait<0>();
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool two = k0 + 128 < e.Skv;  // the second key tile exists
  float sum = 0.f;                    // of this thread's key

  // tile i of this CTA: its head group and first position
  auto tile_at = [&](int i, int& hu, int& p0) {
    const int x = rank + i * cs, q = n_hu == 1 ? x : x / n_hu;
    hu = hk * n_hu + (x - q * n_hu);
    p0 = (t0 + q) * PT;
  };
  if (warp == C::kSumWarps + 1) {
    // ---- query tiles ----
    if (lane == 0) tma_prefetch_desc(&tm_q);
    int i = 0;
    for (; i < n; ++i) {
      const int s = i % C::kStages;
      int hu, p0;
      tile_at(i, hu, p0);
      if (!mbar_wait_warp(&empty[s], ((uint32_t)(i / C::kStages) & 1u) ^ 1u, a.err, abort_flag)) break;
      mbar_arrive_expect_tx_e(&full[s], (uint32_t)(PT * G) * 128u * C::kPanels);
#pragma unroll
      for (int q = 0; q < C::kPanels; ++q)
        tma_load_5d_e(sQ + s * C::kQTile + q * C::kQPanel, &tm_q, &full[s], q * 64, 0, hu, base + p0, 0);
    }
    if (i < n)  // aborted: the copies in flight land before shared memory is released
      for (int u = max(0, i - C::kStages); u < i; ++u)
        mbar_wait(&full[u % C::kStages], (uint32_t)(u / C::kStages) & 1u, nullptr, nullptr, 100000000ull);
  } else if (warp == C::kSumWarps + 2) {
    // ---- -lse / scale of the tiles' rows, as three bf16 terms (2^-24 of it left out), read
    // kAhead tiles before they are stored ----
    int cp[QN / 32], ch[QN / 32];  // this lane's columns: position in the tile, head (-1: no row)
#pragma unroll
    for (int k = 0; k < QN / 32; ++k) {
      const int c = k * 32 + lane;
      cp[k] = c / G;
      ch[k] = c < PT * G ? c % G : -1;
    }
    auto load_lse = [&](int i, float (&v)[QN / 32]) {
      int hu, p0;
      tile_at(i, hu, p0);
#pragma unroll
      for (int k = 0; k < QN / 32; ++k) {
        v[k] = INFINITY;
        if (ch[k] >= 0 && p0 + cp[k] < e.Sq)
          v[k] = a.lse[(size_t)(hu * G + ch[k]) * a.lse_hs + (size_t)(base + p0 + cp[k]) * a.lse_ts];
      }
    };
    const float inv_scale = 1.f / a.scale;
    constexpr int kAhead = 2;
    float v[kAhead][QN / 32];
#pragma unroll
    for (int p = 0; p < kAhead; ++p)
      if (p < n) load_lse(p, v[p]);
    bool ok = true;
    for (int i0 = 0; ok && i0 < n; i0 += kAhead) {
#pragma unroll
      for (int p = 0; p < kAhead; ++p) {
        const int i = i0 + p, s = i % C::kLse;
        if (!ok || i >= n) continue;
        ok = mbar_wait_warp(&emptyL[s], ((uint32_t)(i / C::kLse) & 1u) ^ 1u, a.err, abort_flag);
        if (!ok) continue;
#pragma unroll
        for (int k = 0; k < QN / 32; ++k) {
          const int c = k * 32 + lane;
          float x = -v[p][k] * inv_scale;
          // nothing where there is no row, or it saw no key (lse = -inf) or only infinite ones
          if (x > 1e38f || x < -1e38f) x = -1e38f;
          const uint32_t hi = pack_bf16x2(x, 0.f);
          const float r1 = x - __uint_as_float(hi << 16);
          const uint32_t mid = pack_bf16x2(r1, 0.f);
          const float r2 = r1 - __uint_as_float(mid << 16);
          *reinterpret_cast<uint2*>(sL + s * C::kExtTile + (c >> 3) * 256 + (c & 7) * 16) =
              make_uint2((hi & 0xFFFFu) | mid << 16, pack_bf16x2(r2, 0.f));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&fullL[s]);
        if (i + kAhead < n) load_lse(i + kAhead, v[p]);
      }
    }
  } else if (warp == C::kSumWarps || warp == C::kSumWarps + 3) {
    // ---- MMA: S^T of one key tile (a missing second one only counts on the slots) ----
    const int t = warp == C::kSumWarps ? 0 : 1;
    constexpr uint32_t idesc = idesc_bf16_f32(128, QN, 0, 0);
    const uint64_t dk = smem_desc(smem_u32(sK + t * C::kKTile), 16, 1024, kSwizzle128B);
    const uint64_t dq0 = smem_desc(smem_u32(sQ), 16, 1024, kSwizzle128B);
    const uint64_t d1 = smem_desc(smem_u32(smem + C::kOnesOff), 128, 256, kSwizzleNone);
    const uint64_t dl0 = smem_desc(smem_u32(sL), 128, 256, kSwizzleNone);
    for (int i = 0; i < n; ++i) {
      const int s = i % C::kStages, sl = i % C::kLse, buf = i & 1;
      const uint32_t ph_f = ((uint32_t)(i >> 1) & 1u) ^ 1u, ph_q = (uint32_t)(i / C::kStages) & 1u,
                     ph_l = (uint32_t)(i / C::kLse) & 1u;
      const bool free_f = t == 1 && !two;  // no product, no buffer to wait for
      // all three at once (a trip to each barrier in turn is three times the time, and the
      // tensor pipe runs dry under it), and one by one only where they are not ready
      const bool r0 = free_f || mbar_test(&bar_F[t * 2 + buf], ph_f);
      const bool r1 = mbar_test(&full[s], ph_q), r2 = mbar_test(&fullL[sl], ph_l);
      if (!__all_sync(0xFFFFFFFFu, r0 & r1 & r2)) {
        if (!free_f && !mbar_wait_warp(&bar_F[t * 2 + buf], ph_f, a.err, abort_flag)) break;
        if (!mbar_wait_warp(&full[s], ph_q, a.err, abort_flag)) break;
        if (!mbar_wait_warp(&fullL[sl], ph_l, a.err, abort_flag)) break;
      }
      if (t == 0 || two) {
        tc_fence_after();
        const uint64_t dq = dq0 + (uint64_t)((s * C::kQTile) >> 4);
        const uint32_t d_tmem = tmem + (t * 2 + buf) * 128;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t ok_ = (uint64_t)(((kk >> 2) * C::kKPanel + (kk & 3) * 32) >> 4);
          const uint64_t oq_ = (uint64_t)(((kk >> 2) * C::kQPanel + (kk & 3) * 32) >> 4);
          mma_ss_e(d_tmem, dk + ok_, dq + oq_, idesc, kk > 0 ? 1u : 0u);
        }
        mma_ss_e(d_tmem, d1, dl0 + (uint64_t)((sl * C::kExtTile) >> 4), idesc, 1u);
        mma_commit_e(&bar_S[t * 2 + buf]);
      }
      mma_commit_e(&empty[s]);
      mma_commit_e(&emptyL[sl]);
    }
  } else if (warp < C::kSumWarps) {
    // ---- sums ----
    const int t = (warp >> 2) & 1, par = warp >> 3, r = (warp & 3) * 32 + lane;
    const int j = k0 + t * 128 + r;  // this thread's key
    const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float sl2 = a.scale * kLog2e;
    const uint64_t sl2x2 = f2pack(sl2, sl2);
    const int j_lo = k0 + t * 128, j_hi = j_lo + 127;
    float acc = 0.f;
    bool ok = true;
    for (int i = par; i < n && (t == 0 || two); i += 2) {
      const int buf = par;
      int hu, p0;
      tile_at(i, hu, p0);
      const bool got = mbar_wait(&bar_S[t * 2 + buf], (uint32_t)(i >> 1) & 1u, a.err, abort_flag);
      if (!__all_sync(0xFFFFFFFFu, got)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // columns [c_lo, c_hi) admit this thread's key (a column's position: p0 + c / G)
      int c_lo = 0, c_hi = (int)min((long long)(PT * G), ((long long)e.Sq - p0) * G);
      const long long d0 = (long long)j - off - p0;  // first causal position, tile-relative
      const bool edge = e.Sq - p0 < PT || (a.causal && j_hi > (long long)p0 + off) ||
                        (a.window > 0 && j_hi >= a.n_sink && j_lo <= (long long)p0 + PT - 1 + off - a.window);
      if (edge) {
        if (a.causal && d0 > 0) c_lo = (int)min((long long)QN, d0 * G);
        if (a.window > 0 && j >= a.n_sink) {
          const long long w = d0 + a.window;
          c_hi = w <= 0 ? 0 : (int)min((long long)c_hi, w * G);
        }
      }
      const uint32_t s_addr = lane_addr + (t * 2 + buf) * 128;
      uint64_t a0 = f2pack(0.f, 0.f), a1 = a0;
      uint32_t sr[64];
      auto terms = [&](int c0, auto edge_tag) {  // EDGE: some columns may not admit the key
        constexpr bool EDGE = decltype(edge_tag)::value;
#pragma unroll
        for (int c = 0; c < 64; c += 4) {
          float x0, x1, x2, x3;
          f2unpack(mul2(f2pack(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), sl2x2), x0, x1);
          f2unpack(mul2(f2pack(__uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3])), sl2x2), x2, x3);
          float p[4] = {ex2_approx(x0), ex2_approx(x1), ex2_approx(x2), ex2_approx(x3)};
          if constexpr (EDGE) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (c0 + c + k < c_lo || c0 + c + k >= c_hi) p[k] = 0.f;
          }
          a0 = add2(a0, f2pack(p[0], p[1]));
          a1 = add2(a1, f2pack(p[2], p[3]));
        }
      };
#pragma unroll
      for (int c0 = 0; c0 < QN; c0 += 64) {
        tmem_ld32(s_addr + c0, sr);
        tmem_ld32(s_addr + c0 + 32, sr + 32);
        tmem_wait_ld();
        if (c0 + 64 == QN) {  // all of S^T has been read: the MMA may overwrite it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_F[t * 2 + buf]);
        }
        if (edge) terms(c0, std::true_type{});
        else terms(c0, std::false_type{});
      }
      float s0, s1;
      f2unpack(add2(a0, a1), s0, s1);
      acc += s0 + s1;
    }
    sum = ok ? acc : NAN;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::kSumWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  } else if (warp < C::kSumWarps) {  // the query ring is free: its last tile has been read
    sSum[threadIdx.x] = sum;  // [parity][key]
  }
  if (cs > 1) cluster_sync_all();  // every rank's sums are written
  else __syncthreads();
  if (rank == 0 && threadIdx.x < C::kKeys) {
    const int j = k0 + (int)threadIdx.x;
    float w = sum + sSum[C::kKeys + threadIdx.x];
    for (int r = 1; r < cs; ++r)
      w += ld_cluster_f32(mapa_shared(smem_u32(sSum + threadIdx.x), (uint32_t)r)) +
           ld_cluster_f32(mapa_shared(smem_u32(sSum + C::kKeys + threadIdx.x), (uint32_t)r));
    if (j < e.Skv) put_weight(a, b, hk, j, w);
  }
  if (cs > 1) cluster_sync_all();  // and read before their CTA's shared memory goes
}

template <int D>
cudaError_t launch_rows(const KeyWeightArgs& a, int rows, cudaStream_t stream) {
  using C = RowCfg<D>;
  const long long units = (long long)a.B * a.Hkv;
  const int cap = a.kv.max_pages * a.kv.page_size;
  // ranges of 128 to 2048 keys: one wave of four CTAs an SM if that is enough (4 units of 32000
  // keys: 7 us, 9 with ranges of half the length, 12 of a quarter)
  const long long share = (units * cap + 4 * 152 - 1) / (4 * 152);
  const int chunk = (int)std::min(2048LL, std::max(1LL, (share + 127) / 128) * 128);
  auto kern = rows <= 8 ? key_weights_rows_kernel<D, 1> : key_weights_rows_kernel<D, 2>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)(units * ((cap + chunk - 1) / chunk)), kRowWarps * 32, C::kSmem, stream>>>(a, chunk);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_tiles(const KeyWeightArgs& a, cudaStream_t stream) {
  using C = TileCfg<D>;
  auto kern = key_weights_tiles_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const int cap = a.kv.max_pages * a.kv.page_size;
  const int blocks = (cap + C::kKeys - 1) / C::kKeys;
  const long long units = (long long)blocks * a.B * a.Hkv;
  const int PT = C::QN / a.pack;
  const long long q_tiles = ((long long)a.max_sq + PT - 1) / PT * (a.Hq / a.Hkv / a.pack);
  // CTAs of a cluster, while SMs are idle and each keeps two query tiles: clusters of four
  // reach nearly every SM, of eight 120 of them (15 clusters), so eight only where all run at
  // once (52 units of a 3314-token prompt: 84, 48, 73 us in clusters of 2, 4, 8)
  int cs = 1;
  while (cs < 4 && units * cs < 152 && q_tiles >= 4 * cs) cs *= 2;
  if (cs == 4 && units <= 15 && q_tiles >= 16) cs = 8;
  cudaLaunchConfig_t cfg = {};
  if (units * cs > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  cfg.gridDim = dim3((unsigned)(units * cs));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cs;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a.tm_q, a, (int)a.pack, cs);
}

}  // namespace

bool key_weights_few_rows(int max_sq, int G) { return (long long)max_sq * G <= kRowsMax; }
int key_weights_q_rows(int d) { return d == 256 ? TileCfg<256>::QN : TileCfg<128>::QN; }

cudaError_t launch_key_weights(const KeyWeightArgs& a, cudaStream_t stream) {
  const bool few = key_weights_few_rows(a.max_sq, a.Hq / a.Hkv);
  const int rows = a.max_sq * (a.Hq / a.Hkv);
  switch (a.d) {
    case 64: return few ? launch_rows<64>(a, rows, stream) : launch_tiles<64>(a, stream);
    case 128: return few ? launch_rows<128>(a, rows, stream) : launch_tiles<128>(a, stream);
    case 256: return few ? launch_rows<256>(a, rows, stream) : launch_tiles<256>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
