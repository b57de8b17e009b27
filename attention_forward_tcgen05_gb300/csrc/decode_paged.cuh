// decode_paged.cuh -- the kernel of decode_paged.cu and decode_window.cu: one-token GQA decode over
// a paged cache, split-KV partials and their LSE-weighted merge in one launch, the split rule and
// combine of decode.cu.
//
// One CTA per (sequence, KV head, split), groups of up to 16 query heads; its warps take
// 32-key runs of the split in turn and share nothing until the end.  Each warp gathers 16
// keys of K and V at a time into a ring of its own (cp.async groups: no barrier, no
// producer warp), and does on its own fragments
//   S^T = K Q^T        16 keys x 8 heads per mma, the queries resident in registers,
//   P = 2^(S - m),     m a running reference that is moved (and O rescaled) only when a
//                      score exceeds it by 2^8, so that the usual step needs no maximum
//                      across lanes; it cancels in O / l,
//   O^T += V^T P^T     P^T by movmatrix from the score fragments.
// O, l and m are fp32.  P goes into the product as bf16 terms.  For a bf16 output two (the
// value and its remainder: at most 2^-17 of P left out).  For an fp32 output three (2^-25),
// and each step's product starts from zero and is added to O in fp32, as the mma's own
// accumulation truncates: against fp64 on 131k keys that is off by 5e-7 of O, two terms
// accumulated in the mma by 2.9e-6, fp32 matrix products by 9e-7; the third term costs 1.5 %
// where HBM bounds and 15 % with 16 heads.  With heads as the 8-wide side of the
// mma a step of 16 keys costs about 250 warp instructions at d = 128 against 700 on fp32
// cores per head group of 4, and the kernel runs at the rate of the gathers.
#pragma once
#include <cmath>

#include "decode_common.cuh"
#include "internal.h"
#include "mma.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr float kMoveThreshold = 8.f;  // log2: the reference m moves when a score exceeds it by 2^8

// CTAs of one SM (also the split rule's)
constexpr int decode_paged_ctas(int d, int nb) { return d == 256 ? 1 : (nb == 2 ? 2 : (d == 128 ? 3 : 4)); }

template <int D, int NB, int W>
struct DecodePagedCfg {
  static constexpr int kHeads = 8 * NB;
  static constexpr int kPanel = 16 * 128;          // one 64-column panel of 16 keys
  static constexpr int kTile = 16 * D * 2;         // K or V of 16 keys
  static constexpr int kStage = 2 * kTile;
  // A step of 16 keys takes a warp 0.7 us, mostly waiting on its own instructions, so an SM
  // needs many warps more than deep rings.  Narrow CTAs (W = 4) share it and hide one another's
  // start and end: three at d = 128 (1024 units of about 550 keys: 51 us against 53 with two of
  // three stages; 64 ragged sequences of up to 8192: 192 against 210), four at d = 64 (64 x 8
  // units of up to 8000 keys: 106 us, 116 with three of four stages, 110 with five of two).  A
  // wide CTA has an SM to itself, for calls of few CTAs (4 units of 16000 keys in 32 splits: 13.8
  // us with 8 warps, 14.2 with 12, 18.7 with 4, whatever their rings' depth; d = 64, 6 units of
  // up to 131072: 38 us with 12 or 16 warps, 41 with 8), and at d = 256, where 6 warps of two
  // stages fill it (64 x 4 units of up to 4000 keys: 123 us, 140 with 4).
  static constexpr int kStages =
      W > 4 ? 196608 / (W * kStage) : (D == 64 && NB == 2 ? 4 : (D == 128 && NB == 1 ? 2 : 3));
  static constexpr int kAhead = W > 4 ? kStages / 2 + 1 : 1;  // runs whose pool rows are known ahead
  static constexpr int kRing = W * kStages * kStage;
  static constexpr int kComb = W * kHeads * (D + 2) * 4;
  static constexpr int kSmem = (kRing > kComb ? kRing : kComb) + 1024;
  static constexpr int kMinBlocks = W > 4 ? 1 : decode_paged_ctas(D, NB);
};

// F32: the output is fp32 (see above); else bf16.
// WIN (a.window, a.n_sink; decode_window.cu): the split's rows are those of the list of admitted keys,
// the sinks before the window and then the window, [0, ns) and [ns + gap, L); no other key's page is
// looked up.  Groups of more than 16 heads then take a.head_ctas CTAs, a.cta_heads heads each (they
// share the keys through L2).
template <int D, int NB, bool F32, int W, bool WIN>
__global__ void __launch_bounds__(W * 32, DecodePagedCfg<D, NB, W>::kMinBlocks)
    decode_paged_kernel(const DecodeArgs a) {
  using C = DecodePagedCfg<D, NB, W>;
  constexpr int ST = C::kStages, AH = C::kAhead;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int G = a.Hq / a.Hkv, head0 = 0;  // heads of this CTA, the first of them in the group
  const int n_h = WIN ? a.Hkv * a.head_ctas : a.Hkv;
  const int pos = (int)(blockIdx.x / n_h);
  int hk = (int)(blockIdx.x % n_h);
  const int b = pos / a.n_splits, s_idx = pos % a.n_splits;
  if constexpr (WIN) {
    head0 = hk % a.head_ctas * a.cta_heads;
    hk /= a.head_ctas;
  }
  const size_t orow0 = (size_t)b * a.Hq + (size_t)hk * G + head0;  // (sequence, first query head)
  if constexpr (WIN) G = min(a.cta_heads, G - head0);
  int L = a.kv_lens[b];
  L = L < 0 ? 0 : (L > a.max_kv ? a.max_kv : L);
  int ns = 0, gap = 0;  // row u of the list is key u, or u + gap from ns on
  if constexpr (WIN) {
    const int first = L > a.window ? L - a.window : 0;
    ns = min(a.n_sink, first);
    gap = first - ns;
    L -= gap;
  }
  long long chunk = ((long long)L + a.n_splits - 1) / a.n_splits;
  if (chunk < a.min_rows) chunk = a.min_rows;
  if (chunk < 1) chunk = 1;
  const long long lo_ll = (long long)s_idx * chunk, hi_ll = lo_ll + chunk;
  const int lo = (int)(lo_ll < L ? lo_ll : L), hi = (int)(hi_ll < L ? hi_ll : L);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));

  // one split is the result itself: no partials, no merge
  auto put = [&](int g, int t, float x, float lse) {
    const size_t row = orow0 + g;
    if (a.n_splits > 1) {
      a.part_o[(row * a.n_splits + s_idx) * D + t] = x;
      if (t == 0) a.part_lse[row * a.n_splits + s_idx] = lse;
    } else {
      if (a.o_bf16) reinterpret_cast<uint16_t*>(a.o)[row * D + t] = (uint16_t)pack_bf16x2(x, 0.f);
      else reinterpret_cast<float*>(a.o)[row * D + t] = x;
      if (t == 0) a.lse[row] = lse;
    }
  };
  if (lo >= hi) {  // empty split: o = 0, lse = -inf
    for (int i = threadIdx.x; i < G * D; i += W * 32) put(i / D, i % D, 0.f, -INFINITY);
  } else {
    uint8_t* ring = smem + warp * ST * C::kStage;
    // this warp's 16-key steps: step i covers keys from lo + ((i / 2) * W + warp) * 32 + (i % 2) * 16
    const int runs = (hi - lo + 31) / 32;
    const int n = 2 * (runs > warp ? (runs - warp + W - 1) / W : 0);
    auto key0 = [&](int i) { return lo + ((i >> 1) * W + warp) * 32 + (i & 1) * 16; };
    int ri = -1, rn[AH][1];  // pool rows of the run being issued, and of the next ones
    auto rows_of = [&](int j0, int (&out)[1]) {
      if constexpr (WIN) {
        const int u = j0 + lane;
        out[0] = u < hi ? paged_row(a.kv, b, u < ns ? u : u + gap, a.err) : -1;
      } else {
        paged_rows<1>(a.kv, b, j0, hi, lane, a.err, out);
      }
    };
#pragma unroll
    for (int r = 0; r < AH; ++r)
      if (2 * r < n || r == 0) rows_of(key0(2 * r), rn[r]);
    auto issue = [&](int i) {
      if (i < n) {
        if ((i & 1) == 0) {
          ri = rn[0][0];
#pragma unroll
          for (int r = 0; r + 1 < AH; ++r) rn[r][0] = rn[r + 1][0];
          if (i + 2 * AH < n) rows_of(key0(i + 2 * AH), rn[AH - 1]);
        }
        const uint32_t dst = smem_u32(ring + (i % ST) * C::kStage);
        paged_gather_rows<D, 16>(dst, C::kPanel, a.kv.k, a.Hkv, hk, lane, ri, (i & 1) * 16);
        paged_gather_rows<D, 16>(dst + C::kTile, C::kPanel, a.kv.v, a.Hkv, hk, lane, ri, (i & 1) * 16);
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) issue(i);

    uint32_t qf[NB][D / 16][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int g = nb * 8 + (lane >> 2);
      load_q_frags<D>(qf[nb], [&](int r) { return a.q + (orow0 + r) * D; }, g, g < G, lane);
    }
    float o[NB][D / 16][4], m[NB][2], l[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      m[nb][0] = m[nb][1] = -INFINITY;
      l[nb][0] = l[nb][1] = 0.f;
#pragma unroll
      for (int t = 0; t < D / 16; ++t) o[nb][t][0] = o[nb][t][1] = o[nb][t][2] = o[nb][t][3] = 0.f;
    }
    const float sl2 = a.scale * kLog2e;

    for (int i = 0; i < n; ++i) {
      issue(i + ST - 1);
      cp_async_wait<ST - 1>();
      __syncwarp();
      const uint32_t kt = smem_u32(ring + (i % ST) * C::kStage), vt = kt + C::kTile;
      // S^T: key lane / 4 (+ 8), heads 2 (lane % 4) + {0, 1}; two chains along the head dim
      float s[NB][4], s2[NB][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nb][e] = s2[nb][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t f[4];
        ldmatrix_x4(frag_keys<C::kPanel>(kt, kk, lane), f);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) mma_16816((kk & 1) ? s2[nb] : s[nb], f, qf[nb][kk][0], qf[nb][kk][1]);
      }
      const int left = hi - key0(i);  // keys of this step that exist (may be <= 0)
      bool move = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[nb][e] = (s[nb][e] + s2[nb][e]) * sl2;
          if (left < 16 && (lane >> 2) + (e >> 1) * 8 >= left) s[nb][e] = -INFINITY;
          move = move || s[nb][e] > m[nb][e & 1] + kMoveThreshold;
        }
      }
      if (__any_sync(0xFFFFFFFFu, move)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(s[nb][e], s[nb][e + 2]);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, off));
            const float mn = fmaxf(m[nb][e], x);
            const float c = m[nb][e] == mn ? 1.f : ex2_approx(m[nb][e] - mn);
            m[nb][e] = mn;
            l[nb][e] *= c;
#pragma unroll
            for (int t = 0; t < D / 16; ++t) {
              o[nb][t][e] *= c;
              o[nb][t][e + 2] *= c;
            }
          }
        }
      }
      uint32_t ph[NB][2], pl[NB][2], pr[NB][2];  // P^T in three terms
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // keys lane / 4 + 8 h
          // (a warp whose keys are all missing so far has m = -inf: no term)
          const float p0 = m[nb][0] == -INFINITY ? 0.f : ex2_approx(s[nb][2 * h] - m[nb][0]);
          const float p1 = m[nb][1] == -INFINITY ? 0.f : ex2_approx(s[nb][2 * h + 1] - m[nb][1]);
          l[nb][0] += p0;
          l[nb][1] += p1;
          const uint32_t v = pack_bf16x2(p0, p1);
          const float r0 = p0 - __uint_as_float(v << 16), r1 = p1 - __uint_as_float(v & 0xFFFF0000u);
          const uint32_t w = pack_bf16x2(r0, r1);
          ph[nb][h] = movmatrix_trans(v);
          pl[nb][h] = movmatrix_trans(w);
          if constexpr (F32)
            pr[nb][h] = movmatrix_trans(pack_bf16x2(r0 - __uint_as_float(w << 16), r1 - __uint_as_float(w & 0xFFFF0000u)));
        }
      }
#pragma unroll
      for (int t = 0; t < D / 16; ++t) {
        uint32_t f[4];
        ldmatrix_x4_trans(frag_dims<C::kPanel>(vt, t, lane), f);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if constexpr (F32) {
            float c[4] = {0.f, 0.f, 0.f, 0.f};
            mma_16816(c, f, pr[nb][0], pr[nb][1]);
            mma_16816(c, f, pl[nb][0], pl[nb][1]);
            mma_16816(c, f, ph[nb][0], ph[nb][1]);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[nb][t][k] += c[k];
          } else {
            mma_16816(o[nb][t], f, ph[nb][0], ph[nb][1]);
            mma_16816(o[nb][t], f, pl[nb][0], pl[nb][1]);
          }
        }
      }
      __syncwarp();  // every lane has read the stage before it is refilled
    }

    // ---- the warps' (m, l, O) through shared memory ----
    cp_async_wait<0>();
    __syncthreads();
    float* comb = reinterpret_cast<float*>(smem);  // [warp][head][D + 2]
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[nb][e];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
        float* cw = comb + (warp * C::kHeads + nb * 8 + (lane & 3) * 2 + e) * (D + 2);
#pragma unroll
        for (int t = 0; t < D / 16; ++t) {
          cw[t * 16 + (lane >> 2)] = o[nb][t][e];
          cw[t * 16 + 8 + (lane >> 2)] = o[nb][t][e + 2];
        }
        if (lane < 4) {
          cw[D] = m[nb][e];
          cw[D + 1] = x;
        }
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < G * D; i += W * 32) {
      const int g = i / D, t = i % D;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < W; ++w) M = fmaxf(M, comb[(w * C::kHeads + g) * (D + 2) + D]);
      float ls = 0.f, acc = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float* cw = comb + (w * C::kHeads + g) * (D + 2);
        const float f = ex2_approx(cw[D] - M);  // warps without keys: m = -inf -> 0
        ls = fmaf(cw[D + 1], f, ls);
        acc = fmaf(cw[t], f, acc);
      }
      put(g, t, acc / ls, (M + log2f(ls)) * kLn2);
    }
  }
  if (a.n_splits == 1) return;
  // (partials loaded at once: 8, 16 or 24 took 22.4, 21.3, 21.0 us for 48 splits of 4 units)
  constexpr int kBatch = D == 256 ? 16 : 24;
  combine_if_last<D, W, kBatch>(a.done + orow0, a.n_splits, a.part_o, a.part_lse, a.o, a.lse, orow0, G, a.o_bf16,
                             [] { __syncthreads(); });
}

template <int D, int NB, int W, bool WIN>
cudaError_t launch_t(const DecodeArgs& a, cudaStream_t stream) {
  using C = DecodePagedCfg<D, NB, W>;
  auto kern = a.o_bf16 ? decode_paged_kernel<D, NB, false, W, WIN> : decode_paged_kernel<D, NB, true, W, WIN>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const long long ctas = (long long)a.B * a.n_splits * a.Hkv * (WIN ? a.head_ctas : 1);
  if (ctas > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  kern<<<(unsigned)ctas, W * 32, C::kSmem, stream>>>(a);
  return cudaGetLastError();
}

// A CTA takes a whole group of up to 16 heads (decode_paged: larger ones run on the prefill's tiles,
// paged_api.cu).
template <int D, int NB, bool WIN>
cudaError_t launch_nb(const DecodeArgs& a, cudaStream_t stream) {
  const long long ctas = (long long)a.B * a.n_splits * a.Hkv * (WIN ? a.head_ctas : 1);
  if constexpr (D == 256) return launch_t<D, NB, NB == 1 ? 6 : 4, WIN>(a, stream);  // (two mma sides: registers for 4)
  else if (ctas <= 152) return launch_t<D, NB, D == 64 && NB == 1 ? 12 : 8, WIN>(a, stream);
  else return launch_t<D, NB, 4, WIN>(a, stream);
}
template <int D, bool WIN>
cudaError_t launch_d(const DecodeArgs& a, cudaStream_t stream) {
  return (WIN ? a.cta_heads : a.Hq / a.Hkv) <= 8 ? launch_nb<D, 1, WIN>(a, stream) : launch_nb<D, 2, WIN>(a, stream);
}
template <bool WIN>
cudaError_t launch_paged_decode(const DecodeArgs& a, cudaStream_t stream) {
  switch (a.d) {
    case 64: return launch_d<64, WIN>(a, stream);
    case 128: return launch_d<128, WIN>(a, stream);
    case 256: return launch_d<256, WIN>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace
}  // namespace attn
