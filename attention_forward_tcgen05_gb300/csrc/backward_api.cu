// backward_api.cu -- the C ABI of the prefill's gradients (include/attn.h): argument
// validation, the workspace's layout and the launches of prefill_backward.cuh.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "attn.h"
#include "internal.h"

namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool ok16(const void* p) { return p != nullptr && aligned(p, 16); }
bool ok4(const void* p) { return p != nullptr && aligned(p, 4); }

// Sizes common to the two forms; rows: of q in all, Sq / Skv: of the longest sequence.
struct Sizes {
  int B, Hq, Hkv;
  long long rows;
  int Sq, Skv, d;
};

int check_sizes(const Sizes& z) {
  if (z.B < 0 || z.Hq < 1 || z.Hkv < 1 || z.Hq % z.Hkv != 0 || z.rows < 0 || z.Sq < 0 || z.Skv < 0)
    return ATTN_ERR_INVALID_ARG;
  if (z.d != 64 && z.d != 128) return ATTN_ERR_UNSUPPORTED;
  if (z.rows * z.Hq >= (1LL << 31) || (long long)z.B * z.Skv * z.Hkv >= (1LL << 31)) return ATTN_ERR_INVALID_ARG;
  if ((long long)z.Hq * z.d >= (1LL << 31)) return ATTN_ERR_INVALID_ARG;
  // items of all heads, 16 more a block for its run's cost (prefill_backward.cuh): counted in 32 bits, a
  // CTA's share of them beyond the last
  const long long tq = (z.Sq + 63LL) / 64, tk = (z.Skv + 63LL) / 64, heads = (long long)z.B * z.Hq;
  auto over = [&](long long blocks, long long items) {
    return (double)heads * (double)blocks * (double)(items + 16) > 2e9;
  };
  if (over((tk + 1) / 2, tq) || over((tq + 1) / 2, tk)) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

// Byte offsets of the workspace's parts.
struct Layout {
  size_t pre[4], joined, stat, ext1, ext2, part_k, part_q, bytes;
  int ctas;
};
Layout layout_of(const Sizes& z) {
  Layout l;
  const long long tq = (z.Sq + 127LL) / 128, tk = (z.Skv + 127LL) / 128;
  // one CTA an SM, none without an item of its own (two for two forms)
  l.ctas = (int)std::max(2LL, std::min<long long>(attn::kBackwardCtas, tq * z.B * tk * z.Hq));
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t p = at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  for (int i = 0; i < 4; ++i) l.pre[i] = take((size_t)(z.B * (i % 2 == 0 ? tk : tq) + 1) * 4);
  l.joined = take((size_t)4 * attn::kBackwardCtas * 4);
  l.stat = take((size_t)z.rows * z.Hq * 8);
  l.ext1 = take(((size_t)z.rows * z.Hq + 128) * 16);
  l.ext2 = take(((size_t)z.rows * z.Hq + 128) * 16);
  l.part_k = take((size_t)l.ctas * 2 * 128 * z.d * 2 * 4);
  l.part_q = take((size_t)l.ctas * 2 * 128 * z.d * 4);
  l.bytes = at;
  return l;
}

int backward_impl(const attn_bf16_t* dout, const attn_bf16_t* q, const attn_bf16_t* k, const attn_bf16_t* v,
                  const void* o, const float* lse, const float* dlse, attn_bf16_t* dq, attn_bf16_t* dk,
                  attn_bf16_t* dv, const int* cu_q, const int* kv_lens, const Sizes& z, int causal, int window,
                  int n_sink, float scale, int o_dtype, int fill, void* work, unsigned long long work_bytes,
                  attn_stream_t stream) {
  int rc = check_sizes(z);
  if (rc != ATTN_OK) return rc;
  if (window < 0 || n_sink < 0 || (window > 0 && !causal)) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || scale <= 0.f) return ATTN_ERR_INVALID_ARG;
  // (lse / scale is formed)
  if (scale < 1e-30f || scale > 1e30f || (o_dtype != ATTN_F32 && o_dtype != ATTN_BF16)) return ATTN_ERR_UNSUPPORTED;
  const bool rows = z.rows > 0, keys = z.Skv > 0;
  if (z.B == 0 || (!rows && !keys)) return ATTN_OK;
  if (rows && (!ok16(dout) || !ok16(q) || !ok16(o) || !ok4(lse) || !aligned(dlse, 4) || !ok16(dq)))
    return ATTN_ERR_INVALID_ARG;
  if (keys && (!ok16(k) || !ok16(v) || !ok16(dk) || !ok16(dv))) return ATTN_ERR_INVALID_ARG;
  const Layout l = layout_of(z);
  if (!work || !aligned(work, 256) || work_bytes < l.bytes) return ATTN_ERR_INVALID_ARG;
  // one pass's gradients are written while the other still reads, the workspace all along
  const long long nq = z.rows * z.Hq, nk = (long long)z.B * z.Skv * z.Hkv;
  struct Bytes {
    const void* p;
    long long n;
  };
  const Bytes written[4] = {{dq, nq * z.d * 2}, {dk, nk * z.d * 2}, {dv, nk * z.d * 2}, {work, (long long)l.bytes}};
  const Bytes read[9] = {{dout, nq * z.d * 2}, {q, nq * z.d * 2}, {o, nq * z.d * (o_dtype == ATTN_BF16 ? 2 : 4)},
                         {k, nk * z.d * 2}, {v, nk * z.d * 2}, {lse, nq * 4}, {dlse, nq * 4},
                         {cu_q, (z.B + 1LL) * 4}, {kv_lens, z.B * 4LL}};
  auto meet = [](const Bytes& x, const Bytes& y) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
    return a && b && x.n > 0 && y.n > 0 && a < b + y.n && b < a + x.n;
  };
  for (int i = 0; i < 4; ++i) {
    for (const Bytes& x : read)
      if (meet(written[i], x)) return ATTN_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (meet(written[i], written[j])) return ATTN_ERR_INVALID_ARG;
  }
  attn::BackwardArgs a;
  std::memset(&a, 0, sizeof(a));
  // (the longest sequence has the most pairs; shorter ones of a packed batch may have few all the same)
  const bool two = attn::backward_two_terms(z.Sq, z.Skv, causal, window, n_sink);
  a.forms = two ? attn::kTwoTerms : (cu_q ? attn::kOneTerm | attn::kTwoTerms : attn::kOneTerm);
  const bool any = rows && keys && z.Sq > 0;  // else the gradients are zeros
  if (any) {
    // packed rows are one batch slab
    const int ns = cu_q ? (int)z.rows : z.Sq, nb = cu_q ? 1 : z.B;
    rc = attn::encode_panel_map(&a.tm_q, q, z.d, z.Hq, ns, nb, 128);
    if (rc == ATTN_OK) rc = attn::encode_panel_map(&a.tm_do, dout, z.d, z.Hq, ns, nb, 128);
    if (rc == ATTN_OK) rc = attn::encode_panel_map(&a.tm_k, k, z.d, z.Hkv, z.Skv, z.B, 128);
    if (rc == ATTN_OK) rc = attn::encode_panel_map(&a.tm_v, v, z.d, z.Hkv, z.Skv, z.B, 128);
    // (tiles of 64 rows: BwdCfg::TN)
    const bool fine = (a.forms & attn::kTwoTerms) != 0, kv64 = fine || z.d == 128;
    if (rc == ATTN_OK && kv64) rc = attn::encode_panel_map(&a.tm_q64, q, z.d, z.Hq, ns, nb, 64);
    if (rc == ATTN_OK && kv64) rc = attn::encode_panel_map(&a.tm_do64, dout, z.d, z.Hq, ns, nb, 64);
    if (rc == ATTN_OK && fine) rc = attn::encode_panel_map(&a.tm_k64, k, z.d, z.Hkv, z.Skv, z.B, 64);
    if (rc == ATTN_OK && fine) rc = attn::encode_panel_map(&a.tm_v64, v, z.d, z.Hkv, z.Skv, z.B, 64);
    if (rc != ATTN_OK) return rc;
  }
  a.dout = dout; a.o = o; a.lse = lse; a.dlse = dlse;
  a.dq = dq; a.dk = dk; a.dv = dv;
  a.cu_q = cu_q; a.kv_lens = kv_lens;
  a.B = z.B; a.Hq = z.Hq; a.Hkv = z.Hkv; a.Sq = z.Sq; a.Skv = z.Skv; a.total_q = (int)z.rows; a.d = z.d;
  a.causal = causal ? 1 : 0; a.window = window; a.n_sink = n_sink;
  a.o_bf16 = o_dtype == ATTN_BF16 ? 1 : 0;
  a.scale = scale;
  a.fill = fill ? 1 : 0;
  uint8_t* w = static_cast<uint8_t*>(work);
  for (int i = 0; i < 4; ++i) a.pre[i] = reinterpret_cast<int*>(w + l.pre[i]);
  a.joined = reinterpret_cast<int*>(w + l.joined);
  a.stat = reinterpret_cast<float2*>(w + l.stat);
  a.ext1 = reinterpret_cast<uint4*>(w + l.ext1);
  a.ext2 = reinterpret_cast<uint4*>(w + l.ext2);
  a.part_k = reinterpret_cast<float*>(w + l.part_k);
  a.part_q = reinterpret_cast<float*>(w + l.part_q);
  a.ctas = l.ctas;
  a.err = attn::device_err_word();
  if (a.err == nullptr) return ATTN_ERR_CUDA;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = attn::launch_backward_prep(a, any, s);
  if (e == cudaSuccess && any)
    e = two ? attn::launch_backward_fine(a, s) : (cu_q ? attn::launch_backward_packed(a, s) : attn::launch_backward(a, s));
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

extern "C" {

unsigned long long attn_prefill_backward_workspace(int B, int Hq, int Hkv, long long total_q, int max_sq, int max_kv,
                                                   int d) {
  const Sizes z{B, Hq, Hkv, total_q, max_sq, max_kv, d};
  return check_sizes(z) == ATTN_OK ? (unsigned long long)layout_of(z).bytes : 0ull;
}

int attn_prefill_backward(const attn_bf16_t* dout, const attn_bf16_t* q, const attn_bf16_t* k, const attn_bf16_t* v,
                          const void* o, const float* lse, const float* dlse, attn_bf16_t* dq, attn_bf16_t* dk,
                          attn_bf16_t* dv, int B, int Hq, int Hkv, int Sq, int Skv, int d, int causal, int window,
                          int n_sink, float scale, int o_dtype, void* work, unsigned long long work_bytes,
                          attn_stream_t stream) {
  const Sizes z{B, Hq, Hkv, (long long)B * Sq, Sq, Skv, d};
  return backward_impl(dout, q, k, v, o, lse, dlse, dq, dk, dv, nullptr, nullptr, z, causal, window, n_sink, scale,
                       o_dtype, 1, work, work_bytes, stream);
}

int attn_prefill_varlen_backward(const attn_bf16_t* dout, const attn_bf16_t* q, const attn_bf16_t* kcache,
                                 const attn_bf16_t* vcache, const void* o, const float* lse, const float* dlse,
                                 attn_bf16_t* dq, attn_bf16_t* dkcache, attn_bf16_t* dvcache, const int* cu_seqlens_q,
                                 const int* kv_lens, int B, int Hq, int Hkv, int total_q, int max_sq, int max_kv,
                                 int d, int causal, int window, int n_sink, float scale, int o_dtype, int fill,
                                 void* work, unsigned long long work_bytes, attn_stream_t stream) {
  const Sizes z{B, Hq, Hkv, total_q, max_sq, max_kv, d};
  if (B > 0 && (!ok4(cu_seqlens_q) || !ok4(kv_lens))) {
    const int rc = check_sizes(z);
    return rc != ATTN_OK ? rc : ATTN_ERR_INVALID_ARG;
  }
  return backward_impl(dout, q, kcache, vcache, o, lse, dlse, dq, dkcache, dvcache, cu_seqlens_q, kv_lens, z, causal,
                       window, n_sink, scale, o_dtype, fill, work, work_bytes, stream);
}

}  // extern "C"
