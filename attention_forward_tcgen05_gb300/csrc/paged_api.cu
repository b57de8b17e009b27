// paged_api.cu -- the C ABI of the paged-cache serving calls (include/attn.h): argument
// validation and launches of rope.cu, prefill_paged.cu, decode_paged.cu, decode_window.cu,
// key_weights.cu and evict.cu.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <utility>

#include "attn.h"
#include "internal.h"

namespace {

constexpr int kSms = 152;               // SMs of a GB300
constexpr long long kMaxKeys = 1LL << 30;  // keys of one sequence's table, slots of a pool

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool ok16(const void* p) { return p != nullptr && aligned(p, 16); }
bool ok4(const void* p) { return p != nullptr && aligned(p, 4); }
bool ok_dim(int d) { return d == 64 || d == 128 || d == 256; }
bool ok_scale(float s) { return std::isfinite(s) && s > 0.f; }
int from_cuda(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }
cudaStream_t stream_of(attn_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// Sizes of a cache: a table [B][max_pages] over a pool, or (no table) one page of
// page_size keys per sequence.
int check_cache(const int* table, int B, int max_pages, int page_size, int num_pages) {
  if (max_pages < 1 || page_size < 1 || num_pages < 0) return ATTN_ERR_INVALID_ARG;
  if ((long long)max_pages * page_size > kMaxKeys || (long long)num_pages * page_size > 2 * kMaxKeys - 1)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(table, 4)) return ATTN_ERR_INVALID_ARG;
  if (table == nullptr && (max_pages != 1 || num_pages < B)) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

int check_heads(int B, int Hq, int Hkv) {
  return B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 ? ATTN_ERR_INVALID_ARG : ATTN_OK;
}

// Bytes of a slot (its Hkv rows), which the row gathers hold in 32 bits.
int check_slot(int Hkv, int d) { return (long long)Hkv * d >= (1LL << 31) ? ATTN_ERR_INVALID_ARG : ATTN_OK; }

// Bytes [p + t * stride, p + t * stride + width) for t in [0, n) (stride >= width), and whether two such
// sets meet.
struct ByteRows {
  const void* p;
  long long stride, width, n;
};
bool rows_overlap(ByteRows a, ByteRows b) {
  for (ByteRows* x : {&a, &b}) {
    if (x->p == nullptr || x->n <= 0 || x->width <= 0) return false;
    if (x->stride == x->width) *x = ByteRows{x->p, x->n * x->width, x->n * x->width, 1};
  }
  if (a.n > b.n) std::swap(a, b);
  const long long d = (long long)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
  auto down = [](long long x, long long y) { return x / y - (x % y < 0); };
  if (a.stride == b.stride) {
    // rows i of a and j of b meet where -b.width < d + (j - i) * stride < a.width: at most two j - i
    const long long m0 = down(-d, a.stride);
    for (long long m = m0; m <= m0 + 1; ++m)
      if (m > -a.n && m < b.n && d + m * a.stride > -b.width && d + m * a.stride < a.width) return true;
    return false;
  }
  if (d >= (a.n - 1) * a.stride + a.width || d + (b.n - 1) * b.stride + b.width <= 0) return false;
  for (long long i = 0; i < a.n; ++i) {  // (one row, but where both have gaps of their own)
    const long long at = i * a.stride - d;                                  // of the row, from b's first
    const long long j = std::max(0LL, down(at - b.width, b.stride) + 1);  // the first row of b that ends behind it
    if (j < b.n && j * b.stride < at + a.width) return true;
  }
  return false;
}

attn::PagedKV cache(const attn_bf16_t* k, const attn_bf16_t* v, const int* table, int max_pages, int page_size,
                    int num_pages) {
  return attn::PagedKV{k, v, table, max_pages, page_size, num_pages, 0};
}

// Whether a decode runs on the prefill's tensor-core tiles, a group's heads as their rows,
// instead of on warp-level mma, where heads above 8 cost as much again and above 16 read
// their keys again.  A tile's start and end take 7 us, so bf16 outputs of groups of 9 to 16
// go there while one wave of tiles holds them (64 units of up to 8000 keys, groups of 16: 38
// against 52 us; 256 units of up to 300 keys: 20 against 13 us), larger groups always (64
// units, groups of 32: 38 against 74 us; at d = 256, groups of 20: 68 against 134 us).  fp32
// outputs of up to 16 heads stay: the tiles keep P to two terms, mma to three.
bool decode_on_tiles(int B, int Hq, int Hkv, int o_dtype) {
  const int G = Hq / Hkv;
  return G > 16 || (G > 8 && o_dtype == ATTN_BF16 && (long long)B * Hkv <= kSms);
}

// Query heads that share a tile of `rows` rows: the largest divisor of G whose whole
// positions fill at least 7/8 of the tile (1 always does).
int pack_heads(int G, int rows) {
  for (int p = G < rows ? G : rows; p > 1; --p)
    if (G % p == 0 && rows / p * p * 8 >= rows * 7) return p;
  return 1;
}

// Key splits of a prefill over pages with `pack` heads a tile, and their least rows.
int prefill_splits(int B, int Hq, int total_q, int max_sq, int max_kv, int d, int pack, int* min_rows) {
  const int pos = attn::kPrefillTileM / pack;
  const bool halves = d <= 128 && max_sq <= pos;
  // blocks of query rows that exist, one unit each, and a unit's time for a tile of keys
  const long long block = d <= 128 && !halves ? 2 * pos : pos;
  const long long blocks = std::min<long long>((long long)total_q / block + B, (max_sq + block - 1) / block * B);
  const long long units = std::max(1LL, blocks * (Hq / pack));
  const double tile_us = halves ? 1.2 : (d == 64 ? 1.4 : 1.8);
  const double tiles = (max_kv + 127LL) / 128;
  // One wave of units takes its longest; several take their sum's share and half of a longest.
  // A batch's sequences are 0.6 or 0.8 of the longest on average, the two weighted alike: with
  // 0.6 alone 4 chunks of 8 rows over 8000 keys got 13 splits, a second wave (29 us; 21 with 8).
  // The partials go out and come in again, and the merge is a launch.
  double best = 0;
  int n_best = 1;
  for (int n = 1; n <= 32 && n <= std::max(1.0, tiles / 2); ++n) {
    const double rows = std::ceil(tiles / n);  // of a split, in tiles
    const double longest = rows * tile_us + 8.0;
    double us = 0;
    for (const double mean : {B > 1 ? 0.6 : 1.0, B > 1 ? 0.8 : 1.0}) {
      const double live =
          (double)units * std::max(1.0, std::min((double)n, mean * tiles / rows + (n > 1 && B > 1 ? 0.5 : 0)));
      us += live <= kSms ? longest : ((double)units * mean * tiles * tile_us + live * 8.0) / kSms + 0.5 * longest;
      if (n > 1) us += 4.0 + (double)total_q * Hq * d * 8.0 * n * mean / 5.0e6;
    }
    if (n == 1 || us < best * 0.97) {
      best = us;
      n_best = n;
    }
  }
  *min_rows = (int)std::min(std::ceil(tiles / n_best) * 128, (double)0x7FFFFF80);
  return n_best;
}

// Key splits of a decode on warp-level mma, `units` CTAs a split of up to `heads` query heads over at
// most max_kv keys, and their least rows.
int mma_splits(double units, int heads, int B, int max_kv, int d, int* min_rows) {
  const long long alone = (long long)(kSms / units);  // splits of a unit while each has an SM
  long long n;
  if (alone >= (d == 256 ? 1 : 4)) {
    // one CTA of many warps an SM; above 32 splits only of 1024 keys and more, as the merge
    // grows with them (4 units of 16000 keys: 13.8 us with 32, 14.9 with 38; of 117000: 48 with
    // 38, 52 with 19; one unit of 100000: 24 with 64, 31 with 32)
    n = std::min(std::min(alone, 64LL), std::max(32LL, max_kv / 1024LL));
  } else if (alone == 1 && max_kv <= 2048) {
    n = 1;  // short sequences whole, with an SM each (128 units: 15.8 us, 21 with narrow CTAs)
  } else {
    // as many narrow CTAs as run at once.  A batch's lengths differ, so a few splits are
    // rounded up (64 units of up to 8000 keys: 26.6 us with 8 splits, 29.3 with 2 wide ones);
    // from half a wave of units on, whole sequences do best (1024 units of up to 1000 keys: 51
    // against 59 us)
    const double q = attn::decode_paged_slots(d, heads, kSms) / units;
    n = q < 2 ? 1 : (long long)(q <= 8 && B > 1 ? std::ceil(q) : q);
  }
  n = std::max(1LL, std::min(n, (max_kv + 191LL) / 192));
  *min_rows = n > 1 ? 192 : 1;
  return (int)n;
}

// The same for the windowed decode, whose sequences are mostly as long as the window: the splits of
// least estimated time.  A call's start and end take 7.5 us and a merge 4 and more; a warp takes 0.7 us
// for 16 keys (more with two mma sides or d = 256) while HBM keeps up; launches of up to an SM's worth of
// CTAs run wide ones (decode_paged.cuh), others waves of narrow ones, the last of which is not
// full.  (512 units of 4100 keys, a wave and an eighth whole: 173 us whole, 160 in three; 1024 units of
// 260: 37 whole, 60 in two; 64 units of 2000, groups of 20: 18 whole, 25 in five; 8 units of 4100: 29
// whole, 14 in 19.)
int window_splits(double units, int heads, int keys, int d, int* min_rows) {
  const bool two = heads > 8;  // mma sides
  const double step = 0.7 * (two ? 1.2 : 1.0) * (d == 256 ? 2.0 : 1.0) / 16;
  const int wide = d == 256 ? (two ? 4 : 6) : (d == 64 && !two ? 12 : 8);
  const double slots = attn::decode_paged_slots(d, heads, kSms);
  const double row_us = 4.0 * d / 6.5e6;  // of K and V of a key at the rate of HBM
  double best = 0;
  int n_best = 1;
  for (int n = 1; n <= 64 && n <= std::max(1, (keys + 63) / 64); ++n) {
    const double rows = std::ceil((double)keys / n), ctas = units * n;
    double us = 7.5 + (n > 1 ? 4.0 + 0.08 * n : 0.0);
    if (ctas <= kSms) {
      us += std::max(rows * step / wide, ctas * rows * row_us);
    } else {
      const double full = std::floor(ctas / slots), rest = ctas - full * slots;
      us += full * (1.5 + std::max(rows * step / 4, slots * rows * row_us));
      if (rest > 0) us += std::max(rows * step / 4, rest * rows * row_us);
    }
    if (n == 1 || us < best * 0.99) {
      best = us;
      n_best = n;
    }
  }
  *min_rows = n_best > 1 ? 64 : 1;
  return n_best;
}

// Query heads of a CTA of the windowed decode and its CTAs a group: groups of more than 16 are shared
// evenly.
int window_head_ctas(int G) { return (G + attn::kMaxHeadsPerCta - 1) / attn::kMaxHeadsPerCta; }

// The launches of a prefill over pages (arguments checked, a.pack and the rows set): query and
// output maps over [nb][ns][Hq][d], pool maps, the kernel, and the merge of key splits into
// m.
int launch_paged(attn::PrefillArgs& a, const attn_bf16_t* q, int ns, int nb, attn::MergeArgs& m, cudaStream_t s) {
  a.err = attn::device_err_word();
  if (a.err == nullptr) return ATTN_ERR_CUDA;
  int rc = attn::encode_q_map(&a.tm_q, q, a.d, a.pack, a.Hq, ns, nb, attn::kPrefillTileM);
  a.o_tma = (a.o_bf16 && a.n_splits <= 1) ? 1 : 0;
  if (rc == ATTN_OK && a.o_tma) rc = attn::encode_q_map(&a.tm_o, a.o, a.d, a.pack, a.Hq, ns, nb, attn::kPrefillTileM);
  // Tensor copies of the largest power of two of rows (8 to 128; the swizzle repeats every 8)
  // that divides the page; other pages are gathered.  Pages of 16 / 64 keys, copies against
  // gathers: 164 / 162 against 248 / 242 us (eight chunks, 145 GFLOP), the same to 128 rows: the
  // producer warps' instructions are what the softmax warps miss.
  for (a.kv.box_rows = 128; a.kv.box_rows >= 8 && a.kv.page_size % a.kv.box_rows != 0;) a.kv.box_rows /= 2;
  if (a.kv.box_rows < 8) a.kv.box_rows = 0;
  if (rc == ATTN_OK && a.kv.box_rows > 0) {
    rc = attn::encode_pool_map(&a.tm_k, a.kv.k, a.d, a.Hkv, a.kv.page_size, a.kv.num_pages, a.kv.box_rows);
    if (rc == ATTN_OK)
      rc = attn::encode_pool_map(&a.tm_v, a.kv.v, a.d, a.Hkv, a.kv.page_size, a.kv.num_pages, a.kv.box_rows);
  }
  if (rc != ATTN_OK) return rc;
  rc = from_cuda(a.o_bf16 ? attn::launch_prefill_paged(a, s) : attn::launch_prefill_paged_f32(a, s));
  if (rc != ATTN_OK || a.n_splits == 1) return rc;
  m.part_o = a.part_o; m.part_lse = a.part_lse; m.o = a.o; m.lse = a.lse;
  m.Hq = a.Hq; m.n_splits = a.n_splits; m.d = a.d; m.o_bf16 = a.o_bf16;
  return from_cuda(attn::launch_merge(m, s));
}

int rope_append_impl(const attn_bf16_t* q, const attn_bf16_t* k, const attn_bf16_t* v, long long q_stride,
                     long long k_stride, long long v_stride, const int* positions, const int* axes, int n_axes,
                     const double* inv_freq, attn_bf16_t* q_out, attn_bf16_t* kcache, attn_bf16_t* vcache, const int* page_table,
                     const int* cu_seqlens_q, const int* kv_lens, int B, int Hq, int Hkv, int total, int d,
                     int rot_dim, int interleaved, float amp, int max_pages, int page_size, int num_pages,
                     attn_stream_t stream) {
  int rc = check_heads(B, Hq, Hkv);
  if (rc != ATTN_OK) return rc;
  if (total < 0 || (cu_seqlens_q == nullptr && total != B) || !std::isfinite(amp)) return ATTN_ERR_INVALID_ARG;
  if (!ok_dim(d) || rot_dim < 0 || rot_dim > d || rot_dim % 16 != 0) return ATTN_ERR_UNSUPPORTED;
  rc = check_cache(page_table, B, max_pages, page_size, num_pages);
  if (rc != ATTN_OK) return rc;
  if (B == 0 || total == 0) return ATTN_OK;
  if (!ok16(k) || !ok16(v) || !ok16(kcache) || !ok16(vcache) || !ok4(kv_lens)) return ATTN_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr) || !aligned(q, 16) || !aligned(q_out, 16)) return ATTN_ERR_INVALID_ARG;
  if (axes && (n_axes < 1 || n_axes > attn::kMaxRopeAxes || !ok4(axes) || !positions)) return ATTN_ERR_INVALID_ARG;
  if (!aligned(positions, 4) || !aligned(cu_seqlens_q, 4)) return ATTN_ERR_INVALID_ARG;
  if (rot_dim > 0 && (inv_freq == nullptr || !aligned(inv_freq, 8))) return ATTN_ERR_INVALID_ARG;
  // rows of tokens: at least the heads' width, in whole 16-byte units
  if (k_stride < (long long)Hkv * d || v_stride < (long long)Hkv * d || k_stride % 8 || v_stride % 8)
    return ATTN_ERR_INVALID_ARG;
  if (q && (q_stride < (long long)Hq * d || q_stride % 8)) return ATTN_ERR_INVALID_ARG;
  // in place only over itself: a contiguous q
  if (q && q == q_out && q_stride != (long long)Hq * d) return ATTN_ERR_INVALID_ARG;
  if ((long long)(Hq + 2LL * Hkv) * (d / 16) > 0x7FFFFFFFLL) return ATTN_ERR_INVALID_ARG;
  attn::RopeArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = q; a.k = k; a.v = v;
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.positions = positions; a.axes = axes; a.n_axes = axes ? n_axes : 1; a.inv_freq = inv_freq; a.q_out = q_out;
  a.kc = kcache; a.vc = vcache;
  a.kv = cache(kcache, vcache, page_table, max_pages, page_size, num_pages);
  a.cu_q = cu_seqlens_q; a.kv_lens = kv_lens;
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.total = total; a.d = d; a.rot = rot_dim;
  a.interleaved = interleaved ? 1 : 0; a.amp = amp;
  a.err = attn::device_err_word();
  if (a.err == nullptr) return ATTN_ERR_CUDA;
  return from_cuda(attn::launch_rope_append(a, stream_of(stream)));
}

}  // namespace

extern "C" {

int attn_rope_append(const attn_bf16_t* q, const attn_bf16_t* k, const attn_bf16_t* v, long long q_stride,
                     long long k_stride, long long v_stride, const int* positions, const double* inv_freq,
                     attn_bf16_t* q_out, attn_bf16_t* kcache, attn_bf16_t* vcache, const int* page_table,
                     const int* cu_seqlens_q, const int* kv_lens, int B, int Hq, int Hkv, int total, int d,
                     int rot_dim, int interleaved, float amp, int max_pages, int page_size, int num_pages,
                     attn_stream_t stream) {
  return rope_append_impl(q, k, v, q_stride, k_stride, v_stride, positions, nullptr, 1, inv_freq, q_out, kcache, vcache,
                          page_table, cu_seqlens_q, kv_lens, B, Hq, Hkv, total, d, rot_dim, interleaved, amp,
                          max_pages, page_size, num_pages, stream);
}

int attn_rope_append_axes(const attn_bf16_t* q, const attn_bf16_t* k, const attn_bf16_t* v, long long q_stride,
                          long long k_stride, long long v_stride, const int* positions, const int* axes, int n_axes,
                          const double* inv_freq, attn_bf16_t* q_out, attn_bf16_t* kcache, attn_bf16_t* vcache,
                          const int* page_table, const int* cu_seqlens_q, const int* kv_lens, int B, int Hq, int Hkv,
                          int total, int d, int rot_dim, int interleaved, float amp, int max_pages, int page_size,
                          int num_pages, attn_stream_t stream) {
  if (n_axes < 1 || n_axes > attn::kMaxRopeAxes) return ATTN_ERR_INVALID_ARG;
  if (rot_dim == 0) return ATTN_ERR_UNSUPPORTED;  // (an append alone has no axes)
  if (B > 0 && total > 0 && (!ok4(axes) || !ok4(positions))) return ATTN_ERR_INVALID_ARG;
  return rope_append_impl(q, k, v, q_stride, k_stride, v_stride, positions, axes, n_axes, inv_freq, q_out, kcache,
                          vcache, page_table, cu_seqlens_q, kv_lens, B, Hq, Hkv, total, d, rot_dim, interleaved, amp,
                          max_pages, page_size, num_pages, stream);
}

int attn_rope_rotate(const attn_bf16_t* q, const attn_bf16_t* k, long long q_stride, long long k_stride,
                     const int* positions, const int* axes, int n_axes, const double* inv_freq, attn_bf16_t* q_out,
                     attn_bf16_t* k_out, long long q_out_stride, long long k_out_stride, int Hq, int Hk, int total,
                     int d, int rot_dim, int interleaved, int inverse, float amp, attn_stream_t stream) {
  if (Hq < 0 || Hk < 0 || Hq + (long long)Hk < 1 || total < 0 || !std::isfinite(amp)) return ATTN_ERR_INVALID_ARG;
  if (n_axes < 1 || n_axes > attn::kMaxRopeAxes || (axes == nullptr && n_axes != 1)) return ATTN_ERR_INVALID_ARG;
  if (d < 16 || d > 256 || d % 16 != 0 || rot_dim < 16 || rot_dim > d || rot_dim % 16 != 0) return ATTN_ERR_UNSUPPORTED;
  if (total == 0) return ATTN_OK;
  const struct {
    const attn_bf16_t *in, *out;
    long long stride, out_stride;
    int H;
  } sides[2] = {{q, q_out, q_stride, q_out_stride, Hq}, {k, k_out, k_stride, k_out_stride, Hk}};
  for (const auto& x : sides) {
    if (x.H == 0) continue;
    const long long w = (long long)x.H * d;
    if (!ok16(x.in) || !ok16(x.out) || x.stride < w || x.out_stride < w || x.stride % 8 || x.out_stride % 8)
      return ATTN_ERR_INVALID_ARG;
  }
  // outputs over inputs or one another would be turned twice, but for a side in place over itself
  ByteRows in[2], out[2];
  for (int i = 0; i < 2; ++i) {
    const auto& x = sides[i];
    in[i] = ByteRows{x.in, x.stride * 2, x.H * (long long)d * 2, total};
    out[i] = ByteRows{x.out, x.out_stride * 2, x.H * (long long)d * 2, total};
  }
  for (int i = 0; i < 2; ++i) {
    const bool same = sides[i].in == sides[i].out && sides[i].stride == sides[i].out_stride;
    if (!same && rows_overlap(out[i], in[i])) return ATTN_ERR_INVALID_ARG;
    if (rows_overlap(out[i], in[1 - i])) return ATTN_ERR_INVALID_ARG;
  }
  if (rows_overlap(out[0], out[1])) return ATTN_ERR_INVALID_ARG;
  if (!ok4(positions) || !aligned(axes, 4) || inv_freq == nullptr || !aligned(inv_freq, 8)) return ATTN_ERR_INVALID_ARG;
  // (eight tokens' chunks, and a CTA's threads beyond them, are counted in 32 bits)
  if ((Hq + (long long)Hk) * (d / 16) > (1LL << 27)) return ATTN_ERR_INVALID_ARG;
  attn::RotateArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = q; a.k = k; a.q_out = q_out; a.k_out = k_out;
  a.q_stride = q_stride; a.k_stride = k_stride; a.qo_stride = q_out_stride; a.ko_stride = k_out_stride;
  a.positions = positions; a.axes = axes; a.n_axes = n_axes; a.inv_freq = inv_freq;
  a.Hq = Hq; a.Hk = Hk; a.total = total; a.d = d; a.rot = rot_dim;
  a.interleaved = interleaved ? 1 : 0; a.inverse = inverse ? 1 : 0; a.amp = amp;
  a.err = attn::device_err_word();
  if (a.err == nullptr) return ATTN_ERR_CUDA;
  return from_cuda(attn::launch_rope_rotate(a, stream_of(stream)));
}

int attn_prefill_paged_splits(int B, int Hq, int Hkv, int total_q, int max_sq, int max_kv, int d, int* min_rows) {
  if (check_heads(B, Hq, Hkv) != ATTN_OK || total_q < 0 || max_sq < 0 || max_kv < 0 || !ok_dim(d) ||
      min_rows == nullptr)
    return ATTN_ERR_INVALID_ARG;
  return prefill_splits(B, Hq, total_q, max_sq, max_kv, d, pack_heads(Hq / Hkv, attn::kPrefillTileM), min_rows);
}

int attn_prefill_paged(const attn_bf16_t* q, const attn_bf16_t* kcache, const attn_bf16_t* vcache, void* o, float* lse,
                       const int* page_table, const int* cu_seqlens_q, const int* kv_lens, int B, int Hq, int Hkv,
                       int total_q, int max_sq, int max_pages, int page_size, int num_pages, int d, int causal,
                       int window, int n_sink, float scale, int n_splits, int min_rows_per_split, float* part_o,
                       float* part_lse, int o_dtype, attn_stream_t stream) {
  int rc = check_heads(B, Hq, Hkv);
  if (rc != ATTN_OK) return rc;
  if (total_q < 0 || max_sq < 0 || window < 0 || n_sink < 0 || !ok_scale(scale)) return ATTN_ERR_INVALID_ARG;
  if (n_splits < 1 || n_splits > 1024 || min_rows_per_split < 0) return ATTN_ERR_INVALID_ARG;
  if (window > 0 && !causal) return ATTN_ERR_INVALID_ARG;
  if (!ok_dim(d) || (o_dtype != ATTN_F32 && o_dtype != ATTN_BF16)) return ATTN_ERR_UNSUPPORTED;
  if (window > 0 && n_splits > 1) return ATTN_ERR_UNSUPPORTED;
  rc = check_cache(page_table, B, max_pages, page_size, num_pages);
  if (rc == ATTN_OK) rc = check_slot(Hkv, d);
  if (rc != ATTN_OK) return rc;
  if (B == 0 || total_q == 0 || max_sq == 0) return ATTN_OK;
  if (!ok16(q) || !ok16(kcache) || !ok16(vcache) || !ok16(o) || !ok16(lse) || !ok4(cu_seqlens_q) || !ok4(kv_lens) ||
      !ok4(page_table))
    return ATTN_ERR_INVALID_ARG;
  if (n_splits > 1 && (!ok16(part_o) || !ok4(part_lse))) return ATTN_ERR_INVALID_ARG;
  if ((long long)total_q * Hq >= (1LL << 31) || (long long)max_sq * (Hq / Hkv) >= (1LL << 30))
    return ATTN_ERR_INVALID_ARG;
  attn::PrefillArgs a;
  std::memset(&a, 0, sizeof(a));
  a.o = o;
  a.lse = lse;
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.Sq = max_sq; a.Skv = max_pages * page_size; a.d = d;
  a.causal = causal ? 1 : 0;
  a.o_bf16 = o_dtype == ATTN_BF16 ? 1 : 0;
  a.scale = scale;
  a.window = window;
  a.n_sink = n_sink;
  a.cu_q = cu_seqlens_q;
  a.kv_lens = kv_lens;
  a.total_q = total_q;
  a.pack = pack_heads(Hq / Hkv, attn::kPrefillTileM);
  a.n_splits = n_splits;
  a.split_min = std::min(min_rows_per_split, max_pages * page_size);  // (rounded up to a tile there)
  a.part_o = part_o;
  a.part_lse = part_lse;
  // every sequence's rows fit one tile: the other tile takes half of the keys
  a.halves = (window == 0 && d <= 128 && max_sq <= attn::kPrefillTileM / a.pack) ? 1 : 0;
  a.kv = cache(kcache, vcache, page_table, max_pages, page_size, num_pages);
  attn::MergeArgs m;
  m.B = total_q;
  m.lse_by_head = 1;
  m.cu_q = cu_seqlens_q;
  m.n_seq = B;
  return launch_paged(a, q, total_q, 1, m, stream_of(stream));
}

int attn_decode_paged_splits(int B, int Hq, int Hkv, int max_kv, int d, int o_dtype, int* min_rows) {
  if (check_heads(B, Hq, Hkv) != ATTN_OK || max_kv < 0 || !ok_dim(d) || min_rows == nullptr ||
      (o_dtype != ATTN_BF16 && o_dtype != ATTN_F32))
    return ATTN_ERR_INVALID_ARG;
  if (decode_on_tiles(B, Hq, Hkv, o_dtype))
    return prefill_splits(B, Hq, B, 1, max_kv, d, std::min(Hq / Hkv, attn::kPrefillTileM), min_rows);
  return mma_splits(std::max(1.0, (double)B * Hkv), Hq / Hkv, B, max_kv, d, min_rows);
}

int attn_decode_paged(const attn_bf16_t* q, const attn_bf16_t* kcache, const attn_bf16_t* vcache,
                      const int* page_table, const int* kv_lens, int B, int Hq, int Hkv, int d, int max_pages,
                      int page_size, int num_pages, float scale, int n_splits, int min_rows_per_split, float* part_o,
                      float* part_lse, void* o, float* lse, int o_dtype, unsigned int* counters,
                      attn_stream_t stream) {
  int rc = check_heads(B, Hq, Hkv);
  if (rc == ATTN_OK) rc = check_cache(page_table, B, max_pages, page_size, num_pages);
  if (rc == ATTN_OK && ok_dim(d)) rc = check_slot(Hkv, d);
  if (rc == ATTN_OK)
    // (the dense cache's row limit does not apply: max_kv = 1 here)
    rc = attn::check_decode_split_args(q, kcache, vcache, kv_lens, B, Hq, Hkv, d, 1, scale, n_splits,
                                       min_rows_per_split, part_o, part_lse, n_splits > 1);
  if (rc == ATTN_OK)
    rc = attn::check_merge_args(part_o, part_lse, o, lse, B, Hq, n_splits, d, o_dtype, n_splits > 1);
  if (rc != ATTN_OK || B == 0) return rc;
  if (!ok4(page_table) || (n_splits > 1 && !ok4(counters))) return ATTN_ERR_INVALID_ARG;
  if (decode_on_tiles(B, Hq, Hkv, o_dtype)) {
    // a group's heads as the rows of one tensor-core tile: its keys are read once
    attn::PrefillArgs p;
    std::memset(&p, 0, sizeof(p));
    p.o = o; p.lse = lse;
    p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.Sq = 1; p.Skv = max_pages * page_size; p.d = d;
    p.causal = 1;
    p.o_bf16 = o_dtype == ATTN_BF16 ? 1 : 0;
    p.scale = scale;
    p.kv_lens = kv_lens;
    p.pack = Hq / Hkv;
    p.n_splits = n_splits; p.split_min = std::min(min_rows_per_split, max_pages * page_size);
    p.part_o = part_o; p.part_lse = part_lse;
    p.halves = d <= 128 ? 1 : 0;
    p.kv = cache(kcache, vcache, page_table, max_pages, page_size, num_pages);
    attn::MergeArgs m;
    m.B = B;
    m.lse_by_head = 0;
    m.cu_q = nullptr;
    m.n_seq = 0;
    return launch_paged(p, q, 1, B, m, stream_of(stream));
  }
  attn::DecodeArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = q; a.kv_lens = kv_lens; a.part_o = part_o; a.part_lse = part_lse;
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.d = d; a.max_kv = max_pages * page_size;
  a.n_splits = n_splits; a.min_rows = min_rows_per_split; a.scale = scale;
  a.done = counters; a.o = o; a.lse = lse; a.o_bf16 = o_dtype == ATTN_BF16 ? 1 : 0;
  a.kv = cache(kcache, vcache, page_table, max_pages, page_size, num_pages);
  a.err = attn::device_err_word();
  if (a.err == nullptr) return ATTN_ERR_CUDA;
  return from_cuda(attn::launch_decode_paged(a, stream_of(stream)));
}

int attn_decode_window_splits(int B, int Hq, int Hkv, int max_kv, int window, int n_sink, int d, int* min_rows) {
  if (check_heads(B, Hq, Hkv) != ATTN_OK || max_kv < 0 || window < 1 || n_sink < 0 || !ok_dim(d) ||
      min_rows == nullptr)
    return ATTN_ERR_INVALID_ARG;
  const int keys = (int)std::min<long long>(max_kv, (long long)window + n_sink);
  const int G = Hq / Hkv, ctas = window_head_ctas(G);
  return window_splits(std::max(1.0, (double)B * Hkv * ctas), (G + ctas - 1) / ctas, keys, d, min_rows);
}

int attn_decode_window(const attn_bf16_t* q, const attn_bf16_t* kcache, const attn_bf16_t* vcache,
                       const int* page_table, const int* kv_lens, int B, int Hq, int Hkv, int d, int max_pages,
                       int page_size, int num_pages, int window, int n_sink, float scale, int n_splits,
                       int min_rows_per_split, float* part_o, float* part_lse, void* o, float* lse, int o_dtype,
                       unsigned int* counters, attn_stream_t stream) {
  int rc = check_heads(B, Hq, Hkv);
  if (rc == ATTN_OK && (window < 1 || n_sink < 0)) rc = ATTN_ERR_INVALID_ARG;
  if (rc == ATTN_OK) rc = check_cache(page_table, B, max_pages, page_size, num_pages);
  if (rc == ATTN_OK && ok_dim(d)) rc = check_slot(Hkv, d);
  if (rc == ATTN_OK)
    // (the dense cache's row limit does not apply: max_kv = 1 here)
    rc = attn::check_decode_split_args(q, kcache, vcache, kv_lens, B, Hq, Hkv, d, 1, scale, n_splits,
                                       min_rows_per_split, part_o, part_lse, n_splits > 1);
  if (rc == ATTN_OK)
    rc = attn::check_merge_args(part_o, part_lse, o, lse, B, Hq, n_splits, d, o_dtype, n_splits > 1);
  if (rc != ATTN_OK || B == 0) return rc;
  if (n_splits > 1 && !ok4(counters)) return ATTN_ERR_INVALID_ARG;
  attn::DecodeArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = q; a.kv_lens = kv_lens; a.part_o = part_o; a.part_lse = part_lse;
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.d = d; a.max_kv = max_pages * page_size;
  a.n_splits = n_splits; a.min_rows = min_rows_per_split; a.scale = scale;
  a.done = counters; a.o = o; a.lse = lse; a.o_bf16 = o_dtype == ATTN_BF16 ? 1 : 0;
  a.kv = cache(kcache, vcache, page_table, max_pages, page_size, num_pages);
  a.window = window; a.n_sink = n_sink;
  a.head_ctas = window_head_ctas(Hq / Hkv);
  a.cta_heads = (Hq / Hkv + a.head_ctas - 1) / a.head_ctas;
  a.err = attn::device_err_word();
  if (a.err == nullptr) return ATTN_ERR_CUDA;
  return from_cuda(attn::launch_decode_window(a, stream_of(stream)));
}

int attn_key_weights(const attn_bf16_t* q, const float* lse, const attn_bf16_t* kcache, const int* page_table,
                     const int* cu_seqlens_q, const int* kv_lens, float* weights, long long w_stride, int B, int Hq,
                     int Hkv, int total_q, int max_sq, int d, int max_pages, int page_size, int num_pages, int causal,
                     int window, int n_sink, float scale, int accumulate, attn_stream_t stream) {
  int rc = check_heads(B, Hq, Hkv);
  if (rc != ATTN_OK) return rc;
  if (total_q < 0 || max_sq < 0 || window < 0 || n_sink < 0 || !ok_scale(scale)) return ATTN_ERR_INVALID_ARG;
  if (window > 0 && !causal) return ATTN_ERR_INVALID_ARG;
  if (cu_seqlens_q == nullptr && (total_q != B || max_sq != 1)) return ATTN_ERR_INVALID_ARG;
  if (!ok_dim(d) || scale < 1e-30f || scale > 1e30f) return ATTN_ERR_UNSUPPORTED;  // (lse / scale is formed)
  rc = check_cache(page_table, B, max_pages, page_size, num_pages);
  if (rc == ATTN_OK) rc = check_slot(Hkv, d);
  if (rc != ATTN_OK) return rc;
  if (w_stride < (long long)max_pages * page_size) return ATTN_ERR_INVALID_ARG;
  if (B == 0) return ATTN_OK;
  if (!ok16(kcache) || !ok4(kv_lens) || !ok4(weights) || !aligned(cu_seqlens_q, 4)) return ATTN_ERR_INVALID_ARG;
  if (total_q == 0) max_sq = 0;  // no rows: the sums are zero (or stay, if accumulated)
  else if (!ok16(q) || !ok4(lse)) return ATTN_ERR_INVALID_ARG;
  if ((long long)total_q * Hq >= (1LL << 31) || (long long)max_sq * (Hq / Hkv) >= (1LL << 30) ||
      (long long)B * Hkv > 0x7FFFFFFFLL)
    return ATTN_ERR_INVALID_ARG;
  attn::KeyWeightArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = q; a.lse = lse;
  a.lse_hs = cu_seqlens_q ? total_q : 1;  // [Hq][total_q], or the decode's [B][Hq]
  a.lse_ts = cu_seqlens_q ? 1 : Hq;
  a.kv = cache(kcache, nullptr, page_table, max_pages, page_size, num_pages);
  a.cu_q = cu_seqlens_q; a.kv_lens = kv_lens;
  a.weights = weights; a.w_stride = w_stride;
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.total_q = total_q; a.max_sq = max_sq; a.d = d;
  a.causal = causal ? 1 : 0; a.window = window; a.n_sink = n_sink; a.accumulate = accumulate ? 1 : 0;
  a.scale = scale;
  a.err = attn::device_err_word();
  if (a.err == nullptr) return ATTN_ERR_CUDA;
  if (!attn::key_weights_few_rows(max_sq, Hq / Hkv)) {
    const int rows = attn::key_weights_q_rows(d);
    a.pack = pack_heads(Hq / Hkv, rows);
    rc = attn::encode_q_map(&a.tm_q, q, d, a.pack, Hq, total_q, 1, rows);
    if (rc != ATTN_OK) return rc;
  }
  return from_cuda(attn::launch_key_weights(a, stream_of(stream)));
}

int attn_evict(const float* weights, float* weights_out, long long w_stride, attn_bf16_t* kcache, attn_bf16_t* vcache,
               const int* page_table, const int* kv_lens, int B, int Hkv, int d, int max_pages, int page_size,
               int num_pages, int budget, int n_recent, int n_sink, attn_bf16_t* k_dst, attn_bf16_t* v_dst,
               const int* dst_table, int dst_max_pages, int dst_page_size, int dst_num_pages, int* kept, int* new_lens,
               attn_stream_t stream) {
  int rc = check_heads(B, Hkv, Hkv);
  if (rc != ATTN_OK) return rc;
  if (budget < 1 || n_recent < 0 || n_sink < 0 || (long long)n_recent + n_sink > budget) return ATTN_ERR_INVALID_ARG;
  if (!ok_dim(d)) return ATTN_ERR_UNSUPPORTED;
  rc = check_cache(page_table, B, max_pages, page_size, num_pages);
  if (rc != ATTN_OK) return rc;
  const long long cap = (long long)max_pages * page_size;
  if (w_stride < cap) return ATTN_ERR_INVALID_ARG;
  const bool in_place = k_dst == nullptr;
  if (in_place != (v_dst == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (!in_place) {
    rc = check_cache(dst_table, B, dst_max_pages, dst_page_size, dst_num_pages);
    if (rc != ATTN_OK) return rc;
    if ((long long)dst_max_pages * dst_page_size < (budget < cap ? budget : cap)) return ATTN_ERR_INVALID_ARG;
    // a destination that is the source itself is the in-place form, called as such
    if (k_dst == kcache && v_dst == vcache && dst_table == page_table) return ATTN_ERR_INVALID_ARG;
  }
  if ((long long)B * Hkv > 0x7FFFFFFFLL) return ATTN_ERR_INVALID_ARG;
  if (B == 0) return ATTN_OK;
  if (!ok4(weights) || !aligned(weights_out, 4) || !ok16(kcache) || !ok16(vcache) || !ok4(kv_lens) || !ok4(kept) ||
      !ok4(new_lens) || !aligned(k_dst, 16) || !aligned(v_dst, 16))
    return ATTN_ERR_INVALID_ARG;
  attn::EvictArgs a;
  std::memset(&a, 0, sizeof(a));
  a.weights = weights; a.weights_out = weights_out; a.w_stride = w_stride;
  a.src = cache(kcache, vcache, page_table, max_pages, page_size, num_pages);
  a.in_place = in_place ? 1 : 0;
  if (in_place) {
    a.dst = a.src;
    a.dk = kcache; a.dv = vcache;
  } else {
    a.dst = cache(k_dst, v_dst, dst_table, dst_max_pages, dst_page_size, dst_num_pages);
    a.dk = k_dst; a.dv = v_dst;
  }
  a.kv_lens = kv_lens; a.new_lens = new_lens; a.kept = kept;
  a.B = B; a.Hkv = Hkv; a.d = d; a.budget = budget; a.n_recent = n_recent; a.n_sink = n_sink;
  a.err = attn::device_err_word();
  if (a.err == nullptr) return ATTN_ERR_CUDA;
  return from_cuda(attn::launch_evict(a, stream_of(stream)));
}

}  // extern "C"
