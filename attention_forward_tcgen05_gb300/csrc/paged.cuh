// paged.cuh -- rows of a paged K/V cache: the page-table lookup and the 16-byte
// asynchronous copies that gather them into shared memory.
//
// A cache is a pool of pages, k / v [num_pages][page_size][Hkv][d]; key j of
// sequence b lies in slot j % page_size of page table[b][j / page_size].  One cp.async of a
// warp moves 512 bytes of 32 / (d / 8) rows, from any page size and any first row, and a row
// that does not exist arrives as zeros without being read; the decode and the key weights,
// which HBM bounds, gather every row so, each warp for itself.  The prefill, whose softmax
// warps want the issue slots, copies pages of 8 rows and more by TMA (paged_api.cu) and
// gathers only a sequence's last tile and other pages.
#pragma once
#include "internal.h"
#include "ptx.cuh"

namespace attn {

// Pool row (page * page_size + slot) of key j, or -1 if the table's entry is not a
// page of the pool (recorded in the error word; such a row reads as zeros).  A dense
// cache [B][page_size] (table == nullptr) is one page per sequence.
__device__ __forceinline__ int paged_row(const PagedKV& kv, int b, int j, uint32_t* err) {
  if (kv.table == nullptr) return b * kv.page_size + j;
  const int e = (int)((unsigned)j / (unsigned)kv.page_size);
  const int page = __ldg(kv.table + (size_t)b * kv.max_pages + e);
  if ((unsigned)page >= (unsigned)kv.num_pages) {
    atomicCAS(err, kErrNone, kErrBadShape);
    return -1;
  }
  return page * kv.page_size + (j - e * kv.page_size);
}

// 16 bytes global -> shared, past L1; bytes = 0 writes zeros and reads nothing
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The pool rows of 32 * NR consecutive keys from j0, as lane registers: lane's ri[h]
// is the row of key j0 + 32 h + lane, -1 at or past `end`.
template <int NR>
__device__ __forceinline__ void paged_rows(const PagedKV& kv, int b, int j0, int end, int lane, uint32_t* err,
                                           int (&ri)[NR]) {
#pragma unroll
  for (int h = 0; h < NR; ++h) {
    const int j = j0 + 32 * h + lane;
    ri[h] = j < end ? paged_row(kv, b, j, err) : -1;
  }
}

// The whole warp gathers ROWS rows (D bf16 of KV head hk each; the rows of lanes from
// `first` on in ri) into a tile of D / 64 panels of 128-byte swizzled rows, `panel_bytes`
// apart (the layout a 128B-swizzled tensor copy gives; `dst` on a 1024-byte boundary).
template <int D, int ROWS>
__device__ __forceinline__ void paged_gather_rows(uint32_t dst, int panel_bytes, const uint16_t* pool, int Hkv, int hk,
                                                  int lane, int ri, int first) {
  constexpr int CPR = D / 8;     // 16-byte chunks of a row
  constexpr int RPI = 32 / CPR;  // rows of one warp copy
  const int c = lane % CPR, rsub = lane / CPR;
  const uint32_t lane_dst = dst + (c >> 3) * panel_bytes + rsub * 128;
  const int cx = (c & 7) ^ rsub;  // rsub < RPI <= 4 and rows step by RPI: the XORs below do not meet
  const uint8_t* base = reinterpret_cast<const uint8_t*>(pool + (size_t)hk * D + c * 8);
  const uint32_t row_bytes = (uint32_t)Hkv * D * 2u;
#pragma unroll 8
  for (int i = 0; i < ROWS / RPI; ++i) {
    const int r = __shfl_sync(0xFFFFFFFFu, ri, first + i * RPI + rsub);
    const uint8_t* src = base + (uint64_t)(uint32_t)max(r, 0) * row_bytes;
    cp_async16(lane_dst + i * RPI * 128 + ((cx ^ ((i * RPI) & 7)) << 4), src, r < 0 ? 0u : 16u);
  }
}
template <int D, int NR>
__device__ __forceinline__ void paged_gather(uint32_t dst, int panel_bytes, const uint16_t* pool, int Hkv, int hk,
                                             int lane, const int (&ri)[NR]) {
#pragma unroll
  for (int h = 0; h < NR; ++h)
    paged_gather_rows<D, 32>(dst + h * 32 * 128, panel_bytes, pool, Hkv, hk, lane, ri[h], 0);
}

}  // namespace attn
