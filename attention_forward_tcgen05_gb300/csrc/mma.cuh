// mma.cuh -- warp-level matrix fragments (ldmatrix, mma.sync m16n8k16) for the kernels that
// stream keys from HBM with a few query rows per key.  There the tensor work per byte is
// far below what a tcgen05 tile would cost to set up, drain and read back from TMEM, and a
// warp that keeps its scores in registers needs no other warp.
#pragma once
#include <cstdint>

namespace attn {

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// c[16 x 8] += a[16 x 16] b[16 x 8], bf16 in, fp32 accumulators
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// transpose of an 8 x 8 matrix of 16-bit elements held as a fragment
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Lane addresses of the A fragments of 16 keys held as 128-byte swizzled rows (16 rows a
// panel of 64 columns, kPanel bytes apart): key r, 16-byte chunk c at
//   (c / 8) * kPanel + r * 128 + ((c % 8) ^ (r % 8)) * 16.
// keys x dims (S^T = K Q^T): k-step kk covers chunks 2 kk, 2 kk + 1.
template <int kPanel>
__device__ __forceinline__ uint32_t frag_keys(uint32_t tile, int kk, int lane) {
  const int r = lane & 15, c = 2 * kk + (lane >> 4);
  return tile + (c >> 3) * kPanel + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}
// dims x keys (O^T = V^T P^T, transposed load): m-tile mt covers chunks 2 mt, 2 mt + 1.
template <int kPanel>
__device__ __forceinline__ uint32_t frag_dims(uint32_t tile, int mt, int lane) {
  const int r = (lane & 7) + ((lane >> 4) << 3), c = 2 * mt + ((lane >> 3) & 1);
  return tile + (c >> 3) * kPanel + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// B fragments of a query block: rows n = lane / 4 (row0 + n, zero at or past `rows`), dims
// 16 kk + 2 (lane % 4) + {0, 1} and + 8.  `q` points to row 0's head dim; rows are
// `stride` elements apart through the index function.
template <int D, class RowPtr>
__device__ __forceinline__ void load_q_frags(uint32_t (&f)[D / 16][2], RowPtr row_ptr, int row, bool live, int lane) {
  const uint16_t* p = live ? row_ptr(row) : nullptr;
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    f[kk][0] = live ? *reinterpret_cast<const uint32_t*>(p + kk * 16 + (lane & 3) * 2) : 0u;
    f[kk][1] = live ? *reinterpret_cast<const uint32_t*>(p + kk * 16 + 8 + (lane & 3) * 2) : 0u;
  }
}

}  // namespace attn
