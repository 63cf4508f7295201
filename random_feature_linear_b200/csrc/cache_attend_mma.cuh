// Interface between the cache attention's launches and its tensor-core kernels.
#pragma once

#include "cache_attend.cuh"
#include "tc_common.cuh"

namespace dark {
namespace cache {

// Rows that one CTA of the tensor-core range kernel takes at once. Over 1024 own keys of 64
// sequences, 4 key heads, d = 64: 12 rows take 28.2 us in blocks of 16 and 34.0 of 8, 32 rows 46.0
// and 51.0 (d = 128: 12 rows 51.5 and 71.3, 20 rows 84.7 and 84.1, 64 rows 118.5 and 165.9).
inline int mma_rows(int dp, int rows) { return dp <= 128 && rows > 8 ? 16 : 8; }
cudaError_t launch_ranges_mma(const Params& q);

// The prefix's ranges for more rows, which share the keys in a CTA: 32 rows as hi + lo, or 64.
inline int share_rows(int dp, int all) { return dp <= 128 && all > 32 ? 64 : 32; }
cudaError_t launch_prefix_mma(const Params& q);

// Rows of a block of the tcgen05 kernel (dp <= 128), keys of its tiles.
constexpr int kTcRows = 256, kTcKeys = 128;
cudaError_t launch_prefix_tc(const Params& q);

// The queries y = M^T M q on the tensor cores, and the cut of the own keys.
cudaError_t launch_queries_mma(const Params& q);

// ---- copies, fragments and products of the mma.sync kernels

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma16816_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte chunk `c` of row `row` in a tile of DP bf16 columns: chunks
// XORed with the row's low bits, so that eight rows at one chunk hit eight bank groups.
template <int DP>
__device__ __forceinline__ uint32_t tile_off(int row, int c) {
  return (uint32_t)(row * DP * 2 + ((c ^ (row & 7)) << 4));
}

// Queries for the tensor cores: y = hi + lo in bf16 (16 bits of significand together;
// one bf16 alone would move the exponents by up to 2^-8 relative, as much again as the rounding
// of the output). hi rows first, then all lo rows, dp columns each.
__device__ __forceinline__ void store_query_hi_lo(__nv_bfloat16* y, int64_t nrows, int64_t row,
                                                  int dp, int c, float v) {
  const __nv_bfloat16 hi = __float2bfloat16_rn(v);
  y[row * dp + c] = hi;
  y[(nrows + row) * dp + c] = __float2bfloat16_rn(v - __bfloat162float(hi));
}

}  // namespace cache
}  // namespace dark
