// Interface between the cache attention's launches and its tensor-core kernels.
#pragma once

#include "cache_attend.cuh"

namespace dark {
namespace cache {

// Rows that one CTA of the tensor-core range kernel takes at once.
inline int mma_rows(int dp, int rows) { return dp <= 128 && rows > 8 ? 16 : 8; }
cudaError_t launch_ranges_mma(const Params& q);

// Rows of a tile block of the tcgen05 kernel, keys of its tiles.
inline int tc_rows(int dp) { return dp == 256 ? 128 : 256; }
constexpr int kTcKeys = 128;
cudaError_t launch_prefix_tc(const Params& q);

// Queries for the tensor cores: y = hi + lo in bf16 (16 bits of significand together;
// one bf16 alone would move the exponents by 2^-9 relative, as much again as the rounding
// of the output). hi rows first, then all lo rows, dp columns each.
__device__ __forceinline__ void store_query_hi_lo(__nv_bfloat16* y, int64_t nrows, int64_t row,
                                                  int dp, int c, float v) {
  const __nv_bfloat16 hi = __float2bfloat16_rn(v);
  y[row * dp + c] = hi;
  y[(nrows + row) * dp + c] = __float2bfloat16_rn(v - __bfloat162float(hi));
}

}  // namespace cache
}  // namespace dark
