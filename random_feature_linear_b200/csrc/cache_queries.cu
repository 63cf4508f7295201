// Cache attention, first launch (bf16): the queries after the geometry,
// y = 2 (c_m M)^T (c_m M) q, on the tensor cores, and the cut of the own keys.
//
// 16 rows of one query head a CTA; a warp takes 16 rows i of c_m M at a time, its scores
// p_i = (c_m M)_i q are the first operand of the second product as they come out of the
// first (the layout of accumulators and operands agree), and the warps' sums of y are
// joined at the end. q is exact in fp16 above 2^-17 and below 65504 (larger values give
// non-finite outputs, which the join reports), c_m M is fp16 as stored, and p goes as hi + lo
// in fp16, scaled by a power of two for each query, so that its largest |p_i| lies between 2^10
// and 2^15 (the power follows a p_i past that): p may have any size, and y keeps 22 bits of every
// p_i above 2^-13 of the largest (2^-35 of the largest below). For prefixes on tcgen05 y is
// stored in fp16 as well (past 65504: reported).
//
// Bound by latency: one read of M's rows (r d 2 bytes, shared by the CTAs of a head in L2).
#include "cache_attend_mma.cuh"
#include "cache_sched.cuh"

namespace dark {
namespace cache {
namespace {

constexpr int kRows = 16;

template <int DP>
struct Cfg {
  static constexpr uint32_t kTile = 16 * DP * 2;       // 16 rows of DP fp16 columns
};

template <int DP, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) queries_mma_kernel(const __grid_constant__ Params q) {
  constexpr uint32_t kTile = Cfg<DP>::kTile;
  constexpr int NS = DP / 16, NT = DP / 8, CH = DP / 8;
  pdl_launch();
  if (blockIdx.x == gridDim.x - 1) {
    if (blockIdx.y == 0) make_sched(q);
    return;
  }
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t s0 = tc::smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int d = q.a.d, r = q.a.r, h = blockIdx.y, n0 = blockIdx.x * kRows, n = q.a.B * q.a.T;
  const __half* w = (const __half*)q.a.w + ((int64_t)(q.a.heads_w == 1 ? 0 : h) * (q.a.m + r) + q.a.m) * d;
  // queries: the first tile of shared memory; then two tiles of M a warp
  const uint32_t ring = s0 + kTile + warp * 2 * kTile;
  const int tiles = (r + 15) / 16, mine = tiles > warp ? (tiles - warp + WARPS - 1) / WARPS : 0;
  auto issue = [&](int i) {
    const int i0 = (warp + i * WARPS) * 16;
    if (i < mine) {
#pragma unroll
      for (int k = 0; k < 16 * CH / 32; ++k) {
        const int idx = k * 32 + lane, row = idx / CH, c = idx % CH;
        const bool ok = i0 + row < r && c * 8 < d;
        cp16(ring + (i & 1) * kTile + tile_off<DP>(row, c), w + (ok ? (int64_t)(i0 + row) * d + c * 8 : 0), ok);
      }
    }
    cp_commit();
  };
  issue(0);
  issue(1);
  for (int idx = tid; idx < kRows * CH; idx += WARPS * 32) {
    const int row = idx / CH, c = idx % CH, k = n0 + row;
    uint32_t v[4] = {0u, 0u, 0u, 0u};
    if (k < n && c * 8 < d) {
      const int b = k / q.a.T, tt = k - b * q.a.T;
      const __nv_bfloat16* src = (const __nv_bfloat16*)q.a.q + b * q.a.qs[0] + h * q.a.qs[1] + tt * q.a.qs[2] + c * 8;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __half2 x = __floats2half2_rn(__bfloat162float(src[2 * e]), __bfloat162float(src[2 * e + 1]));
        v[e] = *reinterpret_cast<const uint32_t*>(&x);
      }
    }
    tc::st_shared_v4(s0 + tile_off<DP>(row, c), v[0], v[1], v[2], v[3]);
  }
  __syncthreads();
  const int lr = lane & 7, lg = lane >> 3;
  uint32_t a[NS][4];
#pragma unroll
  for (int s = 0; s < NS; ++s) ldsm4(a[s], s0 + tile_off<DP>((lg & 1) * 8 + lr, 2 * s + (lg >> 1)));
  float o[NT][4];
#pragma unroll
  for (int k = 0; k < NT; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[k][e] = 0.f;
  // exponent fields of |2 p_i| (rows g, g + 8) that the scale puts at 2^10; o is y 2^(137 - ex)
  int ex[2] = {15, 15};
  for (int i = 0; i < mine; ++i) {
    cp_wait<1>();
    __syncwarp();
    const uint32_t m0 = ring + (i & 1) * kTile;
    float p[2][4] = {};
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      uint32_t b[4];
      ldsm4(b, m0 + tile_off<DP>((lg >> 1) * 8 + lr, 2 * s + (lg & 1)));
      mma16816_f16(p[0], a[s], b[0], b[1]);
      mma16816_f16(p[1], a[s], b[2], b[3]);
    }
    int top[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float m = fmaxf(fmaxf(fabsf(p[0][2 * e]), fabsf(p[0][2 * e + 1])),
                            fmaxf(fabsf(p[1][2 * e]), fabsf(p[1][2 * e + 1])));
      top[e] = __float_as_int(2.f * m) >> 23;
      top[e] = max(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
      top[e] = max(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
    }
    if (i == 0) {
      ex[0] = max(ex[0], top[0]);
      ex[1] = max(ex[1], top[1]);
    } else if (__any_sync(0xffffffffu, top[0] > ex[0] + 4 || top[1] > ex[1] + 4)) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int now = top[e] > ex[e] + 4 ? top[e] : ex[e], field = 127 + ex[e] - now;
        const float f = __int_as_float(field > 0 ? field << 23 : 0);       // (2^-127 and less: 0)
        ex[e] = now;
#pragma unroll
        for (int k = 0; k < NT; ++k) {
          o[k][2 * e] *= f;
          o[k][2 * e + 1] *= f;
        }
      }
    }
    uint32_t hi[4], lo[4];                             // rows g, g + 8 by columns 2 t, 2 t + 8
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float s = __int_as_float((265 - ex[e & 1]) << 23);             // 2 * 2^(137 - ex)
      const float x = s * p[e >> 1][(e & 1) * 2], y = s * p[e >> 1][(e & 1) * 2 + 1];
      const __half2 hh = __floats2half2_rn(x, y);
      const __half2 ll = __floats2half2_rn(x - __low2float(hh), y - __high2float(hh));
      hi[e] = *reinterpret_cast<const uint32_t*>(&hh);
      lo[e] = *reinterpret_cast<const uint32_t*>(&ll);
    }
#pragma unroll
    for (int k = 0; k < NT; k += 2) {
      uint32_t b[4];
      ldsm4_t(b, m0 + tile_off<DP>((lg & 1) * 8 + lr, k + (lg >> 1)));
      mma16816_f16(o[k], hi, b[0], b[1]);
      mma16816_f16(o[k], lo, b[0], b[1]);
      mma16816_f16(o[k + 1], hi, b[2], b[3]);
      mma16816_f16(o[k + 1], lo, b[2], b[3]);
    }
    __syncwarp();
    issue(i + 2);
  }
  cp_wait<0>();
  __syncthreads();
  // the warps' sums, in order of the warps; rows 8 words apart from a multiple of the 32 banks
  constexpr int LD = DP + 8;
  float* sum = reinterpret_cast<float*>(smem);         // [warp][16][LD]
  const float back[2] = {__int_as_float((ex[0] - 10) << 23), __int_as_float((ex[1] - 10) << 23)};
#pragma unroll
  for (int k = 0; k < NT; ++k) {
    float* to = sum + (warp * 16 + g) * LD + 8 * k + 2 * t;
    *reinterpret_cast<float2*>(to) = make_float2(o[k][0] * back[0], o[k][1] * back[0]);
    *reinterpret_cast<float2*>(to + 8 * LD) = make_float2(o[k][2] * back[1], o[k][3] * back[1]);
  }
  __syncthreads();
  const int gg = h % q.G, hk = h / q.G;
  const int64_t rows = (int64_t)q.a.Hk * q.p.all;
  bool over = false;
  for (int idx = tid; idx < kRows * DP; idx += WARPS * 32) {
    const int row = idx / DP, c = idx - row * DP, k = n0 + row;
    if (k >= n) break;
    float v = 0.f;
#pragma unroll
    for (int x = 0; x < WARPS; ++x) v += sum[(x * 16 + row) * LD + c];
    const int b = k / q.a.T, tt = k - b * q.a.T;
    const int64_t to = (int64_t)hk * q.p.all + (b * q.G + gg) * q.a.T + tt;
    store_query_hi_lo(at<__nv_bfloat16>(q.a, q.p.o_y), rows, to, DP, c, v);
    if (q.p.tc) {
      const __half y = __float2half_rn(v);
      at<__half>(q.a, q.p.o_y16)[to * DP + c] = y;
      if (__hisinf(y)) {                                // (padding may hold anything)
        const int64_t last = min((int64_t)q.a.lens[b], (int64_t)q.a.max_pages * q.a.page);
        over |= !(q.a.flags & DARK_CAUSAL) || last - q.a.T + tt >= 0;
      }
    }
  }
  if (over) report(q.a.dev_status, DARK_ERR_NUMERIC);
}

template <int DP, int WARPS>
cudaError_t launch(const Params& q) {
  static int smem_set[64];
  const int smem = (int)max((1 + 2 * WARPS) * Cfg<DP>::kTile, (uint32_t)WARPS * 16 * (DP + 8) * 4);
  cudaError_t e = set_smem_limit_once((const void*)queries_mma_kernel<DP, WARPS>, smem, smem_set);
  if (e != cudaSuccess) return e;
  const int n = q.a.B * q.a.T;
  queries_mma_kernel<DP, WARPS><<<dim3((n + kRows - 1) / kRows + 1, q.a.H), WARPS * 32, smem, q.a.stream>>>(q);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_queries_mma(const Params& q) {
  return q.p.dp == 64 ? launch<64, 4>(q) : q.p.dp == 128 ? launch<128, 8>(q) : launch<256, 8>(q);
}

}  // namespace cache
}  // namespace dark
