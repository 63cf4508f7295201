// The cut of the sequences' own keys into ranges, made by one block of the launch that
// computes the queries (the lengths are known on the device only).
#pragma once

#include "cache_attend.cuh"

namespace dark {
namespace cache {

// The cut of the own keys: ranges of `chunk` keys, as short as `cap` ranges allow (so
// that a few long sequences spread over the GPU too).
__device__ inline void make_sched(const Params& q) {
  __shared__ int part[33];
  __shared__ long long wsum[32];
  __shared__ int chunk_s;
  int4* range = sched_range(q);
  int *off = sched_off(q), *len = sched_len(q);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x / 32;
  const int64_t most = (int64_t)q.a.max_pages * q.a.page;
  long long sum = 0;
  for (int b = tid; b < q.a.B; b += blockDim.x) {
    int64_t n = q.a.lens[b];
    if (n < 0 || n > most) {
      report(q.a.dev_status, DARK_ERR_INVALID_ARG);
      n = n < 0 ? 0 : most;
    }
    len[b] = (int)n;
    sum += n;
  }
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) wsum[warp] = sum;
  __syncthreads();
  if (tid == 0) {
    long long all = 0;
    for (int w = 0; w < nw; ++w) all += wsum[w];
    // sum ceil(len / chunk) <= all / chunk + B <= cap
    const long long room = q.p.cap - q.a.B > 0 ? q.p.cap - q.a.B : 1;
    long long c = (all + room - 1) / room;
    c = (c + kKeyStep - 1) / kKeyStep * kKeyStep;
    // no sequence is longer than 2^30 keys: longer ranges change nothing
    const int least = q.p.mma ? 2 * kKeyStep : kKeyStep;   // (fp32: a tile; 20.5 us against 25.4)
    chunk_s = c < least ? least : c < (1 << 30) ? (int)c : 1 << 30;
  }
  __syncthreads();
  const int chunk = chunk_s;
  int base = 0;
  for (int b0 = 0; b0 < q.a.B; b0 += blockDim.x) {
    const int b = b0 + tid;
    const int n = b < q.a.B ? (int)(((long long)len[b] + chunk - 1) / chunk) : 0;
    int x = n;
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) part[warp] = x;
    __syncthreads();
    int before = base;
    for (int w = 0; w < warp; ++w) before += part[w];
    if (b < q.a.B) {
      off[b] = before + x - n;
      for (int i = 0; i < n; ++i)
        range[before + x - n + i] = make_int4(b, i * chunk, min((i + 1) * (long long)chunk, (long long)len[b]), len[b]);
    }
    int all = 0;
    for (int w = 0; w < nw; ++w) all += part[w];
    base += all;
    __syncthreads();
  }
  if (tid == 0) off[q.a.B] = base;
  for (int i = base + tid; i < q.p.cap; i += blockDim.x) range[i] = make_int4(0, 0, 0, 0);
}

}  // namespace cache
}  // namespace dark
