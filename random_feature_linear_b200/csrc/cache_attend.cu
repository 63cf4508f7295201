// Exact-mode attention of T queries of every sequence over a paged cache, for a batch
// whose sequences share one prefix (README, section "Attention modes": in the exact
// mode M acts on queries and keys and ordinary softmax attention follows; section
// "Encoder-decoder model and generation": the exact mode decodes against cached keys
// and values).
//
// The cache holds keys as they are, so the geometry goes to the query's side:
//   y = log2(e) M^T M q / sqrt(d),  s_j = y . k_j,  out = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m).
// Three launches: the queries y with the cut of the own keys into ranges (lengths are
// known on the device only); partial sums of every range (prefix ranges hold the rows of
// the whole batch, so the prefix is read once for all sequences); the join.
//
// This file: the first and last launch, the plan, and the fp32 kernel of the ranges,
// which takes every type, size and layout. bf16 rows of 16-byte multiples take the
// tensor-core kernels.
#include <math.h>
#include <string.h>

#include "cache_attend_mma.cuh"
#include "cache_sched.cuh"

namespace dark {
namespace cache {
namespace {

constexpr int kPrepRows = 8, kPrepTile = 32;         // (256 threads: one a row of M and query)
constexpr long long kPrefixCtas = 2, kOwnCtas = 4;

// --------------------------------------------------- queries in fp32 (SIMT) --

// y of kPrepRows rows of one query head: p = 2 (c_m M) q, y = (c_m M)^T p, kPrepTile rows of
// c_m M at a time through shared memory (read once for both products): a thread a (row of
// M, query) for p, then a thread a column of all queries for y. Sums in fp32.
template <typename T>
__global__ void __launch_bounds__(256) queries_kernel(const __grid_constant__ Params q) {
  using W = typename WeightOf<T>::type;
  pdl_launch();
  if (blockIdx.x == gridDim.x - 1) {
    if (blockIdx.y == 0) make_sched(q);
    return;
  }
  extern __shared__ float sm[];
  const int d = q.a.d, r = q.a.r, tid = threadIdx.x, ld = d + 1;
  float* x = sm;                                         // [kPrepRows][ld]
  float* wt = x + kPrepRows * ld;                        // [kPrepTile][ld]
  float* p = wt + kPrepTile * ld;                        // [kPrepTile][kPrepRows]
  const int h = blockIdx.y, n0 = blockIdx.x * kPrepRows;     // rows (b, t) of head h
  const int n = q.a.B * q.a.T;
  const W* w = (const W*)q.a.w + ((int64_t)(q.a.heads_w == 1 ? 0 : h) * (q.a.m + r) + q.a.m) * d;
  for (int i = tid; i < kPrepRows * d; i += 256) {
    const int row = i / d, c = i - row * d, k = n0 + row;
    float v = 0.f;
    if (k < n) {
      const int b = k / q.a.T, t = k - b * q.a.T;
      v = to_f32(((const T*)q.a.q)[b * q.a.qs[0] + h * q.a.qs[1] + t * q.a.qs[2] + c]);
    }
    x[row * ld + c] = v;
  }
  float s[kPrepRows];
#pragma unroll
  for (int k = 0; k < kPrepRows; ++k) s[k] = 0.f;
  for (int i0 = 0; i0 < r; i0 += kPrepTile) {
    const int here = min(kPrepTile, r - i0);
    __syncthreads();                                     // the last tile's readers are done
#pragma unroll 8
    for (int i = tid; i < here * d; i += 256) {
      const int row = i / d;
      wt[row * ld + i - row * d] = to_f32(w[(int64_t)i0 * d + i]);
    }
    __syncthreads();
    {
      const int i = tid / kPrepRows, k = tid % kPrepRows;
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (i < here)
        for (int c = 0; c < d; c += 4)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = fmaf(wt[i * ld + c + e], x[k * ld + c + e], v[e]);
      p[i * kPrepRows + k] = 2.f * ((v[0] + v[1]) + (v[2] + v[3]));
    }
    __syncthreads();
    if (tid < d)
      for (int i = 0; i < here; ++i) {
        const float u = wt[i * ld + tid];
#pragma unroll
        for (int k = 0; k < kPrepRows; ++k) s[k] = fmaf(u, p[i * kPrepRows + k], s[k]);
      }
  }
  const int g = h % q.G, hk = h / q.G;
  if (tid < d)
    for (int k = 0; k < kPrepRows && n0 + k < n; ++k) {
      const int b = (n0 + k) / q.a.T, t = (n0 + k) - b * q.a.T;
      at<float>(q.a, q.p.o_y)[((int64_t)hk * q.p.all + (b * q.G + g) * q.a.T + t) * q.p.dp + tid] = s[k];
    }
}

// ------------------------------------------------------ ranges in fp32 (SIMT) --

// RB rows against one key range, KT keys at a time: NT threads as RB / 4 row groups of four
// rows. Scores and sums are register tiles of four rows (by KT / CG keys, by up to 16
// columns); the running exponent and weight of a row live in shared memory. Keys and values
// have a buffer each, so that the next keys load under the softmax and the values' product,
// the next values under the next scores; a tile's page numbers are looked up a tile ahead.
// Bound by fp32 multiply-adds for many rows, by the key and value rows' latency for few.
template <typename T, int RB, int KT, int NT>
__global__ void __launch_bounds__(NT) range_kernel(const __grid_constant__ Params q, int prefix, int own) {
  constexpr int RG = RB / 4, CG = NT / RG, KJ = KT / CG, NJ = (256 + 4 * CG - 1) / (4 * CG);
  static_assert(KT % CG == 0 && KT <= NT, "keys over column groups");
  const int hk = blockIdx.y;
  pdl_wait();
  pdl_launch();
  const Item it = item_of(q, blockIdx.x, hk, RB, prefix != 0, own != 0);
  if (!it.any) return;
  extern __shared__ __align__(16) float sm[];
  const int d = q.a.d, ld = d + 4, tid = threadIdx.x;
  float* ys = sm;                         // [RB][ld]
  float* ks = ys + RB * ld;               // [KT][ld]
  float* vs = ks + KT * ld;               // [KT][ld]
  float* sc = vs + KT * ld;               // [KT][RB + 4]: scores, then weights
  float* mx = sc + KT * (RB + 4);         // [RB] reference exponent
  float* lw = mx + RB;                    // [RB] weight
  float* fac = lw + RB;                   // [RB] factor of the sums so far
  int* lim = (int*)(fac + RB);            // [RB] visible keys
  int64_t* rows = (int64_t*)(lim + RB);   // [2][KT] rows of the cache
  const float* y = at<float>(q.a, q.p.o_y) + ((int64_t)hk * q.p.all + it.row0) * q.p.dp;

  auto lookup = [&](int j0) {                            // one key a thread
    if (tid >= KT || j0 + tid >= it.k1) return (int64_t)-1;
    const int64_t row = cache_row(q.a, it.pages, j0 + tid, hk);
    if (row < 0) report(q.a.dev_status, DARK_ERR_INVALID_ARG);
    return row;
  };
  auto fill = [&](const void* pool, float* dst, int tile) {            // zeros past the range
    const int per = d / 4;
    int k = tid / per, c = tid - k * per;
    const int dk = NT / per, dc = NT - dk * per;
    for (; k < KT;) {
      const int64_t row = rows[(tile & 1) * KT + k];
      const T* src = (const T*)pool + (row < 0 ? 0 : row * d + 4 * c);
      float* to = dst + k * ld + 4 * c;
      if constexpr (sizeof(T) == 4) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         (uint32_t)__cvta_generic_to_shared(to)),
                     "l"(src), "r"(row < 0 ? 0 : 16)
                     : "memory");
      } else {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row >= 0) v = make_float4(to_f32(src[0]), to_f32(src[1]), to_f32(src[2]), to_f32(src[3]));
        *reinterpret_cast<float4*>(to) = v;
      }
      k += dk;
      c += dc;
      if (c >= per) {
        c -= per;
        ++k;
      }
    }
    cp_commit();
  };

  int64_t next = lookup(it.k0);
  if (tid < KT) rows[tid] = next;
  for (int i = tid; i < RB * d; i += NT) {
    const int row = i / d, c = i - row * d;
    ys[row * ld + c] = row < it.nrows ? y[(int64_t)row * q.p.dp + c] : 0.f;
  }
  if (tid < RB) {
    mx[tid] = -INFINITY;
    lw[tid] = 0.f;
    lim[tid] = tid < it.nrows ? visible_keys(q, it, tid) : 0;
  }
  const int rg = tid / CG, cg = tid % CG;
  float acc[4][NJ][4];
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[r][j][e] = 0.f;
  __syncthreads();
  fill(q.a.kp, ks, 0);
  fill(q.a.vp, vs, 0);

  for (int j0 = it.k0, tile = 0; j0 < it.k1; j0 += KT, ++tile) {
    const bool more = j0 + KT < it.k1;
    next = lookup(j0 + KT);
    cp_wait<1>();                                        // the keys
    __syncthreads();
    float s[4][KJ];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int k = 0; k < KJ; ++k) s[r][k] = 0.f;
#pragma unroll 2
    for (int c = 0; c < d; c += 4) {
      float4 a[4], b[KJ];
#pragma unroll
      for (int r = 0; r < 4; ++r) a[r] = *reinterpret_cast<const float4*>(ys + (rg * 4 + r) * ld + c);
#pragma unroll
      for (int k = 0; k < KJ; ++k) b[k] = *reinterpret_cast<const float4*>(ks + (cg + k * CG) * ld + c);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int k = 0; k < KJ; ++k) {
          s[r][k] = fmaf(a[r].x, b[k].x, s[r][k]);
          s[r][k] = fmaf(a[r].y, b[k].y, s[r][k]);
          s[r][k] = fmaf(a[r].z, b[k].z, s[r][k]);
          s[r][k] = fmaf(a[r].w, b[k].w, s[r][k]);
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int k = 0; k < KJ; ++k) {
        const int key = j0 + cg + k * CG, row = rg * 4 + r;
        sc[(cg + k * CG) * (RB + 4) + row] = key < it.k1 && key < lim[row] ? s[r][k] : -INFINITY;
      }
    if (more && tid < KT) rows[((tile + 1) & 1) * KT + tid] = next;
    __syncthreads();
    if (more) fill(q.a.kp, ks, tile + 1); else cp_commit();
    // a warp takes rows warp, warp + warps, ...: exponent, weights, factor
    for (int row = tid >> 5; row < RB; row += NT / 32) {
      float top = -INFINITY;
      for (int k = tid & 31; k < KT; k += 32) top = fmaxf(top, sc[k * (RB + 4) + row]);
      top = warp_max(top);
      const float old = mx[row], now = fmaxf(old, top), ref = now == -INFINITY ? 0.f : now;
      float sum = 0.f;
      for (int k = tid & 31; k < KT; k += 32) {
        const float p = exp2f(sc[k * (RB + 4) + row] - ref);
        sc[k * (RB + 4) + row] = p;
        sum += p;
      }
      sum = warp_sum(sum);
      if ((tid & 31) == 0) {
        const float f = exp2f(old - ref);              // 0 before the first visible key
        fac[row] = f;
        lw[row] = fmaf(lw[row], f, sum);
        mx[row] = now;
      }
    }
    cp_wait<1>();                                        // the values
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float f = fac[rg * 4 + r];
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[r][j][e] *= f;
    }
    const int nk = it.k1 - j0 < KT ? it.k1 - j0 : KT;
    int all = nk;                                      // keys that all four rows see
#pragma unroll
    for (int r = 0; r < 4; ++r) all = min(all, lim[rg * 4 + r] - j0);
    auto add = [&](int k, bool masked) {
      const float4 p = *reinterpret_cast<const float4*>(sc + k * (RB + 4) + rg * 4);
      const float pr[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int c = (cg + j * CG) * 4;
        if (c < d) {
          const float4 v = *reinterpret_cast<const float4*>(vs + k * ld + c);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            // a weight of 0 does not cancel an infinite or NaN value behind the mask
            if (masked && j0 + k >= lim[rg * 4 + r]) continue;
            acc[r][j][0] = fmaf(pr[r], v.x, acc[r][j][0]);
            acc[r][j][1] = fmaf(pr[r], v.y, acc[r][j][1]);
            acc[r][j][2] = fmaf(pr[r], v.z, acc[r][j][2]);
            acc[r][j][3] = fmaf(pr[r], v.w, acc[r][j][3]);
          }
        }
      }
    };
    int k = 0;
#pragma unroll 4
    for (; k < all; ++k) add(k, false);
    for (; k < nk; ++k) add(k, true);
    if (more) {
      __syncthreads();
      fill(q.a.vp, vs, tile + 1);
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = rg * 4 + r;
    if (row >= it.nrows) continue;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int c = (cg + j * CG) * 4;
      if (c < d)
        *reinterpret_cast<float4*>(it.acc + (int64_t)row * d + c) =
            make_float4(acc[r][j][0], acc[r][j][1], acc[r][j][2], acc[r][j][3]);
    }
    if (cg == 0) {
      it.ml[2 * row] = mx[row];
      it.ml[2 * row + 1] = lw[row];
    }
  }
}

// -------------------------------------------------------------------- the join --

// out = sum_i 2^(m_i - m) acc_i / sum_i 2^(m_i - m) l_i over a row's prefix and own ranges.
// W warps a row (one for many rows, four for few), each over the ranges w, w + W, ... of
// every 32 W; lanes take the ranges' exponents and weights 32 at a time, then float4 columns
// of 32 / per ranges at once, so that the ranges' sums load without waiting for one another.
// The order of the sums is fixed. Rows that see no key give zeros. Bound by the loads'
// latency: four at a time (19.1 us at 8192 rows of 10 ranges, d = 128; 20.5 as a loop with
// skipped ranges, 24 with eight at a time; at 512 rows, d = 64: 5.4, 6.6 and 7.8).
template <typename T, int W>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ Params q) {
  __shared__ float4 part[W > 1 ? W : 1][2][32];
  __shared__ float parts[W > 1 ? W : 1][2];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = warp % W;
  const int64_t n = (int64_t)blockIdx.x * (4 / W) + warp / W;
  if (n >= (int64_t)q.a.Hk * q.p.all) return;            // (W = 4: the whole CTA)
  const int hk = (int)(n / q.p.all), row = (int)(n - (int64_t)hk * q.p.all);
  const int b = row / q.p.rows, in = row - b * q.p.rows, g = in / q.a.T, t = in - g * q.a.T;
  const int len = sched_len(q)[b], o0 = sched_off(q)[b], o1 = sched_off(q)[b + 1];
  const bool pad = (q.a.flags & DARK_CAUSAL) && len - q.a.T + t < 0;
  const int d = q.a.d, np = q.a.prefix_len > 0 && !pad ? q.p.p_splits : 0, no = pad ? 0 : o1 - o0;
  const int total = np + no;
  const int64_t pslot = (int64_t)hk * q.p.p_splits * q.p.all + row, pstep = q.p.all;
  const int64_t oslot = ((int64_t)hk * q.p.cap + o0) * q.p.rows + in, ostep = q.p.rows;
  const float2* pml = at<float2>(q.a, q.p.o_pml) + pslot;
  const float2* oml = at<float2>(q.a, q.p.o_oml) + oslot;
  auto ml = [&](int i) {
    return i >= total ? make_float2(-INFINITY, 0.f) : i < np ? pml[i * pstep] : oml[(i - np) * ostep];
  };
  // this warp's ranges w, w + W, ...; columns: `per` lanes a range, float4 c, c + 128
  const int per = d <= 32 ? 8 : d <= 64 ? 16 : 32, sub = lane / per, subs = 32 / per;
  const int c = 4 * (lane % per);
  const float* pa = at<float>(q.a, q.p.o_pacc) + pslot * d;
  const float* oa = at<float>(q.a, q.p.o_oacc) + oslot * d;
  float2 mine = ml(lane * W + w);
  float top = mine.x;
  for (int i = (lane + 32) * W + w; i < total; i += 32 * W) top = fmaxf(top, ml(i).x);
  top = warp_max(top);
  const float ref = top == -INFINITY ? 0.f : top;
  float l = 0.f;
  constexpr int U = 4;
  float4 o[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int i0 = 0; i0 * W + w < total; i0 += 32) {
    if (i0 > 0) mine = ml((i0 + lane) * W + w);
    const float f = exp2f(mine.x - ref);
    l += f * mine.y;
    const int count = min(32, (total - w + W - 1) / W - i0);
    for (int i = 0; i < count; i += U * subs) {          // U loads a lane in flight
      float4 v[U][2];
      float x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = i + u * subs + sub, k = (i0 + at) * W + w;
        x[u] = __shfl_sync(0xffffffffu, f, at & 31);
        if (at >= count) x[u] = 0.f;
        const float* src = k < np ? pa + k * pstep * d : oa + (k - np) * ostep * d;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          v[u][j] = make_float4(0.f, 0.f, 0.f, 0.f);
          // no visible key (a weight of 0): acc is not read
          if (x[u] != 0.f && c + 128 * j < d) v[u][j] = *reinterpret_cast<const float4*>(src + c + 128 * j);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          o[j].x = fmaf(x[u], v[u][j].x, o[j].x);
          o[j].y = fmaf(x[u], v[u][j].y, o[j].y);
          o[j].z = fmaf(x[u], v[u][j].z, o[j].z);
          o[j].w = fmaf(x[u], v[u][j].w, o[j].w);
        }
    }
  }
  l = warp_sum(l);
  for (int s = per; s < 32; s <<= 1) {
    o[0].x += __shfl_xor_sync(0xffffffffu, o[0].x, s);
    o[0].y += __shfl_xor_sync(0xffffffffu, o[0].y, s);
    o[0].z += __shfl_xor_sync(0xffffffffu, o[0].z, s);
    o[0].w += __shfl_xor_sync(0xffffffffu, o[0].w, s);
  }
  if constexpr (W > 1) {                                 // the warps' sums, in order
    part[w][0][lane] = o[0];
    part[w][1][lane] = o[1];
    if (lane == 0) {
      parts[w][0] = top;
      parts[w][1] = l;
    }
    __syncthreads();
    if (w > 0) return;
    float all = -INFINITY;
    for (int k = 0; k < W; ++k) all = fmaxf(all, parts[k][0]);
    l = 0.f;
    o[0] = o[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < W; ++k) {
      const float f = exp2f(parts[k][0] - (all == -INFINITY ? 0.f : all));
      l = fmaf(f, parts[k][1], l);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4 v = part[k][j][lane];
        o[j].x = fmaf(f, v.x, o[j].x);
        o[j].y = fmaf(f, v.y, o[j].y);
        o[j].z = fmaf(f, v.z, o[j].z);
        o[j].w = fmaf(f, v.w, o[j].w);
      }
    }
  }
  T* dst = (T*)q.a.out + b * q.a.os[0] + (int64_t)(hk * q.G + g) * q.a.os[1] + t * q.a.os[2];
  bool bad = false;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float v[4] = {o[j].x, o[j].y, o[j].z, o[j].w};
    if (sub > 0 || c + 128 * j >= d) break;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = l == 0.f ? 0.f : v[e] / l;
      bad |= !isfinite(x);
      dst[c + 128 * j + e] = from_f32<T>(x);
    }
  }
  if (bad) report(q.a.dev_status, DARK_ERR_NUMERIC);
}

// -------------------------------------------------------------------- the plan --

// Rows of a block. fp32: blocks of 64 read the keys less often and compute more a byte, blocks
// of 8 fill more SMs: 32 rows of 8 key heads over 512 and 4096 keys of a prefix, d = 64, 36.8 and
// 84.2 us in blocks of 64, 23.4 and 84.6 of 8; 48 rows 37.3 and 85.1 against 33.6 and 115.6;
// 32 and 48 rows of a sequence's 1024 keys 140 and 144 against 101 and 163.
int row_block(const Plan& p, int rows) {
  if (p.mma) return mma_rows(p.dp, p.rows);
  return rows > 32 ? 64 : 8;
}

// Ranges of the tcgen05 kernel (one CTA an SM): the count whose waves of CTAs, each with
// its tiles and about two tiles' time to start and end, take the least time.
void split_tiles(const CacheAttnArgs& a, Plan* p) {
  const long long tiles = (a.prefix_len + kTcKeys - 1) / kTcKeys;
  const long long blocks = (long long)a.Hk * ((p->all + kTcRows - 1) / kTcRows);
  long long best = -1;
  for (long long s = 1; s <= tiles && (s == 1 || blocks * s <= 4 * 148); ++s) {
    const long long per = (tiles + s - 1) / s, cost = (blocks * s + 147) / 148 * (per + 2);
    if (best < 0 || cost < best) {
      best = cost;
      p->p_chunk = (int)(per * kTcKeys);
    }
  }
  p->p_splits = (a.prefix_len + p->p_chunk - 1) / p->p_chunk;
}

Plan make_plan(const CacheAttnArgs& a) {
  Plan p;
  memset(&p, 0, sizeof(p));
  p.rows = a.H / a.Hk * a.T;
  p.all = a.B * p.rows;
  p.mma = a.dtype == DARK_BF16 && a.d % 8 == 0;
  p.dp = p.mma ? (a.d <= 64 ? 64 : a.d <= 128 ? 128 : 256) : a.d;
  // The prefix's kernel. us of a captured call in a row of such calls, 8 key heads, 16 own keys,
  // d = 64 / 128, by tcgen05 | by warps that share keys | in one launch with the own ranges:
  //   32 rows,   512 keys  16.2 / 19.8 | 16.3 /  19.5 |  12.5 /  15.4
  //   32 rows,  8192       20.9 / 25.6 | 23.3 /  29.9 |  24.4 /  36.1
  //   48 rows, 32768       37.7 / 49.8 | 64.4 /  96.7 |  84.4 / 151.6
  //   64 rows,   512       17.4 / 20.7 | 18.8 /  23.8 |  13.5 /  17.0
  //   64 rows,  2048       17.8 / 21.8 | 20.5 /  27.1 |  19.1 /  26.8
  //  256 rows,   512       21.4 / 27.8 | 22.7 /  33.4 |  20.9 /  29.2
  // (d = 256, 32 rows: 30.5 | 24.6 at 512 keys and 36.5 | 42.7 at 4096 for the last two.) A launch of
  // its own costs 4 to 5 us and is worth it from about 2^17 rows x keys on; tcgen05 would pay from
  // 17 rows on as well, and is kept to 64 rows because it takes keys up to 65504 only.
  p.tc = p.mma && p.dp <= 128 && p.all >= 64 && a.prefix_len >= 256;
  p.share = p.mma && !p.tc && p.all > 16 && a.prefix_len > 0;
  // ranges: about as many CTAs (over key heads, row blocks and ranges) as run at once
  const long long want = kPrefixCtas * 148, want_own = kOwnCtas * 148;
  const int prb = p.share ? share_rows(p.dp, p.all) : row_block(p, p.all);
  const long long pb = (long long)a.Hk * ((p.all + prb - 1) / prb);
  const int steps = (a.prefix_len + kKeyStep - 1) / kKeyStep;
  long long s = (want + pb - 1) / pb;
  const long long most = p.mma ? (steps + 1) / 2 : steps;
  if (s > most) s = most;
  if (s < 1) s = 1;
  p.p_chunk = steps == 0 ? kKeyStep : (int)((steps + s - 1) / s * kKeyStep);
  p.p_splits = steps == 0 ? 1 : (a.prefix_len + p.p_chunk - 1) / p.p_chunk;
  if (p.tc) split_tiles(a, &p);
  const long long ob = (long long)a.Hk * ((p.rows + row_block(p, p.rows) - 1) / row_block(p, p.rows));
  p.cap = a.B + (int)((want_own + ob - 1) / ob);
  size_t o = kWsHeader;
  auto take = [&](size_t n) {
    const size_t at = o;
    o += align_up(n, 256);
    return at;
  };
  const size_t krows = (size_t)a.Hk * p.all;
  p.o_sched = take((size_t)p.cap * 16 + (size_t)(2 * a.B + 1) * 4);
  p.o_y = take(krows * p.dp * 4);
  p.o_y16 = take(p.tc ? krows * p.dp * 2 : 0);
  p.o_pacc = take(a.prefix_len > 0 ? krows * p.p_splits * a.d * 4 : 0);
  p.o_pml = take(a.prefix_len > 0 ? krows * p.p_splits * 8 : 0);
  p.o_oacc = take((size_t)a.Hk * p.cap * p.rows * a.d * 4);
  p.o_oml = take((size_t)a.Hk * p.cap * p.rows * 8);
  p.bytes = o;
  return p;
}

// Bytes that no call with as many sequences, queries a sequence and prefix tokens, or fewer,
// needs more of. (A plan alone may shrink as the call grows: more rows fill the GPU with
// fewer ranges of the prefix, and 64 rows go by other tiles than 63.) Of the splits above:
//  * p_splits <= want / pb + 1 with pb >= Hk max(1, all / prb): Hk all p_splits <= min(all, prb) want +
//    Hk all; on tcgen05 p_splits <= 4 * 148 / blocks or 1 alike with 256-row blocks; and
//    p_splits is at most the prefix's steps, or tiles, everywhere;
//  * cap <= B + want_own / ob + 1 alike, with the row blocks of a sequence.
// Each right-hand side grows with B, T and prefix_len.
size_t bound_bytes(const CacheAttnArgs& a, const Plan& p) {
  const size_t Hk = a.Hk, krows = Hk * p.all, rows = p.rows, all = p.all;
  const size_t want = kPrefixCtas * 148, want_own = kOwnCtas * 148;
  const size_t steps = ((size_t)a.prefix_len + kKeyStep - 1) / kKeyStep;
  const size_t prb = p.mma && p.dp == 256 ? 32 : 64, rb = p.mma ? 16 : 64;
  auto least = [](size_t x, size_t y) { return x < y ? x : y; };
  auto most = [](size_t x, size_t y) { return x > y ? x : y; };
  size_t part = least(least(all, prb) * want + krows, krows * steps);
  if (p.mma && p.dp <= 128 && all >= 64 && a.prefix_len >= 256)
    part = most(part, least(most(least(all, kTcRows) * 4 * 148, krows), krows * ((steps + 1) / 2)));
  const size_t own = krows + least(rows, rb) * want_own + Hk * rows;
  const size_t cap = a.B + (want_own + Hk - 1) / Hk;
  const bool y16 = p.mma && p.dp <= 128 && all >= 64 && a.prefix_len >= 256;
  return kWsHeader + align_up(cap * 16 + (2 * (size_t)a.B + 1) * 4, 256) + align_up(krows * p.dp * 4, 256) +
         align_up(y16 ? krows * p.dp * 2 : 0, 256) + align_up(part * a.d * 4, 256) + align_up(part * 8, 256) +
         align_up(own * a.d * 4, 256) + align_up(own * 8, 256);
}

template <typename T, int RB, int KT, int NT>
cudaError_t launch_range(const Params& q, bool prefix, bool own) {
  static int smem_set[64];
  auto bytes = [](size_t d) {
    return ((RB + 2 * KT) * (d + 4) + (size_t)KT * (RB + 4) + 4 * RB) * 4 + 2 * KT * 8;
  };
  auto* kernel = range_kernel<T, RB, KT, NT>;
  cudaError_t e = set_smem_limit_once((const void*)kernel, (int)bytes(256), smem_set);
  if (e != cudaSuccess) return e;
  long long n = 0;
  if (prefix) n += (long long)q.p.p_splits * ((q.p.all + RB - 1) / RB);
  if (own) n += (long long)q.p.cap * ((q.p.rows + RB - 1) / RB);
  return launch_dependent(kernel, dim3((unsigned)n, q.a.Hk), dim3(NT), bytes(q.a.d), q.a.stream, q,
                          prefix ? 1 : 0, own ? 1 : 0);
}
// 64 rows a CTA where there are more than 32, else 8.
template <typename T>
cudaError_t launch_ranges(const Params& q, bool prefix, bool own) {
  return row_block(q.p, prefix ? q.p.all : q.p.rows) == 64 ? launch_range<T, 64, 64, 256>(q, prefix, own)
                                                          : launch_range<T, 8, 64, 128>(q, prefix, own);
}

template <typename T>
cudaError_t launch_all(const Params& q) {
  const int n = q.a.B * q.a.T;
  cudaError_t e;
  if (q.p.mma) {
    e = launch_queries_mma(q);
  } else {
    const size_t smem = ((size_t)(kPrepRows + kPrepTile) * (q.a.d + 1) + kPrepTile * kPrepRows) * 4;
    queries_kernel<T><<<dim3((n + kPrepRows - 1) / kPrepRows + 1, q.a.H), 256, smem, q.a.stream>>>(q);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  if (q.p.mma) {
    if (q.p.tc) e = launch_prefix_tc(q);
    if (q.p.share) e = launch_prefix_mma(q);
    if (e == cudaSuccess) e = launch_ranges_mma(q);
    if (e != cudaSuccess) return e;
  } else {
    // one launch for the prefix and the own ranges where their row blocks are the same
    const bool prefix = q.a.prefix_len > 0, both = row_block(q.p, q.p.all) == row_block(q.p, q.p.rows);
    if (prefix && !both) e = launch_ranges<T>(q, true, false);
    if (e == cudaSuccess) e = launch_ranges<T>(q, prefix && both, true);
    if (e != cudaSuccess) return e;
  }
  const int64_t rows = (int64_t)q.a.Hk * q.p.all;
  // a warp a row while that gives every SM about eight warps (whole calls, 8 key heads, d = 64,
  // prefix 2048: 128 rows 19.9 us with one warp and 20.1 with four, 256 rows 23.7 and 26.5;
  // 16 rows 13.4 and 12.2)
  return rows >= 8 * num_sms()
             ? launch_dependent(join_kernel<T, 1>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, q.a.stream, q)
             : launch_dependent(join_kernel<T, 4>, dim3((unsigned)rows), dim3(128), 0, q.a.stream, q);
}

}  // namespace
}  // namespace cache

size_t cache_attention_workspace_bytes(const CacheAttnArgs& a) {
  const cache::Plan p = cache::make_plan(a);
  const size_t b = cache::bound_bytes(a, p);
  return b > p.bytes ? b : p.bytes;
}

cudaError_t launch_cache_attention(const CacheAttnArgs& a) {
  cache::Params q;
  q.a = a;
  q.p = cache::make_plan(a);
  q.G = a.H / a.Hk;
  q.box_rows = 0;
  q.stall = test_stall_cycles();
  return a.dtype == DARK_BF16 ? cache::launch_all<__nv_bfloat16>(q) : cache::launch_all<float>(q);
}

}  // namespace dark
