// Norms of queries and keys for each head with the position rotation in the same
// pass, its backward pass, and the append of keys and values to a paged cache.
//
// A row is one head's d values x of one token at position p:
//   n = x / sqrt(mean(x^2) + eps),  y = n gamma           (without gamma: y = x)
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t)      t = 2 pi frac(p turns_i)
// for the pairs i of the first `rot` values. Backward, with u the cotangent turned
// by -t, w = u gamma:  dx = rstd (w - n mean(w n)),  dgamma = sum over rows of u n.
//
// Angles: turns_i is the pair's frequency over 2 pi as a fraction of 2^64, so the
// product p turns_i modulo 2^64 is the exact angle's fraction of a turn for every
// 64-bit position (an fp32 product would be off by a radian at p ~ 1e7); its upper
// 32 bits give an fp32 angle, off by at most 2^-25 turns of pi.
//
// Every kernel is bound by reading and writing its rows (2, 3 or 4 accesses of
// n elements and ~20 instructions an element). A lane group of 1-32 lanes holds a
// row in registers, eight elements a lane: one read, one shuffle reduction, one
// write. A CTA takes a tile of tokens and all heads of a group, so that a token's
// cosines and sines are computed once, in shared memory, for its heads.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace dark {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kTile = 32;                 // tokens of a CTA's tile, at most

// N elements of T as raw words, loaded and stored at once (N sizeof(T) in 2..16).
template <int kBytes> struct Raw;
template <> struct Raw<2> { using type = uint16_t; };
template <> struct Raw<4> { using type = uint32_t; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<16> { using type = uint4; };
template <typename T, int N>
union Pack {
  typename Raw<(int)sizeof(T) * N>::type raw;
  T v[N];
  __device__ Pack() {}
};
template <typename T, int N>
__device__ __forceinline__ void load(Pack<T, N>& p, const T* src) {
  p.raw = *reinterpret_cast<const decltype(p.raw)*>(src);
}
template <typename T, int N>
__device__ __forceinline__ void store(T* dst, const Pack<T, N>& p) {
  *reinterpret_cast<decltype(p.raw)*>(dst) = p.raw;
}

// A lane's unit u of a row: N pairs (2 N elements) in two runs of N. Rotated units
// take the pairs [N u, N u + N); the units behind them 2 N elements in a row.
template <int N>
struct Unit {
  int lo, hi, pair;                       // element offsets; first pair, -1: not rotated
  __device__ Unit(int u, int rot, int inter) {
    const int ru = rot / (2 * N);
    if (u < ru) {
      pair = N * u;
      lo = inter ? 2 * N * u : N * u;
      hi = inter ? lo + N : rot / 2 + N * u;
    } else {
      pair = -1;
      lo = 2 * N * u;                     // = rot + 2 N (u - ru)
      hi = lo + N;
    }
  }
};

// Rotates a unit's 2 N values in place; `s` is +1, or -1 for the transpose.
template <int N>
__device__ __forceinline__ void turn(float (&x)[2 * N], const float2* cs, int inter, float s) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float c = cs[i].x, t = s * cs[i].y;
    float& a = inter ? x[2 * i] : x[i];
    float& b = inter ? x[2 * i + 1] : x[N + i];
    const float a0 = a, b0 = b;
    a = fmaf(a0, c, -b0 * t);
    b = fmaf(a0, t, b0 * c);
  }
}

__device__ __forceinline__ float group_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// What the kernels know of a tile's tokens, in shared memory.
struct Token {
  int b, l;
  int64_t row;                            // append: cache row of head 0, or -1: not written
};

struct Tile {
  uint64_t turns[128];
  Token tok[kTile];
  int64_t pos[kTile];
};

// Tokens [n0, n0 + count) of the call: their places, positions, and cosines and
// sines (cs[token][pair], computed once for all heads of the CTA).
__device__ __forceinline__ void fill_tile(const NormRopeArgs& a, Tile& t, float2* cs, int64_t n0,
                                          int count) {
  const int np = a.rope.dims / 2, tid = threadIdx.x;
  for (int i = tid; i < np; i += kThreads) t.turns[i] = a.rope.turns[i];
  if (tid < count) {
    const int64_t n = n0 + tid;
    Token k;
    k.b = (int)(n / a.L);
    k.l = (int)(n - (int64_t)k.b * a.L);
    k.row = -1;
    int64_t place = k.l;
    if (a.lens != nullptr) {
      const int have = a.lens[k.b];
      place += have;
      const bool fresh = a.new_lens == nullptr || k.l < a.new_lens[k.b];
      if (fresh) {
        const int64_t pg = place / a.page;
        const int id = have >= 0 && pg < a.max_pages ? a.table[(int64_t)k.b * a.max_pages + pg] : -1;
        if (id >= 0 && id < a.pages)
          k.row = (int64_t)id * a.set[0].heads * a.page + place % a.page;
        else
          report(a.dev_status, DARK_ERR_INVALID_ARG);
      }
    }
    t.tok[tid] = k;
    t.pos[tid] = a.positions != nullptr ? (int64_t)a.positions[n] : a.pos0 + place;
  }
  __syncthreads();
  for (int i = tid; i < count * np; i += kThreads) {
    const int k = i / np, p = i - k * np;
    const uint64_t phase = (uint64_t)t.pos[k] * t.turns[p];
    // [-2^31, 2^31) / 2^31 half turns
    const float x = (float)(int32_t)(phase >> 32) * 4.656612873077393e-10f;
    float s, c;
    sincospif(x, &s, &c);
    cs[i] = make_float2(c, s);
  }
  __syncthreads();
}

// Forward: U rows of one head in flight for every lane group. N pairs a unit, NU
// units a lane. Rows are normed where the set has a gamma, turned where `rotate`.
template <typename T, int N, int NU, int U>
__global__ void __launch_bounds__(kThreads) rows_kernel(const __grid_constant__ NormRopeArgs a,
                                                        int lanes, int tile, int hchunk) {
  extern __shared__ __align__(16) uint8_t smem[];
  Tile& t = *reinterpret_cast<Tile*>(smem);
  float2* cs = reinterpret_cast<float2*>(smem + sizeof(Tile));
  const int64_t ntok = (int64_t)a.B * a.L, n0 = (int64_t)blockIdx.x * tile;
  const int count = ntok - n0 < tile ? (int)(ntok - n0) : tile;
  fill_tile(a, t, cs, n0, count);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = 32 / lanes, g = lane / lanes, lu = lane % lanes;
  const int np = a.rope.dims / 2, inter = a.rope.interleaved;
  const int per = rows * U, blocks = (count + per - 1) / per;
  const int h0 = blockIdx.y * hchunk;
  const int nh = a.set[0].heads + a.set[1].heads - h0 < hchunk
                     ? a.set[0].heads + a.set[1].heads - h0 : hchunk;
  bool bad = false;
  for (int it = warp; it < nh * blocks; it += kWarps) {
    const int hh = h0 + it / blocks, k0 = (it % blocks) * per;
    const int which = hh >= a.set[0].heads ? 1 : 0;
    const RowSet& rs = a.set[which];
    const int h = hh - (which ? a.set[0].heads : 0);
    const T* x = (const T*)rs.x + (int64_t)h * rs.xs[1];
    const int rot = rs.rotate ? a.rope.dims : 0;
    const float* gamma =
        rs.gamma == nullptr ? nullptr : rs.gamma + (rs.gheads > 1 ? (int64_t)h * a.d : 0);
    Pack<T, N> lo[U][NU], hi[U][NU];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * rows + g;
      if (k < count && !(a.lens != nullptr && t.tok[k].row < 0)) {
        const T* src = x + (int64_t)t.tok[k].b * rs.xs[0] + (int64_t)t.tok[k].l * rs.xs[2];
#pragma unroll
        for (int e = 0; e < NU; ++e) {
          const int i = lu + e * lanes;
          if (2 * N * i < a.d) {
            const Unit<N> un(i, rot, inter);
            load(lo[u][e], src + un.lo);
            load(hi[u][e], src + un.hi);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * rows + g;
      const bool live = k < count && !(a.lens != nullptr && t.tok[k].row < 0);
      T* dst = nullptr;
      if (live)
        dst = a.lens != nullptr
                  ? (T*)rs.y + (t.tok[k].row + (int64_t)h * a.page) * a.d
                  : (T*)rs.y + (int64_t)h * rs.ys[1] + (int64_t)t.tok[k].b * rs.ys[0] +
                        (int64_t)t.tok[k].l * rs.ys[2];
      if (gamma == nullptr && rot == 0) {            // a plain copy keeps the bits
        if (live) {
#pragma unroll
          for (int e = 0; e < NU; ++e) {
            const int i = lu + e * lanes;
            if (2 * N * i < a.d) {
              store(dst + 2 * N * i, lo[u][e]);
              store(dst + 2 * N * i + N, hi[u][e]);
            }
          }
        }
        continue;
      }
      float v[NU][2 * N], ss = 0.f;
#pragma unroll
      for (int e = 0; e < NU; ++e) {
        const bool has = live && 2 * N * (lu + e * lanes) < a.d;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          v[e][i] = has ? to_f32(lo[u][e].v[i]) : 0.f;
          v[e][N + i] = has ? to_f32(hi[u][e].v[i]) : 0.f;
          ss = fmaf(v[e][i], v[e][i], ss);
          ss = fmaf(v[e][N + i], v[e][N + i], ss);
        }
      }
      float rstd = 1.f;
      if (gamma != nullptr) {
        ss = group_sum(ss, lanes);
        rstd = 1.f / sqrtf(ss / (float)a.d + a.eps);
        bad |= live && !isfinite(ss);                // a sum of squares past fp32
      }
      if (!live) continue;
#pragma unroll
      for (int e = 0; e < NU; ++e) {
        const int i = lu + e * lanes;
        if (2 * N * i >= a.d) continue;
        const Unit<N> un(i, rot, inter);
        if (gamma != nullptr) {
          Pack<float, N> glo, ghi;
          load(glo, gamma + un.lo);
          load(ghi, gamma + un.hi);
#pragma unroll
          for (int j = 0; j < N; ++j) {
            v[e][j] *= rstd * glo.v[j];
            v[e][N + j] *= rstd * ghi.v[j];
          }
        }
        if (un.pair >= 0) turn<N>(v[e], cs + k * np + un.pair, inter, 1.f);
        Pack<T, N> olo, ohi;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          bad |= !isfinite(v[e][j]) || !isfinite(v[e][N + j]);
          olo.v[j] = from_f32<T>(v[e][j]);
          ohi.v[j] = from_f32<T>(v[e][N + j]);
        }
        store(dst + un.lo, olo);
        store(dst + un.hi, ohi);
      }
    }
  }
  if (bad) report(a.dev_status, DARK_ERR_NUMERIC);
}

// Backward. blockIdx.y is a group of at most kWarps heads, a warp keeps one head
// (with fewer heads, several warps share one and split its tokens), and a CTA walks
// tiles blockIdx.x, blockIdx.x + gridDim.x, ...: dgamma stays in registers, one sum a
// tile added to one over the tiles (two levels: the fp32 sums stay short), and each
// warp leaves one row for the reduction below.
template <typename T, int N, int NU>
__global__ void __launch_bounds__(kThreads) rows_bwd_kernel(const __grid_constant__ NormRopeArgs a,
                                                            int lanes, int tile) {
  constexpr int U = NU > 1 ? 1 : 2;
  extern __shared__ __align__(16) uint8_t smem[];
  Tile& t = *reinterpret_cast<Tile*>(smem);
  float2* cs = reinterpret_cast<float2*>(smem + sizeof(Tile));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = 32 / lanes, g = lane / lanes, lu = lane % lanes;
  const int np = a.rope.dims / 2, inter = a.rope.interleaved;
  const int nh = a.set[0].heads + a.set[1].heads;
  const int h0 = blockIdx.y * kWarps;
  const int hg = nh < kWarps ? nh : kWarps, split = kWarps / hg;
  const int hh = h0 + warp % hg, part = warp / hg;
  const bool on = hh < nh && part < split;
  const int which = hh >= a.set[0].heads ? 1 : 0;
  const RowSet& rs = a.set[which];
  const int h = hh - (which ? a.set[0].heads : 0);
  const int rot = rs.rotate ? a.rope.dims : 0;
  const float* gamma =
      rs.gamma == nullptr ? nullptr : rs.gamma + (rs.gheads > 1 ? (int64_t)h * a.d : 0);
  float sum[NU][2 * N];
#pragma unroll
  for (int e = 0; e < NU; ++e)
#pragma unroll
    for (int j = 0; j < 2 * N; ++j) sum[e][j] = 0.f;
  bool bad = false;

  const int64_t ntok = (int64_t)a.B * a.L;
  for (int64_t n0 = (int64_t)blockIdx.x * tile; n0 < ntok; n0 += (int64_t)gridDim.x * tile) {
    const int count = ntok - n0 < tile ? (int)(ntok - n0) : tile;
    __syncthreads();                                 // the last tile's readers are done
    fill_tile(a, t, cs, n0, count);
    if (!on) continue;
    float acc[NU][2 * N];
#pragma unroll
    for (int e = 0; e < NU; ++e)
#pragma unroll
      for (int j = 0; j < 2 * N; ++j) acc[e][j] = 0.f;
    for (int k0 = part * rows * U; k0 < count; k0 += split * rows * U) {
      Pack<T, N> xlo[U][NU], xhi[U][NU], glo[U][NU], ghi[U][NU];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * rows + g;
        if (k >= count) continue;
        const int64_t tb = t.tok[k].b, tl = t.tok[k].l;
        const T* xr = (const T*)rs.x + (int64_t)h * rs.xs[1] + tb * rs.xs[0] + tl * rs.xs[2];
        const T* gr = (const T*)rs.g + (int64_t)h * rs.gs[1] + tb * rs.gs[0] + tl * rs.gs[2];
#pragma unroll
        for (int e = 0; e < NU; ++e) {
          const int i = lu + e * lanes;
          if (2 * N * i >= a.d) continue;
          const Unit<N> un(i, rot, inter);
          if (gamma != nullptr) {
            load(xlo[u][e], xr + un.lo);
            load(xhi[u][e], xr + un.hi);
          }
          load(glo[u][e], gr + un.lo);
          load(ghi[u][e], gr + un.hi);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * rows + g;
        const bool live = k < count;
        float x[NU][2 * N], w[NU][2 * N], ss = 0.f, dot = 0.f;
#pragma unroll
        for (int e = 0; e < NU; ++e) {
          const int i = lu + e * lanes;
          const bool has = live && 2 * N * i < a.d;
          const Unit<N> un(i, rot, inter);
#pragma unroll
          for (int j = 0; j < N; ++j) {
            x[e][j] = has && gamma != nullptr ? to_f32(xlo[u][e].v[j]) : 0.f;
            x[e][N + j] = has && gamma != nullptr ? to_f32(xhi[u][e].v[j]) : 0.f;
            w[e][j] = has ? to_f32(glo[u][e].v[j]) : 0.f;
            w[e][N + j] = has ? to_f32(ghi[u][e].v[j]) : 0.f;
          }
          if (has && un.pair >= 0) turn<N>(w[e], cs + k * np + un.pair, inter, -1.f);   // u
          if (has && gamma != nullptr) {
            Pack<float, N> mlo, mhi;
            load(mlo, gamma + un.lo);
            load(mhi, gamma + un.hi);
#pragma unroll
            for (int j = 0; j < N; ++j) {
              ss = fmaf(x[e][j], x[e][j], ss);
              ss = fmaf(x[e][N + j], x[e][N + j], ss);
              dot = fmaf(w[e][j] * mlo.v[j], x[e][j], dot);
              dot = fmaf(w[e][N + j] * mhi.v[j], x[e][N + j], dot);
            }
          }
        }
        float rstd = 1.f, back = 0.f;
        if (gamma != nullptr) {
          ss = group_sum(ss, lanes);
          dot = group_sum(dot, lanes);
          rstd = 1.f / sqrtf(ss / (float)a.d + a.eps);
          back = dot * rstd * rstd / (float)a.d;     // mean(w n) rstd
          bad |= live && !isfinite(ss);
        }
        if (!live) continue;
        T* dr = (T*)rs.y + (int64_t)h * rs.ys[1] + (int64_t)t.tok[k].b * rs.ys[0] +
                (int64_t)t.tok[k].l * rs.ys[2];
#pragma unroll
        for (int e = 0; e < NU; ++e) {
          const int i = lu + e * lanes;
          if (2 * N * i >= a.d) continue;
          const Unit<N> un(i, rot, inter);
          float dx[2 * N];
          if (gamma != nullptr) {
            Pack<float, N> mlo, mhi;
            load(mlo, gamma + un.lo);
            load(mhi, gamma + un.hi);
#pragma unroll
            for (int j = 0; j < 2 * N; ++j) {
              const float m = j < N ? mlo.v[j % N] : mhi.v[j % N];
              acc[e][j] = fmaf(w[e][j], x[e][j] * rstd, acc[e][j]);
              dx[j] = rstd * fmaf(-x[e][j], back, w[e][j] * m);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 2 * N; ++j) dx[j] = w[e][j];
          }
          Pack<T, N> olo, ohi;
#pragma unroll
          for (int j = 0; j < N; ++j) {
            bad |= !isfinite(dx[j]) || !isfinite(dx[N + j]);
            olo.v[j] = from_f32<T>(dx[j]);
            ohi.v[j] = from_f32<T>(dx[N + j]);
          }
          store(dr + un.lo, olo);
          store(dr + un.hi, ohi);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < NU; ++e)
#pragma unroll
      for (int j = 0; j < 2 * N; ++j) sum[e][j] += acc[e][j];
  }
  if (bad) report(a.dev_status, DARK_ERR_NUMERIC);
  if (!on || gamma == nullptr) return;
  // the warp's row of partial sums: [head][slot][d]
  float* out = a.part + ((int64_t)hh * gridDim.x * split + (int64_t)blockIdx.x * split + part) * a.d;
#pragma unroll
  for (int e = 0; e < NU; ++e) {
    const int i = lu + e * lanes;
    const Unit<N> un(i, rot, inter);
#pragma unroll
    for (int j = 0; j < 2 * N; ++j) {
      float v = sum[e][j];
      for (int o = lanes; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (g == 0 && 2 * N * i < a.d) out[(j < N ? un.lo : un.hi - N) + j] = v;
    }
  }
}

// dgamma rows from the warps' partial rows, in a fixed order and fp64: 32 columns of
// one output row a CTA, warps over the partial rows. blockIdx.y: the output rows of q,
// then of k; a shared gamma's row sums the partial rows of all its heads.
__global__ void __launch_bounds__(1024) dgamma_kernel(const __grid_constant__ NormRopeArgs a,
                                                      int slots) {
  __shared__ double red[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const int q_rows = a.set[0].gamma == nullptr ? 0 : a.set[0].gheads;
  const int which = (int)blockIdx.y >= q_rows ? 1 : 0;
  const RowSet& rs = a.set[which];
  const int o = blockIdx.y - (which ? q_rows : 0);
  const int64_t nrows = (int64_t)slots * (rs.gheads > 1 ? 1 : rs.heads);
  const int64_t first = (which ? (int64_t)a.set[0].heads * slots : 0) + o * nrows;
  double s = 0.0;
  if (c < a.d) {
    const float* src = a.part + first * a.d + c;
    int64_t i = warp;
    for (; i + 7 * 32 < nrows; i += 8 * 32) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = src[(i + u * 32) * a.d];
#pragma unroll
      for (int u = 0; u < 8; ++u) s += v[u];
    }
    for (; i < nrows; i += 32) s += src[i * a.d];
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < a.d) {
    double r = 0.0;
    for (int w = 0; w < 32; ++w) r += red[w][lane];
    rs.dgamma[(int64_t)o * a.d + c] = (float)r;
    if (!isfinite(r)) report(a.dev_status, DARK_ERR_NUMERIC);
  }
}

// Four pairs a unit (8- or 16-byte accesses) need eight-element multiples and
// aligned rows; every other layout takes one pair a unit with scalar accesses.
bool vector_ok(const NormRopeArgs& a) {
  const size_t al = a.dtype == DARK_BF16 ? 8 : 16;
  auto ok = [&](const void* p, const int64_t* s) {
    return p == nullptr || ((uintptr_t)p % al == 0 && s[0] % 4 == 0 && s[1] % 4 == 0 && s[2] % 4 == 0);
  };
  if (a.d % 8 != 0 || a.rope.dims % 8 != 0) return false;
  for (int i = 0; i < 2; ++i) {
    const RowSet& s = a.set[i];
    if (!ok(s.x, s.xs) || !ok(s.y, s.ys) || !ok(s.g, s.gs)) return false;
    if ((uintptr_t)s.gamma % 16 != 0) return false;
  }
  return true;
}

int lanes_for(int d, int pairs) {
  int l = 1;
  while (l < 32 && l * 2 * pairs < d) l *= 2;
  return l;
}

template <typename T>
cudaError_t launch_rows(const NormRopeArgs& a) {
  const bool vec = vector_ok(a);
  const int lanes = lanes_for(a.d, vec ? 4 : 1), rows = 32 / lanes;
  const int nh = a.set[0].heads + a.set[1].heads;
  const int64_t ntok = (int64_t)a.B * a.L;
  // tiles of 32 tokens and all heads in a CTA; with too little work for two CTAs
  // an SM first smaller tiles, then fewer heads
  int tile = kTile, hchunk = nh;
  auto ctas = [&]() { return (ntok + tile - 1) / tile * ((nh + hchunk - 1) / hchunk); };
  while (tile > rows && ctas() < 2 * num_sms()) tile /= 2;
  while (hchunk > 1 && (int64_t)hchunk * tile > (int64_t)rows * kWarps && ctas() < 2 * num_sms())
    hchunk = (hchunk + 1) / 2;
  while ((nh + hchunk - 1) / hchunk > 65535) hchunk *= 2;
  const dim3 grid((unsigned)((ntok + tile - 1) / tile), (nh + hchunk - 1) / hchunk);
  const size_t smem = sizeof(Tile) + (size_t)tile * (a.rope.dims / 2) * sizeof(float2);
  if (vec)
    rows_kernel<T, 4, 1, 4><<<grid, kThreads, smem, a.stream>>>(a, lanes, tile, hchunk);
  else
    rows_kernel<T, 1, 4, 1><<<grid, kThreads, smem, a.stream>>>(a, lanes, tile, hchunk);
  return cudaGetLastError();
}

// CTAs along the tokens of the backward pass: at most four an SM over all head
// groups, and a tile each.
int bwd_ctas(int64_t ntok, int nh) {
  const int groups = (nh + kWarps - 1) / kWarps;
  const int64_t tiles = (ntok + kTile - 1) / kTile;
  const int64_t most = 592 / groups > 0 ? 592 / groups : 1;
  return (int)(tiles < most ? tiles : most);
}
int bwd_split(int nh) { return nh < kWarps ? kWarps / nh : 1; }

template <typename T>
cudaError_t launch_rows_bwd(const NormRopeArgs& a) {
  const bool vec = vector_ok(a);
  const int lanes = lanes_for(a.d, vec ? 4 : 1);
  const int nh = a.set[0].heads + a.set[1].heads;
  const int64_t ntok = (int64_t)a.B * a.L;
  const int ctas = bwd_ctas(ntok, nh);
  // even tiles: with few tokens every CTA gets some
  int64_t per = (ntok + ctas - 1) / ctas;
  const int tile = per < kTile ? (int)per : kTile;
  const dim3 grid(ctas, (nh + kWarps - 1) / kWarps);
  const size_t smem = sizeof(Tile) + (size_t)tile * (a.rope.dims / 2) * sizeof(float2);
  if (vec)
    rows_bwd_kernel<T, 4, 1><<<grid, kThreads, smem, a.stream>>>(a, lanes, tile);
  else
    rows_bwd_kernel<T, 1, 4><<<grid, kThreads, smem, a.stream>>>(a, lanes, tile);
  cudaError_t e = cudaGetLastError();
  const int out_rows = (a.set[0].gamma ? a.set[0].gheads : 0) + (a.set[1].gamma ? a.set[1].gheads : 0);
  if (e != cudaSuccess || out_rows == 0) return e;
  dgamma_kernel<<<dim3((a.d + 31) / 32, out_rows), 1024, 0, a.stream>>>(a, ctas * bwd_split(nh));
  return cudaGetLastError();
}

}  // namespace

size_t norm_rope_bwd_workspace_bytes(int B, int H, int Hk, int L, int d) {
  const int nh = H + Hk;
  return kWsHeader + align_up((size_t)nh * bwd_ctas((int64_t)B * L, nh) * bwd_split(nh) * d * 4, 256);
}

cudaError_t launch_norm_rope(const NormRopeArgs& a) {
  return a.dtype == DARK_BF16 ? launch_rows<__nv_bfloat16>(a) : launch_rows<float>(a);
}

cudaError_t launch_norm_rope_bwd(const NormRopeArgs& a) {
  return a.dtype == DARK_BF16 ? launch_rows_bwd<__nv_bfloat16>(a) : launch_rows_bwd<float>(a);
}

}  // namespace dark
