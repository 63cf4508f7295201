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
// Every kernel is bound by reading and writing its rows (2, 3 or 4 accesses of n
// elements). A lane group of 1-32 lanes holds a row in registers: one read, one shuffle
// reduction, one write.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace dark {
namespace {

constexpr int kMaxThreads = 256;                        // of the backward pass
constexpr int kRowWarps = 4;                            // of the forward pass

// A run of N elements of T as raw words, loaded and stored at once (2 to 16 bytes).
template <typename T, int N>
struct Run {
  static constexpr int kBytes = (int)sizeof(T) * N, kWords = kBytes < 4 ? 1 : kBytes / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* src) {
    if constexpr (kBytes == 16) {
      const uint4 x = *reinterpret_cast<const uint4*>(src);
      w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else if constexpr (kBytes == 8) {
      const uint2 x = *reinterpret_cast<const uint2*>(src);
      w[0] = x.x; w[1] = x.y;
    } else if constexpr (kBytes == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(src);
    } else {
      w[0] = *reinterpret_cast<const uint16_t*>(src);
    }
  }
  __device__ __forceinline__ void store(T* dst) const {
    if constexpr (kBytes == 16) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (kBytes == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else if constexpr (kBytes == 4) *reinterpret_cast<uint32_t*>(dst) = w[0];
    else *reinterpret_cast<uint16_t*>(dst) = (uint16_t)w[0];
  }
};

// A lane's own slot of shared memory: filled by an asynchronous copy (2-byte runs by a
// plain one), read back by the same lane once the copies' group has arrived.
template <typename T, int N>
__device__ __forceinline__ void fetch(uint32_t slot, const T* src, bool ok) {       // zeros if not
  constexpr int kBytes = Run<T, N>::kBytes;
  if constexpr (kBytes == 16) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(slot), "l"(src), "r"(ok ? 16 : 0)
                 : "memory");
  } else if constexpr (kBytes >= 4) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(slot), "l"(src), "n"(kBytes),
                 "r"(ok ? kBytes : 0)
                 : "memory");
  } else {
    const uint16_t v = ok ? *reinterpret_cast<const uint16_t*>(src) : (uint16_t)0;
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(slot), "h"(v) : "memory");
  }
}
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void fetch_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// The 2 N values of a unit as N pairs: N / 2 neighbours from each run, or one value of
// each run for N = 1.
template <typename T, int N>
__device__ __forceinline__ void widen(F2 (&v)[N], const Run<T, N>& lo, const Run<T, N>& hi) {
  constexpr bool bf = sizeof(T) == 2;
  auto low = [](uint32_t w) { return __uint_as_float(bf ? w << 16 : w); };
  if constexpr (N == 1) {
    v[0] = F2(low(lo.w[0]), low(hi.w[0]));
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      if constexpr (bf) {
        v[i] = F2(low(lo.w[i]), __uint_as_float(lo.w[i] & 0xffff0000u));
        v[N / 2 + i] = F2(low(hi.w[i]), __uint_as_float(hi.w[i] & 0xffff0000u));
      } else {
        v[i] = F2(low(lo.w[2 * i]), low(lo.w[2 * i + 1]));
        v[N / 2 + i] = F2(low(hi.w[2 * i]), low(hi.w[2 * i + 1]));
      }
    }
  }
}

// What narrow() has seen of its results: 0 while all are finite, NaN from the first that
// is not.
struct Seen {
  uint32_t h = 0;                         // two bf16
  F2 f = F2(0.f);
  __device__ __forceinline__ void add(float x) { f = fma2(F2(x, 0.f), F2(0.f), f); }
  __device__ __forceinline__ void add(F2 x) { f = fma2(x, F2(0.f), f); }
  __device__ __forceinline__ void add(uint32_t bf16x2) {
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(h) : "r"(bf16x2), "r"(0u));
  }
  __device__ __forceinline__ bool bad() const {
    return !(f.sum() == 0.f) || (h & 0x7fff7fffu) != 0;
  }
};

// Rounds a unit's values to T.
template <typename T, int N>
__device__ __forceinline__ void narrow(Run<T, N>& lo, Run<T, N>& hi, const F2 (&v)[N], Seen& seen) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 x = v[i].get();
      seen.add(v[i]);
      if constexpr (N == 1) {
        lo.w[0] = __float_as_uint(x.x);
        hi.w[0] = __float_as_uint(x.y);
      } else {
        Run<T, N>& r = i < N / 2 ? lo : hi;
        r.w[i % (N / 2) * 2] = __float_as_uint(x.x);
        r.w[i % (N / 2) * 2 + 1] = __float_as_uint(x.y);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 x = v[i].get();
      uint32_t w;
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(x.y), "f"(x.x));
      seen.add(w);
      if constexpr (N == 1) {
        lo.w[0] = w & 0xffffu;
        hi.w[0] = w >> 16;
      } else {
        (i < N / 2 ? lo : hi).w[i % (N / 2)] = w;
      }
    }
  }
}

// A unit's weights (fp32; 16-byte aligned runs where N is 4 or 8).
template <int N>
__device__ __forceinline__ void load_weights(F2 (&w)[N], const float* lo, const float* hi) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(lo) + i);
      const float4 b = __ldg(reinterpret_cast<const float4*>(hi) + i);
      w[2 * i] = F2(a.x, a.y);
      w[2 * i + 1] = F2(a.z, a.w);
      w[N / 2 + 2 * i] = F2(b.x, b.y);
      w[N / 2 + 2 * i + 1] = F2(b.z, b.w);
    }
  } else if constexpr (N == 2) {
    w[0] = F2(__ldg(lo), __ldg(lo + 1));
    w[1] = F2(__ldg(hi), __ldg(hi + 1));
  } else {
    w[0] = F2(__ldg(lo), __ldg(hi));
  }
}

// A lane's unit u of a row: N pairs (2 N elements) in two runs of N. Rotated units
// take the pairs [N u, N u + N); the units behind them 2 N elements in a row.
template <int N, bool INTER>
struct Unit {
  int lo, hi;                             // element offsets of the two runs
  bool turned;
  __device__ Unit(int u, int rot) {
    turned = u < rot / (2 * N);
    const bool split = turned && !INTER;
    lo = split ? N * u : 2 * N * u;
    hi = split ? rot / 2 + N * u : lo + N;
  }
};

// Cosines and sines of a unit's N pairs. turn rotates the unit's values by them.
template <int N>
struct Angles {
  float c[N], s[N];
};
template <int N, bool INTER>
__device__ __forceinline__ void turn(F2 (&v)[N], const Angles<N>& t) {
  if constexpr (INTER || N == 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 x = v[i].get();
      v[i] = F2(fmaf(x.x, t.c[i], -x.y * t.s[i]), fmaf(x.x, t.s[i], x.y * t.c[i]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      // (a, b) -> (a c - b s, b c + a s), the minus in one of the products' operands
      const F2 a = v[i], b = v[N / 2 + i], c(t.c[2 * i], t.c[2 * i + 1]), s(t.s[2 * i], t.s[2 * i + 1]);
      v[i] = fma2(mul2(b, s), F2(-1.f), mul2(a, c));
      v[N / 2 + i] = fma2(b, c, mul2(a, s));
    }
  }
}

__device__ __forceinline__ void angle(int64_t pos, uint64_t turns, float* c, float* s) {
  const uint64_t phase = (uint64_t)pos * turns;
  // [-2^31, 2^31) / 2^31 half turns
  sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, s, c);
}

// Forward and append. A warp takes 32 / lanes tokens and the heads [h0, h0 + hchunk) of
// both sets: a token's cosines and sines are computed once, into registers, and used for
// all its heads, whose rows stream through S slots of shared memory a lane. N pairs a unit,
// NU units a lane.
template <typename T, int N, int NU, int S, bool INTER, bool APPEND>
__global__ void __launch_bounds__(32 * kRowWarps) rows_kernel(const __grid_constant__ NormRopeArgs a,
                                                              int lanes, int hchunk) {
  using R = Run<T, N>;
  __shared__ __align__(16) uint8_t ring[kRowWarps][S][NU][2][32 * R::kBytes];
  __shared__ uint64_t turns[128];          // (lanes that index the parameters take turns)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane / lanes, lu = lane % lanes, rows = 32 / lanes;
  const uint32_t ntok = (uint32_t)a.B * a.L;
  const uint32_t n0 = (blockIdx.x * kRowWarps + warp) * rows, n = n0 + g;
  for (int i = threadIdx.x; i < a.rope.dims / 2; i += 32 * kRowWarps) turns[i] = a.rope.turns[i];
  __syncthreads();
  if (n0 >= ntok) return;
  bool live = n < ntok;
  const int b = live ? n / a.L : 0, l = live ? n - (uint32_t)b * a.L : 0;
  int64_t place = l, row = 0;              // row: of head 0 in the cache
  if constexpr (APPEND) {
    live = live && (a.new_lens == nullptr || l < a.new_lens[b]);
    const int have = live ? a.lens[b] : 0;
    place += have;
    if (live) {
      const int64_t pg = place / a.page;
      const int id = have >= 0 && pg < a.max_pages ? a.table[(int64_t)b * a.max_pages + pg] : -1;
      live = id >= 0 && id < a.pages;
      if (!live) report(a.dev_status, DARK_ERR_INVALID_ARG);
      row = (int64_t)id * a.set[0].heads * a.page + place % a.page;
    }
  }
  // producer: the next head to fetch, its row, and where the second set's rows begin
  const int heads0 = a.set[0].heads, first = (int)blockIdx.y * hchunk;
  const int last = min(first + hchunk, heads0 + a.set[1].heads);
  auto x_of = [&](int w, int h) {
    return (const T*)a.set[w].x + b * a.set[w].xs[0] + l * a.set[w].xs[2] + h * a.set[w].xs[1];
  };
  auto y_of = [&](int w, int h) {
    return APPEND ? (T*)a.set[w].y + (row + (int64_t)h * a.page) * a.d
                  : (T*)a.set[w].y + b * a.set[w].ys[0] + l * a.set[w].ys[2] + h * a.set[w].ys[1];
  };
  int w = first >= heads0 ? 1 : 0;
  int next = first;
  const T* x = x_of(w, first - (w ? heads0 : 0));
  int64_t xh = a.set[w].xs[1];
  bool has[NU];
  int lo_at[NU], hi_at[NU];
#pragma unroll
  for (int e = 0; e < NU; ++e) {
    const Unit<N, INTER> un(lu + e * lanes, a.rope.dims);
    has[e] = live && 2 * N * (lu + e * lanes) < a.d;
    lo_at[e] = un.lo;
    hi_at[e] = un.hi;
  }
  const uint32_t slots = (uint32_t)__cvta_generic_to_shared(&ring[warp][0][0][0][lane * R::kBytes]);
  constexpr uint32_t kRun = 32 * R::kBytes, kStage = NU * 2 * kRun;
  auto issue = [&](uint32_t slot) {
    if (next < last) {
#pragma unroll
      for (int e = 0; e < NU; ++e) {
        fetch<T, N>(slot + 2 * e * kRun, x + lo_at[e], has[e]);
        fetch<T, N>(slot + (2 * e + 1) * kRun, x + hi_at[e], has[e]);
      }
      x += xh;
      if (++next == heads0) {
        x = x_of(1, 0);
        xh = a.set[1].xs[1];
      }
    }
    fetch_commit();
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(slots + i * kStage);

  Angles<N> cs[NU];
  if (a.rope.dims > 0) {
    const int64_t pos = !live ? 0 : a.positions != nullptr ? (int64_t)a.positions[n] : a.pos0 + place;
#pragma unroll
    for (int e = 0; e < NU; ++e) {
      const int p0 = N * (lu + e * lanes);
      if (2 * p0 < a.rope.dims) {
#pragma unroll
        for (int j = 0; j < N; ++j) angle(pos, turns[p0 + j], &cs[e].c[j], &cs[e].s[j]);
      }
    }
  }
  Seen seen;
  const float inv_d = 1.f / (float)a.d;
  F2 gm[NU][N];
#pragma unroll
  for (int e = 0; e < NU; ++e)
#pragma unroll
    for (int i = 0; i < N; ++i) gm[e][i] = F2(0.f);
  uint32_t at = 0, fill = (S - 1) * kStage;                // bytes into the ring
  int hh = first;
#pragma unroll 1
  for (; w < 2; ++w) {                                     // (from here on: the consumer's set)
    const int base = w ? heads0 : 0, end = min(last, base + a.set[w].heads);
    if (hh >= end) continue;
    const bool normed = a.set[w].gamma != nullptr, each = a.set[w].gheads > 1;
    const bool rotate = a.set[w].rotate && a.rope.dims > 0;
    const float* gamma = a.set[w].gamma + (each ? (int64_t)(hh - base) * a.d : 0);
    T* y = y_of(w, hh - base);
    const int64_t yh = APPEND ? (int64_t)a.page * a.d : a.set[w].ys[1];
    bool fresh = normed;                                   // weights still to be loaded
#pragma unroll 1
    for (; hh < end; ++hh, y += yh) {
      fetch_wait<S - 2>();
      R lo[NU], hi[NU];
#pragma unroll
      for (int e = 0; e < NU; ++e) {
        const uint8_t* src = &ring[warp][0][0][0][lane * R::kBytes] + at + 2 * e * kRun;
        lo[e].load(reinterpret_cast<const T*>(src));
        hi[e].load(reinterpret_cast<const T*>(src + kRun));
      }
      issue(slots + fill);                                 // the slot read last time round
      fill = at;
      at = at + kStage == S * kStage ? 0 : at + kStage;
      if (normed || rotate) {                              // a plain copy keeps the bits
        F2 v[NU][N], s2(0.f);
#pragma unroll
        for (int e = 0; e < NU; ++e) widen<T, N>(v[e], lo[e], hi[e]);
        if (normed) {
          if (fresh) {
#pragma unroll
            for (int e = 0; e < NU; ++e)
              if (has[e]) load_weights<N>(gm[e], gamma + lo_at[e], gamma + hi_at[e]);
            gamma += a.d;
            fresh = each;
          }
#pragma unroll
          for (int e = 0; e < NU; ++e)
#pragma unroll
            for (int i = 0; i < N; ++i) s2 = fma2(v[e][i], v[e][i], s2);
          float ss = s2.sum();
          for (int o = lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          seen.add(ss);                                    // a sum of squares past fp32
          const F2 rstd(rsqrtf(fmaf(ss, inv_d, a.eps)));
#pragma unroll
          for (int e = 0; e < NU; ++e)
#pragma unroll
            for (int i = 0; i < N; ++i) v[e][i] = mul2(v[e][i], mul2(rstd, gm[e][i]));
        }
#pragma unroll
        for (int e = 0; e < NU; ++e) {
          if (rotate && 2 * N * (lu + e * lanes) < a.rope.dims) turn<N, INTER>(v[e], cs[e]);
          narrow<T, N>(lo[e], hi[e], v[e], seen);
        }
      }
#pragma unroll
      for (int e = 0; e < NU; ++e)
        if (has[e]) {
          lo[e].store(y + lo_at[e]);
          hi[e].store(y + hi_at[e]);
        }
    }
  }
  if (seen.bad()) report(a.dev_status, DARK_ERR_NUMERIC);
}

// Partial rows of dgamma: for a shared weight one of every CTA that holds heads of the set
// (head groups `group`, `group` + 1, ...), else `ctas * split` of every head.
struct PartRows {
  int64_t first;                          // of the set
  int rows, group;                        // rows of one output row; the set's first head group
};
// Warps of a CTA: eight, or for more heads the count from five up that leaves the fewest of
// the groups' warps without a head.
__host__ __device__ inline int bwd_warps(int nh) {
  int best = 8;
  for (int w = 7; w >= 5 && nh > 8; --w)
    if ((nh + w - 1) / w * w < (nh + best - 1) / best * best) best = w;
  return best;
}
__host__ __device__ inline int head_split(int nh) { return nh < 8 ? 8 / nh : 1; }
__device__ __forceinline__ PartRows part_rows(const NormRopeArgs& a, int set, int ctas) {
  const int h0 = a.set[0].heads, nh = h0 + a.set[1].heads;
  const int lo = set ? h0 : 0, hi = set ? nh : h0;
  PartRows p;
  p.first = set ? (int64_t)h0 * ctas * head_split(nh) : 0;
  const int w = bwd_warps(nh);
  p.group = lo / w;
  p.rows = a.set[set].gheads > 1 ? ctas * head_split(nh) : ((hi - 1) / w - p.group + 1) * ctas;
  return p;
}

// Backward. blockIdx.y is a group of as many heads as the CTA has warps, a warp keeps one
// head (with fewer heads, several warps share one and split its tokens) and its weights and dgamma
// in registers. A CTA walks its `span` tokens; the rows of its warps stream through S slots
// of shared memory a lane, and the cosines and sines of `tile` tokens at a time lie in
// shared memory for all its heads: pairs 2 j, 2 j + 1 of unit u of token k as one float4
// (two cosines, two sines) at (j tile + k) units + u, so that the lanes of a warp read
// consecutive 16-byte words. Each warp leaves one row of sums for the reduction below.
template <typename T, int N, int NU, int S, bool INTER>
__global__ void __launch_bounds__(kMaxThreads, 2) rows_bwd_kernel(const __grid_constant__ NormRopeArgs a,
                                                               int lanes, int span, int tile) {
  using R = Run<T, N>;
  constexpr int NC = N > 1 ? N / 2 : 1, PC = N > 1 ? 2 : 1;
  constexpr uint32_t kRun = 32 * R::kBytes, kStage = NU * 4 * kRun;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t turns[128];
  const int nw = blockDim.x / 32;
  float* cs = reinterpret_cast<float*>(smem + nw * S * kStage);
  pdl_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = 32 / lanes, g = lane / lanes, lu = lane % lanes;
  const int np = a.rope.dims / 2, units = np / N;
  const int nh = a.set[0].heads + a.set[1].heads;
  const int hg = nh < nw ? nh : nw, split = nw / hg;
  const int hh = blockIdx.y * nw + warp % hg, part = warp / hg;
  const bool on = hh < nh && part < split;
  const int which = hh >= a.set[0].heads ? 1 : 0;
  const RowSet& rs = a.set[which];
  const int h = hh - (which ? a.set[0].heads : 0);
  const int rot = a.rope.dims;
  const bool normed = rs.gamma != nullptr;
  const T* xh = (const T*)rs.x + (int64_t)h * rs.xs[1];
  const T* gh = (const T*)rs.g + (int64_t)h * rs.gs[1];
  T* yh = (T*)rs.y + (int64_t)h * rs.ys[1];
  const uint32_t ntok = (uint32_t)a.B * a.L, t0 = blockIdx.x * span;
  const int count = t0 < ntok ? (int)min((uint32_t)span, ntok - t0) : 0;
  bool has[NU];
#pragma unroll
  for (int e = 0; e < NU; ++e) has[e] = 2 * N * (lu + e * lanes) < a.d;

  int lo_at[NU], hi_at[NU];
#pragma unroll
  for (int e = 0; e < NU; ++e) {
    const Unit<N, INTER> un(lu + e * lanes, rot);
    lo_at[e] = un.lo;
    hi_at[e] = un.hi;
  }
  uint8_t* ring = smem + warp * S * kStage + lane * R::kBytes;
  const uint32_t slots = (uint32_t)__cvta_generic_to_shared(ring);
  const int step = split * rows, mine = part * rows + g;   // tokens mine, mine + step, ...
  // rows of the next token to fetch, moved on by `step` tokens at a time
  int next = mine, next_l = 0;
  const T *xr = nullptr, *gr = nullptr;
  auto seek = [&]() {
    const uint32_t n = t0 + next, b = n / a.L;
    next_l = n - b * a.L;
    xr = xh + (int64_t)b * rs.xs[0] + next_l * rs.xs[2];
    gr = gh + (int64_t)b * rs.gs[0] + next_l * rs.gs[2];
  };
  seek();
  const int64_t x_step = step * rs.xs[2], g_step = step * rs.gs[2], y_step = step * rs.ys[2];
  auto issue = [&](uint32_t slot) {
    const bool ok = on && next < count;
#pragma unroll
    for (int e = 0; e < NU; ++e) {
      const uint32_t to = slot + 4 * e * kRun;
      fetch<T, N>(to, xr + lo_at[e], ok && has[e] && normed);
      fetch<T, N>(to + kRun, xr + hi_at[e], ok && has[e] && normed);
      fetch<T, N>(to + 2 * kRun, gr + lo_at[e], ok && has[e]);
      fetch<T, N>(to + 3 * kRun, gr + hi_at[e], ok && has[e]);
    }
    fetch_commit();
    next += step;
    next_l += step;
    xr += x_step;
    gr += g_step;
    if (next_l >= a.L) seek();
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(slots + i * kStage);

  F2 acc[NU][N], gm[NU][N];
#pragma unroll
  for (int e = 0; e < NU; ++e) {
#pragma unroll
    for (int j = 0; j < N; ++j) acc[e][j] = gm[e][j] = F2(0.f);
    if (on && normed && has[e]) {
      const float* src = rs.gamma + (rs.gheads > 1 ? (int64_t)h * a.d : 0);
      load_weights<N>(gm[e], src + lo_at[e], src + hi_at[e]);
    }
  }
  if (threadIdx.x < np) turns[threadIdx.x] = a.rope.turns[threadIdx.x];
  Seen seen;
  const float inv_d = 1.f / (float)a.d;
  uint32_t from = 0, fill = (S - 1) * kStage;        // bytes into the ring
  int k = mine;                                      // this lane group's next token
  int at_l = a.L;                                    // its row of results (found when needed)
  T* dst = nullptr;
  for (int tile0 = 0; tile0 < count; tile0 += tile) {
    const int here = min(tile, count - tile0);
    __syncthreads();                                 // turns; the last tile's readers are done
    for (int kk = warp; kk < here; kk += nw) {
      const uint32_t n = t0 + tile0 + kk;
      const int64_t pos = a.positions != nullptr ? (int64_t)a.positions[n] : a.pos0 + n % a.L;
      for (int p = lane; p < np; p += 32) {
        const int u = p / N, j = p % N / PC;
        float* to = cs + ((j * tile + kk) * units + u) * 2 * PC + p % PC;
        angle(pos, turns[p], to, to + PC);
      }
    }
    __syncthreads();
    if (!on) continue;
    // a warp's groups are `rows` apart at most and tiles are multiples of `step`: all leave
    // the loop together
#pragma unroll 1
    for (; k - g < tile0 + here; k += step) {
      fetch_wait<S - 2>();
      const bool live = k < count;
      R lo[NU], hi[NU];
      F2 x[NU][N], w[NU][N], ss2(0.f), dot2(0.f);
#pragma unroll
      for (int e = 0; e < NU; ++e) {
        const uint8_t* src = ring + from + 4 * e * kRun;
        lo[e].load(reinterpret_cast<const T*>(src));
        hi[e].load(reinterpret_cast<const T*>(src + kRun));
        widen<T, N>(x[e], lo[e], hi[e]);
        lo[e].load(reinterpret_cast<const T*>(src + 2 * kRun));
        hi[e].load(reinterpret_cast<const T*>(src + 3 * kRun));
        widen<T, N>(w[e], lo[e], hi[e]);
      }
      issue(slots + fill);                           // the slot read last time round
      fill = from;
      from = from + kStage == S * kStage ? 0 : from + kStage;
#pragma unroll
      for (int e = 0; e < NU; ++e) {
        const int i = lu + e * lanes;
        if (live && 2 * N * i < rot) {               // w = u, the cotangent turned back
          Angles<N> t;
#pragma unroll
          for (int j = 0; j < NC; ++j) {
            const float* src = cs + ((j * tile + k - tile0) * units + i) * 2 * PC;
            if constexpr (N > 1) {
              const float4 v = *reinterpret_cast<const float4*>(src);
              t.c[2 * j] = v.x;
              t.c[2 * j + 1] = v.y;
              t.s[2 * j] = -v.z;
              t.s[2 * j + 1] = -v.w;
            } else {
              t.c[0] = src[0];
              t.s[0] = -src[1];
            }
          }
          turn<N, INTER>(w[e], t);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
          ss2 = fma2(x[e][j], x[e][j], ss2);
          dot2 = fma2(mul2(w[e][j], gm[e][j]), x[e][j], dot2);
        }
      }
      if (normed) {
        float ss = ss2.sum(), dot = dot2.sum();
        for (int o = lanes >> 1; o > 0; o >>= 1) {
          ss += __shfl_xor_sync(0xffffffffu, ss, o);
          dot += __shfl_xor_sync(0xffffffffu, dot, o);
        }
        seen.add(ss);
        const float r = rsqrtf(fmaf(ss, inv_d, a.eps));
        const F2 rstd(r), back(-dot * inv_d * r * r * r);        // -mean(w n) rstd^2
#pragma unroll
        for (int e = 0; e < NU; ++e)
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const F2 wr = mul2(w[e][j], rstd);
            acc[e][j] = fma2(wr, x[e][j], acc[e][j]);
            w[e][j] = fma2(wr, gm[e][j], mul2(x[e][j], back));
          }
      }
      if (at_l >= a.L) {
        const uint32_t n = t0 + k, b = n / a.L;
        at_l = n - b * a.L;
        dst = yh + (int64_t)b * rs.ys[0] + at_l * rs.ys[2];
      }
#pragma unroll
      for (int e = 0; e < NU; ++e) {
        narrow<T, N>(lo[e], hi[e], w[e], seen);
        if (live && has[e]) {
          lo[e].store(dst + lo_at[e]);
          hi[e].store(dst + hi_at[e]);
        }
      }
      dst += y_step;
      at_l += step;
    }
  }
  fetch_wait<0>();
  if (seen.bad()) report(a.dev_status, DARK_ERR_NUMERIC);
  // the warps' rows of sums in shared memory (in the place of the rings and angles)
  __syncthreads();
  float* sums = reinterpret_cast<float*>(smem);      // [warp][d]
#pragma unroll
  for (int e = 0; e < NU; ++e)
#pragma unroll
    for (int j = 0; j < 2 * N; ++j) {
      const int i = N == 1 ? 0 : j / 2;              // value j of (lo run, hi run)
      float v = j % 2 == 0 ? acc[e][i].get().x : acc[e][i].get().y;
      for (int o = lanes; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (g == 0 && has[e]) sums[warp * a.d + (j < N ? lo_at[e] : hi_at[e] - N) + j] = v;
    }
  __syncthreads();
  // one partial row for every set with a shared weight, or one for every head
  for (int c = threadIdx.x; c < a.d; c += blockDim.x)
    for (int s = 0; s < 2; ++s) {
      const RowSet& r = a.set[s];
      if (r.gamma == nullptr) continue;
      const PartRows pr = part_rows(a, s, gridDim.x);
      const int base = s ? a.set[0].heads : 0;
      float v = 0.f;
      bool any = false;
      for (int i = 0; i < nw; ++i) {
        const int hi = blockIdx.y * nw + i % hg, p = i / hg;
        if (hi >= nh || p >= split || hi < base || hi >= base + r.heads) continue;
        any = true;
        v += sums[i * a.d + c];
        if (r.gheads > 1) {
          a.part[(pr.first + ((int64_t)(hi - base) * gridDim.x + blockIdx.x) * split + p) * a.d + c] = v;
          v = 0.f;
        }
      }
      if (any && r.gheads == 1)
        a.part[(pr.first + (int64_t)(blockIdx.y - pr.group) * gridDim.x + blockIdx.x) * a.d + c] = v;
    }
}

// dgamma rows from the partial rows, in a fixed order and fp64: 32 columns of one output
// row a CTA, warps over the partial rows. blockIdx.y: the output rows of q, then of k.
__global__ void __launch_bounds__(512) dgamma_kernel(const __grid_constant__ NormRopeArgs a, int ctas) {
  constexpr int kW = 16;
  __shared__ double red[kW][33];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const int q_rows = a.set[0].gamma == nullptr ? 0 : a.set[0].gheads;
  const int which = (int)blockIdx.y >= q_rows ? 1 : 0;
  const RowSet& rs = a.set[which];
  const int o = blockIdx.y - (which ? q_rows : 0);
  const PartRows pr = part_rows(a, which, ctas);
  double s = 0.0;
  if (c < a.d) {
    const float* src = a.part + (pr.first + (int64_t)o * pr.rows) * a.d + c;
    int i = warp;
    for (; i + 7 * kW < pr.rows; i += 8 * kW) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = src[(int64_t)(i + u * kW) * a.d];
#pragma unroll
      for (int u = 0; u < 8; ++u) s += v[u];
    }
    for (; i < pr.rows; i += kW) s += src[(int64_t)i * a.d];
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < a.d) {
    double r = 0.0;
    for (int w = 0; w < kW; ++w) r += red[w][lane];
    rs.dgamma[(int64_t)o * a.d + c] = (float)r;
    if (!isfinite(r)) report(a.dev_status, DARK_ERR_NUMERIC);
  }
}

// Pairs of a unit: the largest run whose accesses (up to 16 bytes) all rows, strides and
// weights are aligned for. Narrower units hold their rows in several units a lane.
int pairs_for(const NormRopeArgs& a) {
  const size_t e = a.dtype == DARK_BF16 ? 2 : 4;
  auto fits = [&](int n) {
    if (a.d % (2 * n) != 0 || a.rope.dims % (2 * n) != 0) return false;
    auto ok = [&](const void* p, const int64_t* s) {
      return p == nullptr || ((uintptr_t)p % (n * e) == 0 && s[0] % n == 0 && s[1] % n == 0 &&
                              s[2] % n == 0);
    };
    for (int i = 0; i < 2; ++i) {
      const RowSet& s = a.set[i];
      if (!ok(s.x, s.xs) || !ok(s.y, s.ys) || !ok(s.g, s.gs)) return false;
      if (n >= 4 && (uintptr_t)s.gamma % 16 != 0) return false;
    }
    return true;
  };
  if (a.dtype == DARK_BF16 && fits(8)) return 8;
  return fits(4) ? 4 : fits(2) ? 2 : 1;
}

int lanes_for(int d, int pairs) {
  int l = 1;
  while (l < 32 && l * 2 * pairs < d) l *= 2;
  return l;
}

// Units a lane needs for d = 256 in 32 lanes.
constexpr int units_of(int n) { return n >= 4 ? 1 : 4 / n; }

template <typename T, int N, bool INTER>
cudaError_t launch_rows(const NormRopeArgs& a) {
  constexpr int NU = units_of(N), S = NU == 1 ? 6 : 3;
  const int lanes = lanes_for(a.d, N), rows = 32 / lanes;
  const int nh = a.set[0].heads + a.set[1].heads;
  const int64_t groups = ((int64_t)a.B * a.L + rows - 1) / rows;
  const int64_t x = (groups + kRowWarps - 1) / kRowWarps;
  // all heads of a token in one warp (its angles are computed once), unless that leaves SMs
  // without two CTAs: 64 tokens of 40 heads, d = 128, 3.5 us cut and 15.6 whole, 2048 tokens of
  // 16 heads, d = 64, 4.7 and 7.8; a head a warp takes 41 us instead of 16.5 at 8192 tokens of 20
  int hchunk = nh;
  while (hchunk > 1 && x * ((nh + hchunk - 1) / hchunk) < 2 * num_sms()) hchunk = (hchunk + 1) / 2;
  while ((nh + hchunk - 1) / hchunk > 65535) hchunk *= 2;
  const dim3 grid((unsigned)x, (nh + hchunk - 1) / hchunk);
  if (a.lens != nullptr)
    rows_kernel<T, N, NU, S, INTER, true><<<grid, 32 * kRowWarps, 0, a.stream>>>(a, lanes, hchunk);
  else
    rows_kernel<T, N, NU, S, INTER, false><<<grid, 32 * kRowWarps, 0, a.stream>>>(a, lanes, hchunk);
  return cudaGetLastError();
}

// CTAs along the tokens of the backward pass: as many over all head groups as run at once
// (16 warps an SM by their registers), and 16 tokens each at least. The workspace follows
// them, so that they are counted for the B200's 148 SMs.
int bwd_ctas(int64_t ntok, int nh) {
  const int w = bwd_warps(nh), groups = (nh + w - 1) / w, most = 148 * (16 / w) / groups;
  const int64_t least = (ntok + 15) / 16;
  return (int)(least < most ? least : most > 1 ? most : 1);
}

template <typename T, int N, bool INTER>
cudaError_t launch_rows_bwd(const NormRopeArgs& a) {
  constexpr int NU = units_of(N), S = NU == 1 ? 4 : 3;
  static int smem_set[64];
  const int lanes = lanes_for(a.d, N);
  const int nh = a.set[0].heads + a.set[1].heads, np = a.rope.dims / 2;
  const int64_t ntok = (int64_t)a.B * a.L;
  const int ctas = bwd_ctas(ntok, nh), step = 32 / lanes * head_split(nh);
  const int span = (int)((ntok + ctas - 1) / ctas);
  // angles of at most 48 KB at a time; tiles a multiple of the tokens of one step
  const int most = (np == 0 ? span : 6144 / np) / step * step, nw = bwd_warps(nh);
  const int tile = most < step ? step : most < span ? most : (span + step - 1) / step * step;
  const size_t ring = (size_t)nw * S * NU * 4 * 32 * N * sizeof(T);
  const size_t smem = ring + (size_t)tile * a.rope.dims * sizeof(float);
  auto* kernel = rows_bwd_kernel<T, N, NU, S, INTER>;
  cudaError_t e = set_smem_limit_once((const void*)kernel, (int)(ring + 49152), smem_set);
  if (e != cudaSuccess) return e;
  const dim3 grid(ctas, (nh + nw - 1) / nw);
  kernel<<<grid, 32 * nw, smem, a.stream>>>(a, lanes, span, tile);
  e = cudaGetLastError();
  const int out_rows = (a.set[0].gamma ? a.set[0].gheads : 0) + (a.set[1].gamma ? a.set[1].gheads : 0);
  if (e != cudaSuccess || out_rows == 0) return e;
  return launch_dependent(dgamma_kernel, dim3((a.d + 31) / 32, out_rows), dim3(512), 0, a.stream, a, ctas);
}

// The instance for a call's type, unit width and pair layout.
// (The backward pass holds four rows' worth of a unit in registers: units of four pairs at
// most, 77 us against 88 with eight at 16384 tokens of 20 heads, d = 128, bf16.)
template <typename T, int N>
cudaError_t launch_n(const NormRopeArgs& a, bool bwd) {
  constexpr int NB = N > 4 ? 4 : N;
  if (a.rope.interleaved) return bwd ? launch_rows_bwd<T, NB, true>(a) : launch_rows<T, N, true>(a);
  return bwd ? launch_rows_bwd<T, NB, false>(a) : launch_rows<T, N, false>(a);
}
cudaError_t launch(const NormRopeArgs& a, bool bwd) {
  const int n = pairs_for(a);
  if (a.dtype == DARK_BF16)
    return n == 8   ? launch_n<__nv_bfloat16, 8>(a, bwd)
           : n == 4 ? launch_n<__nv_bfloat16, 4>(a, bwd)
           : n == 2 ? launch_n<__nv_bfloat16, 2>(a, bwd)
                    : launch_n<__nv_bfloat16, 1>(a, bwd);
  return n == 4 ? launch_n<float, 4>(a, bwd)
         : n == 2 ? launch_n<float, 2>(a, bwd)
                  : launch_n<float, 1>(a, bwd);
}

}  // namespace

size_t norm_rope_bwd_workspace_bytes(int B, int H, int Hk, int L, int d) {
  const int nh = H + Hk;
  return kWsHeader + align_up((size_t)nh * bwd_ctas((int64_t)B * L, nh) * head_split(nh) * d * 4, 256);
}

cudaError_t launch_norm_rope(const NormRopeArgs& a) { return launch(a, false); }
cudaError_t launch_norm_rope_bwd(const NormRopeArgs& a) { return launch(a, true); }

}  // namespace dark
