// Cache attention, key ranges on the tensor cores for few rows (bf16).
//
// A CTA takes one key range and a block of rows, in one of two ways:
//  * few rows (a sequence's own keys; a prefix with up to 16 rows): every warp streams its
//    own tiles of 16 keys (tiles w, w + warps, ...) through a private ring in shared
//    memory (cp.async, 16 bytes a lane, no barrier between warps) for the same 8 or 16 rows,
//    and keeps its own reference exponents, weights and sums, joined once at the end;
//  * a prefix with more rows: all warps share each tile of keys, brought by all of them, and
//    take 8 or 16 rows each, so that the keys are read once for all rows of the block.
//
// mma.sync m16n8k16 has 16 rows. Eight queries fill it twice, as y = hi + lo: rows 0-7 hold
// hi, rows 8-15 lo, and a thread's accumulators of rows g and g + 8 add up to the score; the
// weights P = hi + lo go the same way, so that both products keep 16 bits of significand at
// the price of one product with 16 rows. With more rows, up to d = 128, the tile holds 16
// queries, hi and lo in two products, and weights rounded to bf16 (8-row tiles cost a
// quarter more at 16 rows). A row's reference exponent only moves when a score passes it by 2^8 (sums and
// weights stay far inside fp32), so that sums are rescaled a few times a range.
//
// Bound by the key and value rows (read once for all rows of the block): 4 d bytes a key;
// for short ranges by the latency of their first copies (length, page number, rows).
#include <math.h>

#include "cache_attend_mma.cuh"
#include "tc_common.cuh"

namespace dark {
namespace cache {
namespace {

constexpr int kKeys = 16;                                 // keys of a tile


__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float bf16_half(uint32_t w, int upper) {
  return __uint_as_float(upper ? w & 0xffff0000u : w << 16);
}
// Whether a tile of kKeys rows holds an infinity or NaN (the same answer in all lanes).
template <int DP>
__device__ __forceinline__ bool tile_non_finite(uint32_t tile, int lane) {
  bool bad = false;
  for (int n = lane; n < kKeys * DP / 8; n += 32) {
    const uint4 w = tc::ld_shared_v4(tile + 16 * n);
    for (uint32_t x : {w.x, w.y, w.z, w.w})
      bad |= (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
  }
  return __any_sync(0xffffffffu, bad);
}

// Shared memory of a CTA: rings of `kStages` tiles for each of W warps, or one for all.
// Small rings, so that several CTAs share an SM and one's first copies run under another's
// products (32-key tiles in twice the memory: 19.9 against 17.5 us at 64 sequences of up to
// 1024 keys, d = 64; three stages: 29 against 26 us at 512 keys, d = 128).
template <int DP, bool SHARE>
struct Cfg {
  static constexpr uint32_t kTile = kKeys * DP * 2;       // one matrix of a tile
  static constexpr int W = SHARE || DP == 64 ? 4 : 2;
  static constexpr int kStages = SHARE ? 6 : DP == 64 ? 3 : 2;
  static constexpr uint32_t kRing = kStages * 2 * kTile;
  static constexpr uint32_t kSmem = SHARE ? kRing : W * kRing;
  static_assert(SHARE || kSmem >= W * 16 * (DP + 8 + 2) * 4, "the join's sums");
};

// HL: 8 rows a warp as hi + lo, else 16 rows. SHARE: the warps take different rows.
template <int DP, bool HL, bool SHARE>
__global__ void __launch_bounds__(Cfg<DP, SHARE>::W * 32) range_mma_kernel(const __grid_constant__ Params q) {
  using C = Cfg<DP, SHARE>;
  constexpr int NS = DP / 16, NT = DP / 8;                // k-steps of a score, column tiles
  constexpr int NR = HL ? 1 : 2;                          // rows a thread
  constexpr int W = C::W, RB = 8 * NR * (SHARE ? W : 1), S = C::kStages;
  const int hk = blockIdx.y;
  // The queries and the list of ranges come from an earlier launch. Where the prefix's launch lies
  // in between, this waits for that one too (which had waited for the queries'): only the wait
  // makes results visible, although the own ranges need nothing of the prefix's.
  pdl_wait();
  pdl_launch();
  const Item it = item_of(q, blockIdx.x, hk, RB, SHARE || (q.a.prefix_len > 0 && !q.p.tc && !q.p.share), !SHARE);
  if (!it.any) return;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int r0 = SHARE ? warp * 8 * NR : 0;               // this warp's first row of the block
  const uint32_t ring0 = tc::smem_u32(smem) + (SHARE ? 0 : warp * C::kRing);
  const int d = q.a.d, chunks = d / 8;
  const __nv_bfloat16* kp = (const __nv_bfloat16*)q.a.kp;
  const __nv_bfloat16* vp = (const __nv_bfloat16*)q.a.vp;

  // Where tile i's keys lie: the page (its number is loaded a tile ahead of its use) and row
  // in it of one key a lane (lanes 0-15), or, where no tile reaches over a page's end and rows
  // are not padded, of the tile's first key: then the tile is one run of memory.
  const bool flat = q.a.page % kKeys == 0 && d == DP;
  const int ntiles = (it.k1 - it.k0 + kKeys - 1) / kKeys;
  const int mine = SHARE ? ntiles : ntiles > warp ? (ntiles - warp + W - 1) / W : 0;
  auto first_key = [&](int i) { return it.k0 + (SHARE ? i : warp + i * W) * kKeys; };
  struct Spot {
    int id, in;                                           // in < 0: no key
  };
  auto lookup = [&](int i) {
    const int key = first_key(i) + (flat ? 0 : lane & 15);
    Spot s{0, -1};
    if (i < mine && key < it.k1) {
      const int pg = key / q.a.page;
      s.in = key - pg * q.a.page;
      s.id = __ldcg(it.pages + pg);
    }
    return s;
  };
  auto issue = [&](int i, Spot s) {                       // zeros past the range and past d
    const uint32_t k0 = ring0 + (uint32_t)(i % S) * 2 * C::kTile, v0 = k0 + C::kTile;
    constexpr int CH = DP / 8, T = SHARE ? W * 32 : 32;
    const int me = SHARE ? tid : lane;
    int64_t row = -1;
    if (s.in >= 0) {
      if (s.id >= 0 && s.id < q.a.pages)
        row = ((int64_t)s.id * q.a.Hk + hk) * q.a.page + s.in;
      else
        report(q.a.dev_status, DARK_ERR_INVALID_ARG);
    }
    if (flat) {
      const int live = row < 0 ? 0 : min(kKeys, it.k1 - first_key(i)) * CH;      // 16-byte pieces
      const int64_t o = row < 0 ? 0 : row * DP + me * 8;
#pragma unroll
      for (int n = 0; n < kKeys * CH / T; ++n) {
        const int idx = n * T + me;
        const bool ok = idx < live;
        const uint32_t to = tile_off<DP>(idx / CH, idx % CH);
        const int64_t from = ok ? o + n * T * 8 : 0;
        cp16(k0 + to, kp + from, ok);
        cp16(v0 + to, vp + from, ok);
      }
    } else {
#pragma unroll
      for (int n = 0; n < kKeys * CH / T; ++n) {
        const int idx = n * T + me, r = idx / CH, c = idx % CH;
        const int64_t at = __shfl_sync(0xffffffffu, row, r);
        const bool ok = at >= 0 && c < chunks;
        const int64_t o = ok ? at * d + c * 8 : 0;
        cp16(k0 + tile_off<DP>(r, c), kp + o, ok);
        cp16(v0 + tile_off<DP>(r, c), vp + o, ok);
      }
    }
  };
  Spot next = lookup(S - 1);
  {
    Spot s[S - 1];
#pragma unroll
    for (int i = 0; i < S - 1; ++i) s[i] = lookup(i);
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
      if (i < mine) issue(i, s[i]);
      cp_commit();
    }
  }

  // the rows' queries as A fragments: hi in rows 0-7 and lo in rows 8-15, or rows 0-15 of
  // hi, then of lo
  constexpr int NH = HL ? 1 : 2;
  uint32_t ya[NH][NS][4];
  int lim[NR], seen_by_all = it.k1;
  {
    const __nv_bfloat16* y = at<__nv_bfloat16>(q.a, q.p.o_y);
    const int64_t lo = (int64_t)q.a.Hk * q.p.all * DP;
    const __nv_bfloat16* src[2];
    bool ok[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = r0 + g + (HL ? 0 : 8 * h);
      ok[h] = row < it.nrows;
      src[h] = y + ((int64_t)hk * q.p.all + it.row0 + (ok[h] ? row : 0)) * DP + 2 * t + (HL && h ? lo : 0);
      if (h < NR) {
        lim[h] = ok[h] ? visible_keys(q, it, row) : 0;
        if (ok[h]) seen_by_all = min(seen_by_all, lim[h]);
      }
    }
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          ya[h][s][e] = ok[e & 1] ? __ldcg(reinterpret_cast<const uint32_t*>(src[e & 1] + h * lo + 16 * s + 8 * (e >> 1)))
                                  : 0u;
    for (int o = 4; o < 32; o <<= 1)
      seen_by_all = min(seen_by_all, __shfl_xor_sync(0xffffffffu, seen_by_all, o));
  }
  float o[NT][4], l[NR], ref[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    l[r] = 0.f;
    ref[r] = -INFINITY;
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[n][e] = 0.f;

  const int lr = lane & 7, lg = lane >> 3;                // ldmatrix: row in, and number of, a matrix
  for (int i = 0; i < mine; ++i) {
    cp_wait<S - 2>();
    if (SHARE) __syncthreads(); else __syncwarp();        // (the slot of tile i - 1 is free too)
    {
      const Spot s = next;
      next = lookup(i + S);
      if (i + S - 1 < mine) issue(i + S - 1, s);
      cp_commit();
    }
    const uint32_t k0 = ring0 + (uint32_t)(i % S) * 2 * C::kTile, v0 = k0 + C::kTile;
    float s[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
    for (int st = 0; st < NS; ++st) {
      uint32_t b[4];
      ldsm4(b, k0 + tile_off<DP>((lg >> 1) * 8 + lr, 2 * st + (lg & 1)));
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        mma16816_bf16(s[0], ya[h][st], b[0], b[1]);
        mma16816_bf16(s[1], ya[h][st], b[2], b[3]);
      }
    }
    const int tile0 = first_key(i), key0 = tile0 + 2 * t;
    uint32_t pa[4];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float v[4];                                         // keys key0 + {0, 1, 8, 9} of row g + 8 r
      const int end = min(it.k1, lim[r]);
      float top = -INFINITY;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = HL ? s[e >> 1][e & 1] + s[e >> 1][2 + (e & 1)] : s[e >> 1][2 * r + (e & 1)];
        v[e] = key0 + (e >> 1) * 8 + (e & 1) < end ? x : -INFINITY;
        top = fmaxf(top, v[e]);
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const bool move = top > ref[r] + 8.f;               // (-inf + 8 = -inf: the first visible key)
      if (__any_sync(0xffffffffu, move)) {
        const float now = move ? top : ref[r], f = move ? exp2f(ref[r] - now) : 1.f;
        ref[r] = now;
        l[r] *= f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          o[n][2 * r] *= f;
          o[n][2 * r + 1] *= f;
          if (HL) {
            o[n][2] *= f;
            o[n][3] *= f;
          }
        }
      }
      const float m = ref[r] == -INFINITY ? 0.f : ref[r];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = tc::ex2(v[e] - m);
        l[r] += v[e];
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {                       // operand registers: rows g, g + 8 by keys 0, 8
        uint32_t& first = pa[2 * n + r];
        first = tc::pack_bf16(v[2 * n], v[2 * n + 1]);
        if (HL) pa[2 * n + 1] = tc::pack_bf16(v[2 * n] - bf16_half(first, 0), v[2 * n + 1] - bf16_half(first, 1));
      }
    }
    // A weight of 0 does not cancel an infinite or NaN value of a key that only other rows
    // see (causal, the last T - 1 keys): a tile with one adds its values key by key.
    if (tile0 + kKeys > seen_by_all && tile_non_finite<DP>(v0, lane)) {
#pragma unroll 1
      for (int kk = 0; kk < kKeys; ++kk) {
        const int src = (lane & ~3) | ((kk & 7) >> 1);
#pragma unroll
        for (int r = 0; r < 2; ++r) {                     // (HL: the second is lo of the same row)
          const uint32_t w = __shfl_sync(0xffffffffu, kk < 8 ? pa[r] : pa[2 + r], src);
          if (tile0 + kk >= min(it.k1, lim[HL ? 0 : r])) continue;
          const float p = bf16_half(w, kk & 1);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint32_t x = ld_shared_u32(v0 + tile_off<DP>(kk, n) + 4 * t);
            o[n][2 * r] = fmaf(p, bf16_half(x, 0), o[n][2 * r]);
            o[n][2 * r + 1] = fmaf(p, bf16_half(x, 1), o[n][2 * r + 1]);
          }
        }
      }
      if (!SHARE) __syncwarp();
      continue;
    }
#pragma unroll
    for (int n = 0; n < NT; n += 2) {
      uint32_t b[4];
      ldsm4_t(b, v0 + tile_off<DP>((lg & 1) * 8 + lr, n + (lg >> 1)));
      mma16816_bf16(o[n], pa, b[0], b[1]);
      mma16816_bf16(o[n + 1], pa, b[2], b[3]);
    }
    if (!SHARE) __syncwarp();                             // the slot may be filled again
  }
  cp_wait<0>();

#pragma unroll
  for (int r = 0; r < NR; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
  }
  auto sums = [&](int n, int r) {                         // columns 8 n + 2 t, + 1 of row g + 8 r
    return HL ? make_float2(o[n][0] + o[n][2], o[n][1] + o[n][3]) : make_float2(o[n][2 * r], o[n][2 * r + 1]);
  };
  if constexpr (SHARE) {                                  // a warp's rows are its own
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int row = r0 + 8 * r + g;
      if (row >= it.nrows) continue;
      float* dst = it.acc + (int64_t)row * d + 2 * t;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (8 * n < d) *reinterpret_cast<float2*>(dst + 8 * n) = sums(n, r);
      if (t == 0) *reinterpret_cast<float2*>(it.ml + 2 * row) = make_float2(ref[r], l[r]);
    }
    return;
  }
  // join the warps: references and weights, then sums (in the rings' memory)
  __syncthreads();
  float* sml = reinterpret_cast<float*>(smem);            // [warp][RB][2]
  // rows 8 words apart from a multiple of the 32 banks: a warp's 8 rows share none
  constexpr int LD = DP + 8;
  float* sac = sml + W * RB * 2;                          // [warp][RB][LD]
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int row = 8 * r + g;
    if (t == 0) {
      sml[(warp * RB + row) * 2] = ref[r];
      sml[(warp * RB + row) * 2 + 1] = l[r];
    }
    float* dst = sac + (warp * RB + row) * LD + 2 * t;
#pragma unroll
    for (int n = 0; n < NT; ++n) *reinterpret_cast<float2*>(dst + 8 * n) = sums(n, r);
  }
  __syncthreads();
  for (int idx = tid; idx < it.nrows * (d / 4); idx += W * 32) {
    const int row = idx / (d / 4), c = (idx - row * (d / 4)) * 4;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) top = fmaxf(top, sml[(w * RB + row) * 2]);
    const float r = top == -INFINITY ? 0.f : top;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    float lw = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = exp2f(sml[(w * RB + row) * 2] - r);
      const float4 x = *reinterpret_cast<const float4*>(sac + (w * RB + row) * LD + c);
      lw = fmaf(f, sml[(w * RB + row) * 2 + 1], lw);
      a.x = fmaf(f, x.x, a.x); a.y = fmaf(f, x.y, a.y);
      a.z = fmaf(f, x.z, a.z); a.w = fmaf(f, x.w, a.w);
    }
    *reinterpret_cast<float4*>(it.acc + (int64_t)row * d + c) = a;
    if (c == 0) {
      it.ml[2 * row] = top;
      it.ml[2 * row + 1] = lw;
    }
  }
}

template <int DP, bool HL, bool SHARE>
cudaError_t launch(const Params& q, long long n) {
  using C = Cfg<DP, SHARE>;
  static int smem_set[64];
  cudaError_t e = set_smem_limit_once((const void*)range_mma_kernel<DP, HL, SHARE>, (int)C::kSmem, smem_set);
  if (e != cudaSuccess) return e;
  return launch_dependent(range_mma_kernel<DP, HL, SHARE>, dim3((unsigned)n, q.a.Hk), dim3(C::W * 32),
                          C::kSmem, q.a.stream, q);
}
template <bool HL, bool SHARE>
cudaError_t launch_dp(const Params& q, long long n) {
  if constexpr (HL)
    if (q.p.dp == 256) return launch<256, HL, SHARE>(q, n);
  return q.p.dp == 64 ? launch<64, HL, SHARE>(q, n) : launch<128, HL, SHARE>(q, n);
}

}  // namespace

cudaError_t launch_prefix_mma(const Params& q) {
  const int rb = share_rows(q.p.dp, q.p.all);
  const long long n = (long long)q.p.p_splits * ((q.p.all + rb - 1) / rb);
  return rb == 32 ? launch_dp<true, true>(q, n) : launch_dp<false, true>(q, n);
}

cudaError_t launch_ranges_mma(const Params& q) {
  const int rb = mma_rows(q.p.dp, q.p.rows);
  long long n = (long long)q.p.cap * ((q.p.rows + rb - 1) / rb);
  if (q.a.prefix_len > 0 && !q.p.tc && !q.p.share) n += (long long)q.p.p_splits * ((q.p.all + rb - 1) / rb);
  return rb == 8 ? launch_dp<true, false>(q, n) : launch_dp<false, false>(q, n);
}

}  // namespace cache
}  // namespace dark
