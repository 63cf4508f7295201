// Cache attention, prefix ranges on the tensor cores for many rows (bf16): the rows of the
// whole batch share the prefix's keys, so that a range is a pair of matrix products,
// S = Y K^T and O = P V, over tiles of 128 rows and 128 keys.
//
// A CTA takes one key range and up to RT tiles of 128 rows of one key head. Warps 0-3 (and
// 4-7 for the second tile) turn scores into weights, a thread a row, 64 keys at a time;
// warp 8 brings keys and values, warps 9-12 convert the keys; one lane of warp 13 issues the
// products (a second issuer, one a tile, measured 151 us against 141 at 1024 rows, 32768 keys,
// d = 128). S and O live in TMEM; P replaces S there as bf16 and is the first operand of the second product, which
// starts on the first 64 keys while the others are weighed. While one tile's scores are
// exponentiated the other tile's products run.
//
// Queries are rounded to fp16 and the keys converted to it in shared memory (bf16 keys are
// exact in fp16 between 2^-17 and 65504; anything larger is reported). bf16 queries (rounded
// by up to 2^-8 instead of 2^-11) doubled the error of the result: 3.7e-3 of its size against
// 1.7e-3 at 32768 keys; hi + lo in bf16 keeps it but costs half as many products again (whole
// calls: 241 us against 206 at 1024 rows of 8 heads, 32768 keys, d = 128; 36.5 against 34.9 at
// 64 rows, 4096 keys, d = 64). Four warps convert, one on each scheduler: two took 225 us, three
// 213; conversion from registers, straight from global memory, 235. Weights are rounded to
// bf16; scores, sums and exponents are fp32.
//
// Whole tiles of keys and values come by tensor copies of as many rows as divide both the
// page and the tile (8 at least); tiles that end inside the range's last page, and pages of
// other sizes, by 16-byte asynchronous copies with zeros behind the end (stale rows of a page
// may hold anything, and a weight of 0 does not cancel an infinity). Those take about 2000
// cycles to issue a 128 x 128 tile, twice the products' time.
//
// Bound by shared memory's bandwidth and the chain of a tile: the products alone (no
// weights, no conversion) take 117 us of the launch's 153, the conversion 20, the
// exponentials 16. All exponentials go to the special-function units: a quarter of them as
// polynomials in the multiply-add units measured 212 against 206, since the converting warps
// want the issue slots. Scores as two products of 64 keys, so that a half's weights overlap
// the other half's products, measured 218: such a product costs as much as one of 128 keys.
#include <math.h>

#include "cache_attend_mma.cuh"
#include "tc_common.cuh"
#include "tc_roles.cuh"

namespace dark {
namespace cache {
namespace {

using namespace tc;

constexpr int kT = 128;                               // rows and keys of a tile
constexpr int kSoftWarps = 8, kConv = 128;            // weights; converting threads
constexpr int kThreads = 32 * kSoftWarps + 32 + kConv + 32;
constexpr int NK = 3, NV = 2;                         // slots of key and value tiles

template <int DP>
struct Tc {
  static constexpr int RT = 2;                        // row tiles (TMEM: RT (128 + DP) columns)
  static constexpr int kBlk = kT * 128;               // 128 rows of 64 columns
  static constexpr uint32_t kTile = DP / 64 * kBlk;   // 128 rows of DP columns, bf16
  static constexpr uint32_t oQ = 0, oK = RT * kTile, oV = oK + NK * kTile, oRows = oV + NV * kTile;
  static constexpr uint32_t oBar = oRows + kT * 8, kSmem = oBar + 256 + 1024;
  static constexpr uint32_t tS = 0, tO = RT * 128, kCols = 512;
  static_assert(tO + RT * DP <= kCols, "tmem");
  static_assert(kSmem <= 232448, "shared memory");
};

// D (TMEM) += A (TMEM, bf16 pairs a column) B (shared memory).
__device__ __forceinline__ void mma_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t id,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(id), "r"(accumulate)
      : "memory");
}
// 16 columns of this thread's TMEM lane; complete after tmem_wait_st.
__device__ __forceinline__ void tmem_st16_async(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// Whether any of the converting threads passes `bad`.
__device__ __forceinline__ bool conv_sync_or(bool bad) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)bad), "n"(kConv)
      : "memory");
  return r != 0;
}
struct Bars {
  uint64_t q, never, drain;
  // per row tile: scores, weights of the first and last 64 keys, the first's products, all sums
  uint64_t s[2], p[2][2], h[2], o[2];
  uint64_t kraw[NK], kfull[NK], kempty[NK], vfull[NV], vempty[NV];     // kraw: keys before conversion
  uint32_t tmem;
  int abort;
};

// A row's reference is the largest of its first 64 scores, and moves when the weights of 64
// later ones sum up to more than this: bf16 and fp32 keep their relative precision at any
// size, so that only a sum far inside fp32's range matters, and no maximum is taken meanwhile.
constexpr float kGuard = 4294967296.f;

// Weights of 64 scores of a thread's row (keys c0 ... of the tile; TAIL: only keys below
// `end` count) against the reference r, as bf16 into TMEM columns tp ..., and their sum.
template <bool TAIL>
__device__ __forceinline__ float weigh(const uint32_t (&v)[2][32], uint32_t tp, float r, int c0, int end) {
  const F2 minus_r(-r, -r);
  F2 sum[2] = {F2(0.f, 0.f), F2(0.f, 0.f)};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const F2 x = add2(F2(__uint_as_float(v[k][2 * e]), __uint_as_float(v[k][2 * e + 1])), minus_r);
      float2 p = x.get();
      p = make_float2(ex2(p.x), ex2(p.y));
      if (TAIL) {
        const int c = c0 + 32 * k + 2 * e;
        p.x = c < end ? p.x : 0.f;
        p.y = c + 1 < end ? p.y : 0.f;
      }
      sum[e & 1] = add2(sum[e & 1], F2(p.x, p.y));
      w[e] = pack_bf16(p.x, p.y);
    }
    tmem_st16_async(tp + 16 * k, w);
  }
  return sum[0].sum() + sum[1].sum();
}
template <bool TAIL>
__device__ __forceinline__ float most(const uint32_t (&v)[2][32], int c0, int end) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int e = 0; e < 64; e += 2) {
    const float a = !TAIL || c0 + e < end ? __uint_as_float(v[e / 32][e % 32]) : -INFINITY;
    const float b = !TAIL || c0 + e + 1 < end ? __uint_as_float(v[e / 32][e % 32 + 1]) : -INFINITY;
    m[e / 2 & 3] = fmaxf(m[e / 2 & 3], fmaxf(a, b));
  }
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) range_tc_kernel(const __grid_constant__ Params q,
                                                                const __grid_constant__ CUtensorMap tm_k,
                                                                const __grid_constant__ CUtensorMap tm_v) {
  using C = Tc<DP>;
  constexpr int RT = C::RT, CH = DP / 8;
  static_assert(sizeof(Bars) <= 256, "barriers");
  const int hk = blockIdx.y;
  const Item it = item_of(q, blockIdx.x, hk, RT * kT, true, false);
  if (!it.any) return;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t s0 = smem_u32(sm);
  Bars* bar = reinterpret_cast<Bars*>(sm + C::oBar);
  volatile int* abort = &bar->abort;
  int* status = q.a.dev_status;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tiles = (it.k1 - it.k0 + kT - 1) / kT, rts = it.nrows > kT ? RT : 1;
  const int d = q.a.d, ks = (d + 15) / 16;            // steps of 16 columns

  if (tid == 0) {
    mbar_init(&bar->q, kConv);
    mbar_init(&bar->never, 1);
    mbar_init(&bar->drain, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->s[i], 1);
      mbar_init(&bar->p[i][0], kT);
      mbar_init(&bar->p[i][1], kT);
      mbar_init(&bar->h[i], 1);
      mbar_init(&bar->o[i], 1);
    }
    for (int i = 0; i < NK; ++i) {
      mbar_init(&bar->kraw[i], 1);
      mbar_init(&bar->kfull[i], kConv);
      mbar_init(&bar->kempty[i], 1);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(&bar->vfull[i], 1);
      mbar_init(&bar->vempty[i], 1);
    }
    bar->abort = 0;
    fence_mbar_init();
  }
  __syncwarp();
  if (warp == 0) tmem_alloc(&bar->tmem, C::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem;
  pdl_wait();
  pdl_launch();
  bool go = true;
  if (q.stall > 0) {
    if (tid == 0) wait_one(&bar->never, 0, abort, status, q.stall);
    __syncthreads();
    go = !*abort;
  }

  // tiles that come by tensor copies (the others, at the end of the last range or of pages of
  // odd sizes, by the converting threads)
  const int box = q.box_rows, whole = box > 0 ? (it.k1 - it.k0) / kT : 0;
  if (go && warp == kSoftWarps) {
    // ---- tensor copies K_0, V_0, K_1, V_1, ...
    const int nb = (d + 63) / 64;
    auto wait = [&](uint64_t* b, uint32_t parity) {
      return (bool)__all_sync(0xffffffffu, wait_one(b, parity, abort, status));
    };
    auto copy = [&](const CUtensorMap* map, uint32_t dst, int key0, uint64_t* b) {
      for (int x = lane; x < kT / box * nb; x += 32) {
        const int r = x / nb * box, cb = x % nb, key = key0 + r, pg = key / q.a.page;
        const int id = it.pages[pg];
        const bool good = id >= 0 && id < q.a.pages;
        if (!good) report(status, DARK_ERR_INVALID_ARG);
        // a page outside the cache: outside the map, zeros
        tma_load_3d(dst + cb * C::kBlk + r * 128, map, 64 * cb, key - pg * q.a.page,
                    good ? id * q.a.Hk + hk : q.a.pages * q.a.Hk, b);
      }
      if (lane == 0) mbar_arrive_expect_tx(b, kT * 128 * nb);
      __syncwarp();
    };
    int nk = 0, nv = 0;                               // copies issued
    for (int j = 0; j < whole; ++j) {
      const int key0 = it.k0 + j * kT, ik = j % NK, iv = j % NV;
      if (j >= NK && !wait(&bar->kempty[ik], (j / NK - 1) & 1)) break;
      copy(&tm_k, s0 + C::oK + ik * C::kTile, key0, &bar->kraw[ik]);
      ++nk;
      if (j >= NV && !wait(&bar->vempty[iv], (j / NV - 1) & 1)) break;
      copy(&tm_v, s0 + C::oV + iv * C::kTile, key0, &bar->vfull[iv]);
      ++nv;
    }
    if (*abort && lane == 0) {                        // copies may be on their way
      for (int j = max(0, nk - NK); j < nk; ++j) mbar_wait(&bar->kraw[j % NK], (j / NK) & 1, kWaitCycles / 8);
      for (int j = max(0, nv - NV); j < nv; ++j) mbar_wait(&bar->vfull[j % NV], (j / NV) & 1, kWaitCycles / 8);
    }
    __syncwarp();
  } else if (go && warp > kSoftWarps && warp < kSoftWarps + 1 + kConv / 32) {
    // ---- queries; keys to fp16 in place; tiles without tensor copies. A thread that saw an
    // abort goes on without copying: the barriers stay matched.
    const int t = tid - 32 * (kSoftWarps + 1), c = t % CH;
    const __half* y = at<__half>(q.a, q.p.o_y16) + ((int64_t)hk * q.p.all + it.row0) * DP;
    for (int r = t / CH; r < rts * kT; r += kConv / CH)
      cp16(s0 + C::oQ + (r / kT) * C::kTile + kmajor_off(r % kT, c * 8, C::kBlk),
           y + (r < it.nrows ? (int64_t)r * DP + c * 8 : 0), r < it.nrows);
    cp_commit();
    int64_t* rows = reinterpret_cast<int64_t*>(sm + C::oRows);
    const bool in = c < 2 * ks, has = c * 8 < d;      // (a last half step is zeros)
    bool ok = true;
    auto fetch = [&](const void* pool, uint32_t dst) {
      if (ok && in) {
        const __nv_bfloat16* src = (const __nv_bfloat16*)pool + c * 8;
#pragma unroll 4
        for (int r = t / CH; r < kT; r += kConv / CH) {
          const int64_t row = rows[r];
          const bool live = row >= 0 && has;
          cp16(dst + kmajor_off(r, c * 8, C::kBlk), src + (live ? row * d : 0), live);
        }
      }
      cp_commit();
    };
    __half2 top = __float2half2_rn(0.f);              // largest converted magnitude
    for (int j = 0; j < tiles; ++j) {
      const int ik = j % NK, iv = j % NV, key0 = it.k0 + j * kT;
      const uint32_t tile = s0 + C::oK + ik * C::kTile;
      const bool lone = j >= whole;
      if (lone) {
        if (ok && j >= NK) ok = wait_one(&bar->kempty[ik], (j / NK - 1) & 1, abort, status);
        conv_sync_or(false);                          // the last tile's rows have been used
        for (int k = t; k < kT; k += kConv) {
          const int key = key0 + k;
          int64_t row = -1;
          if (key < it.k1) {
            row = cache_row(q.a, it.pages, key, hk);
            if (row < 0) report(status, DARK_ERR_INVALID_ARG);
          }
          rows[k] = row;
        }
        ok = !conv_sync_or(!ok);
        fetch(q.a.kp, tile);
        if (ok && j >= NV) ok = wait_one(&bar->vempty[iv], (j / NV - 1) & 1, abort, status);
        fetch(q.a.vp, s0 + C::oV + iv * C::kTile);
        cp_wait<1>();                                 // the keys (and the queries)
      } else if (ok) {
        ok = wait_one(&bar->kraw[ik], (j / NK) & 1, abort, status);
      }
      if (ok && in) {
#pragma unroll 4
        for (int r = t / CH; r < kT; r += kConv / CH) {
          const uint32_t at = tile + kmajor_off(r, c * 8, C::kBlk);
          const uint4 v = ld_shared_v4(at);
          auto half2 = [&](uint32_t w) {
            const __half2 h = __floats2half2_rn(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
            top = __hmax2(top, __habs2(h));
            return *reinterpret_cast<const uint32_t*>(&h);
          };
          st_shared_v4(at, half2(v.x), half2(v.y), half2(v.z), half2(v.w));
        }
      }
      if (j == 0 && !lone) cp_wait<0>();              // the queries
      fence_async_smem();
      if (j == 0) mbar_arrive(&bar->q);
      mbar_arrive(&bar->kfull[ik]);
      if (lone) {
        cp_wait<0>();
        fence_async_smem();
        conv_sync_or(false);
        if (t == 0) mbar_arrive(&bar->vfull[iv]);
      }
    }
    if (__hisinf(__low2half(top)) || __hisinf(__high2half(top))) report(status, DARK_ERR_NUMERIC);
  } else if (go && warp == kThreads / 32 - 1) {
    // ---- products: the warp stays together, one lane issues
    {
      const bool lead = elect_one();
      const uint32_t id_s = idesc(kT, kT, false, false, true);
      const uint32_t id_o = idesc(kT, 16 * ks, false, true, false);
      // operands' descriptors: steps add to the address field (one lane issues all products,
      // so that a few instructions a product count)
      const uint64_t dq = sdesc(s0 + C::oQ, 16, 1024), dk = sdesc(s0 + C::oK, 16, 1024);
      const uint64_t dv = sdesc(s0 + C::oV, C::kBlk, 1024);
      auto scores = [&](int x, int j) {               // S_x = Y_x K_j^T
        if (!lead) return;
        const uint64_t a = dq + (uint32_t)(x * (C::kTile >> 4)), b = dk + (uint32_t)(j % NK * (C::kTile >> 4));
#pragma unroll
        for (int s = 0; s < DP / 16; ++s)
          if (s < ks) {
            const uint32_t step = (s / 4 * C::kBlk + s % 4 * 32) >> 4;
            mma(tmem + C::tS + x * kT, a + step, b + step, id_s, s > 0);
          }
        mma_commit(&bar->s[x]);
        if (x == rts - 1) mma_commit(&bar->kempty[j % NK]);
      };
      auto values = [&](int x, int j, int half, bool add) {       // O_x += P_x V_j over half of the keys
        if (!lead) return;
        const uint64_t b = dv + (uint32_t)(j % NV * (C::kTile >> 4) + half * (8192 >> 4));
        const uint32_t a = tmem + C::tS + x * kT + half * 32;
#pragma unroll
        for (int s = 0; s < kT / 32; ++s)
          mma_ts(tmem + C::tO + x * DP, a + 8 * s, b + (s * 2048 >> 4), id_o, add || s > 0);
        if (half == 0) mma_commit(&bar->h[x]);
        else if (x == rts - 1) mma_commit(&bar->vempty[j % NV]);
      };
      auto wait = [&](uint64_t* b, uint32_t parity) {
        return (bool)__all_sync(0xffffffffu, wait_one(b, parity, abort, status));
      };
      bool ok = wait(&bar->q, 0) && wait(&bar->kfull[0], 0);
      if (ok) {
        tc_fence_after();
        for (int x = 0; x < rts; ++x) scores(x, 0);
      }
      for (int j = 0; j < tiles && ok; ++j) {
        const bool more = j + 1 < tiles;
        ok = wait(&bar->vfull[j % NV], (j / NV) & 1);
        for (int x = 0; x < rts && ok; ++x) {
          ok = wait(&bar->p[x][0], j & 1);
          if (!ok) break;
          tc_fence_after();
          values(x, j, 0, j > 0);
          // (the next keys' wait ahead of the weights', off the path to the scores)
          ok = (!more || x > 0 || wait(&bar->kfull[(j + 1) % NK], ((j + 1) / NK) & 1)) &&
               wait(&bar->p[x][1], j & 1);
          if (!ok) break;
          tc_fence_after();
          values(x, j, 1, true);
          if (more)
            scores(x, j + 1);
          else if (lead)
            mma_commit(&bar->o[x]);
        }
        __syncwarp();
      }
      if (lead) drain_mmas(&bar->drain);
      __syncwarp();
    }
  } else if (go && warp / 4 < rts) {
    // ---- weights: this thread's row of tile x
    const int x = warp / 4, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t ts = lanes + C::tS + x * kT, to = lanes + C::tO + x * DP;
    float ref = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < tiles && ok; ++j) {
      ok = __all_sync(0xffffffffu, wait_one(&bar->s[x], j & 1, abort, status));
      if (!ok) break;
      tc_fence_after();
      const int end = it.k1 - it.k0 - j * kT;         // keys of this tile
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const int c0 = 64 * half;
        const uint32_t tp = ts + 32 * half;           // (over scores that were read)
        uint32_t v[2][32];
        tmem_ld_blocks(ts + c0, v);
        const bool tail = end < c0 + 64, first = j == 0 && half == 0;
        float lt = 0.f;
        auto weights = [&]() {
          // all scores so far are -inf, or NaN: no reference (the weights follow the scores)
          const float r = ref == -INFINITY ? 0.f : ref;
          lt = tail ? weigh<true>(v, tp, r, c0, end) : weigh<false>(v, tp, r, c0, end);
        };
        if (!first) weights();
        // their sum tells whether a score has passed the reference too far (or is not finite)
        if (__any_sync(0xffffffffu, first || !(lt <= kGuard))) {
          const float top = tail ? most<true>(v, c0, end) : most<false>(v, c0, end);
          const bool move = first || !(lt <= kGuard);
          const float now = move ? fmaxf(ref, top) : ref, f = now > ref ? exp2f(ref - now) : 1.f;
          ref = now;
          l *= f;
          if (!first) {
            // O holds the earlier tiles (complete: the scores came after them) and, at the
            // second half, the first one's products
            if (half == 1) {
              ok = __all_sync(0xffffffffu, wait_one(&bar->h[x], j & 1, abort, status));
              if (!ok) break;
              tc_fence_after();
            }
            for (int c = 0; c < 16 * ks; c += 16) {
              float o[16];
              tmem_ld16(to + c, o);
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * f);
              tmem_st16_async(to + c, w);
            }
          }
          weights();
        }
        l += lt;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bar->p[x][half]);
      }
    }
    if (ok) ok = __all_sync(0xffffffffu, wait_one(&bar->o[0], 0, abort, status) &&
                                           (rts == 1 || wait_one(&bar->o[1], 0, abort, status)));
    if (ok) {
      tc_fence_after();
      // sums through shared memory (all tiles of the ring have been read): 32 rows of 32
      // columns a warp at a time, so that rows are written in runs of 128 bytes
      float4* box = reinterpret_cast<float4*>(sm + C::oK + warp * 4096);
      const int row0 = x * kT + quad * 32;
      for (int c = 0; c < d; c += 32) {
        float o[32];
        tmem_ld32(to + c, o);
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e)
          box[lane * 8 + (e ^ (lane & 7))] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 4 * i + lane / 8, e = lane & 7;
          const float4 w = box[r * 8 + (e ^ (r & 7))];
          if (row0 + r < it.nrows && c + 4 * e < d)
            *reinterpret_cast<float4*>(it.acc + (int64_t)(row0 + r) * d + c + 4 * e) = w;
        }
      }
      if (x * kT + row < it.nrows)
        *reinterpret_cast<float2*>(it.ml + 2 * (x * kT + row)) = make_float2(ref, l);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

// A map of one pool: boxes of 64 columns and `box` rows of a page of one head.
bool pool_map(const CacheAttnArgs& a, const void* pool, int box, CUtensorMap* map) {
  const uint64_t dims[3] = {(uint64_t)a.d, (uint64_t)a.page, (uint64_t)a.pages * a.Hk};
  const uint64_t strides[2] = {(uint64_t)a.d * 2, (uint64_t)a.page * a.d * 2};
  const uint32_t b[3] = {64, (uint32_t)box, 1};
  return encode_tmap(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, pool, dims, strides, b);
}

template <int DP>
cudaError_t launch(const Params& q, const CUtensorMap& tk, const CUtensorMap& tv) {
  using C = Tc<DP>;
  static int smem_set[64];
  cudaError_t e = set_smem_limit_once((const void*)range_tc_kernel<DP>, (int)C::kSmem, smem_set);
  if (e != cudaSuccess) return e;
  const int rb = C::RT * kT;
  const dim3 grid((unsigned)(q.p.p_splits * ((q.p.all + rb - 1) / rb)), q.a.Hk);
  return launch_dependent(range_tc_kernel<DP>, grid, dim3(kThreads), C::kSmem, q.a.stream, q, tk, tv);
}

}  // namespace

cudaError_t launch_prefix_tc(const Params& q0) {
  Params q = q0;
  CUtensorMap tk = {}, tv = {};
  // rows of a box: a power of two that divides the page, 8 at least (the swizzle's period)
  q.box_rows = q.a.page & -q.a.page;
  if (q.box_rows > kT) q.box_rows = kT;
  if (q.box_rows < 8 || (int64_t)q.a.pages * q.a.Hk >= (int64_t)1 << 31 ||
      !pool_map(q.a, q.a.kp, q.box_rows, &tk) || !pool_map(q.a, q.a.vp, q.box_rows, &tv))
    q.box_rows = 0;
  return q.p.dp == 64 ? launch<64>(q, tk, tv) : launch<128>(q, tk, tv);
}

}  // namespace cache
}  // namespace dark
