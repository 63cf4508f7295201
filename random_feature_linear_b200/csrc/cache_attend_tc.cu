// Cache attention, prefix ranges on the tensor cores for many rows (bf16): the rows of the
// whole batch share the prefix's keys, so that a range is a pair of matrix products,
// S = Y K^T and O = P V, over tiles of 128 rows and 128 keys.
//
// A CTA takes one key range and up to RT tiles of 128 rows of one key head. Warps 0-3 (and
// 4-7 for the second tile) turn scores into weights, a thread a row; warps 8-11 bring keys
// and values; one lane of warp 12 issues the products. S and O live in TMEM; P replaces S
// there as bf16 and is the first operand of the second product. While one tile's scores
// are exponentiated the other tile's products run. A row's reference exponent moves only
// when a score passes it by 2^8, so that O is rescaled a few times a range.
//
// Queries and weights are rounded to bf16 (the products' operand type); scores, sums and
// exponents are fp32. Keys and values come by 16-byte asynchronous copies rather than tensor
// copies: pages may have any size and a range may end inside one.
//
// Bound by the two products (4 rows keys d operations) and the exponentials (rows keys)
// alike: one 128 x 128 tile at d = 128 takes 1024 cycles of either unit.
#include <math.h>

#include "cache_attend_mma.cuh"
#include "tc_common.cuh"
#include "tc_roles.cuh"

namespace dark {
namespace cache {
namespace {

using namespace tc;

constexpr int kT = 128;                               // rows and keys of a tile
constexpr int kThreads = 13 * 32;

template <int DP>
struct Tc {
  static constexpr int RT = DP == 256 ? 1 : 2;        // row tiles (TMEM: RT (128 + DP) columns)
  static constexpr int kBlk = kT * 128;               // 128 rows of 64 columns
  static constexpr uint32_t kTile = DP / 64 * kBlk;   // 128 rows of DP columns, bf16
  static constexpr int kSlots = (int)(131072 / kTile);  // ring of key and value tiles
  static constexpr uint32_t oQ = 0, oRing = RT * kTile, oRows = oRing + kSlots * kTile;
  static constexpr uint32_t oBar = oRows + 2 * kT * 8, kSmem = oBar + 256 + 1024;
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
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// Whether any of the 128 loading threads passes `bad`.
__device__ __forceinline__ bool loaders_sync_or(bool bad) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)bad)
      : "memory");
  return r != 0;
}

// Whether the phase with the given parity has completed (does not wait).
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

struct Bars {
  uint64_t q, never, drain;
  uint64_t s[2], p[2], o[2];              // per row tile: scores, weights, sums are ready
  uint64_t full[8], empty[8];             // ring slots
  uint32_t tmem;
  int abort;
};

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) range_tc_kernel(const __grid_constant__ Params q) {
  using C = Tc<DP>;
  constexpr int RT = C::RT, S = C::kSlots, CH = DP / 8;
  static_assert(S >= 2 && S <= 8, "ring");
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
    mbar_init(&bar->q, 128);
    mbar_init(&bar->never, 1);
    mbar_init(&bar->drain, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->s[i], 1);
      mbar_init(&bar->p[i], 128);
      mbar_init(&bar->o[i], 1);
    }
    for (int i = 0; i < S; ++i) {
      mbar_init(&bar->full[i], 128);
      mbar_init(&bar->empty[i], 1);
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

  if (go && warp >= 8 && warp < 12) {
    // ---- queries, then tiles K_0, V_0, K_1, V_1, ... through the ring; a copy is handed
    // over when this thread's part of it has arrived. The threads agree on an abort before
    // each key tile (they share the tile's row numbers).
    const int t = tid - 256, c = t % CH;
    const __nv_bfloat16* y = at<__nv_bfloat16>(q.a, q.p.o_y) + ((int64_t)hk * q.p.all + it.row0) * DP;
    for (int r = t / CH; r < rts * kT; r += kT / CH)
      cp16(s0 + C::oQ + (r / kT) * C::kTile + kmajor_off(r % kT, c * 8, C::kBlk),
           y + (r < it.nrows ? (int64_t)r * DP + c * 8 : 0), r < it.nrows);
    cp_commit();
    int64_t* rows = reinterpret_cast<int64_t*>(sm + C::oRows);
    const bool in = c < 2 * ks, has = c * 8 < d;      // (a last half step is zeros)
    const int n = 2 * tiles;
    // row of the cache that this thread looks up for tile j; the page a tile ahead of its use
    auto lookup = [&](int j) {
      const int key = it.k0 + j * kT + t;
      if (key >= it.k1) return (int64_t)-1;
      const int64_t row = cache_row(q.a, it.pages, key, hk);
      if (row < 0) report(status, DARK_ERR_INVALID_ARG);
      return row;
    };
    int64_t next_row = lookup(0);
    int done = 0;                                     // copies handed over (this thread's part)
    auto hand_over = [&](int issued) {                // copy `done`, of `issued` so far
      switch (issued - done) {
        case 1: cp_wait<0>(); break;
        case 2: cp_wait<1>(); break;
        case 3: cp_wait<2>(); break;
        default: cp_wait<3>(); break;
      }
      fence_async_smem();
      if (done == 0) mbar_arrive(&bar->q);            // (the queries' group came first)
      mbar_arrive(&bar->full[done % S]);
      ++done;
    };
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const int slot = i % S, j = i / 2;
      if (ok && i >= S) {
        // while the slot is still read, hand over what has arrived
        const uint32_t parity = (i / S - 1) & 1;
        while (done < i && !mbar_test(&bar->empty[slot], parity)) hand_over(i);
        ok = wait_one(&bar->empty[slot], parity, abort, status);
      }
      if (!(i & 1)) {
        rows[(j & 1) * kT + t] = next_row;
        ok = !loaders_sync_or(!ok);
        if (!ok) break;
      }
      if (ok && in) {
        const __nv_bfloat16* pool = (const __nv_bfloat16*)(i & 1 ? q.a.vp : q.a.kp) + c * 8;
        const uint32_t dst = s0 + C::oRing + slot * C::kTile;
#pragma unroll 4
        for (int r = t / CH; r < kT; r += kT / CH) {
          const int64_t row = rows[(j & 1) * kT + r];
          const bool live = row >= 0 && has;
          cp16(dst + kmajor_off(r, c * 8, C::kBlk), pool + (live ? row * d : 0), live);
        }
      }
      cp_commit();
      if (!(i & 1) && j + 1 < tiles) next_row = lookup(j + 1);
      if (i - done >= 3) hand_over(i + 1);
    }
    while (ok && done < n) hand_over(n);
    cp_wait<0>();
  } else if (go && warp == 12) {
    // ---- products
    if (lane == 0) {
      const uint32_t id_s = idesc(kT, kT, false, false, false);
      const uint32_t id_o = idesc(kT, 16 * ks, false, true, false);
      auto scores = [&](int x, int i) {               // S_x = Y_x K^T, keys in ring copy i
        const uint32_t a = s0 + C::oQ + x * C::kTile, b = s0 + C::oRing + (i % S) * C::kTile;
        for (int s = 0; s < ks; ++s)
          mma(tmem + C::tS + x * kT, sdesc(a + (s / 4) * C::kBlk + (s % 4) * 32, 16, 1024),
              sdesc(b + (s / 4) * C::kBlk + (s % 4) * 32, 16, 1024), id_s, s > 0);
        mma_commit(&bar->s[x]);
      };
      auto values = [&](int x, int i, bool add) {     // O_x += P_x V, values in ring copy i
        const uint32_t b = s0 + C::oRing + (i % S) * C::kTile;
        for (int s = 0; s < kT / 16; ++s)
          mma_ts(tmem + C::tO + x * DP, tmem + C::tS + x * kT + 8 * s,
                 sdesc(b + s * 2048, C::kBlk, 1024), id_o, add || s > 0);
      };
      bool ok = wait_one(&bar->q, 0, abort, status) && wait_one(&bar->full[0], 0, abort, status);
      if (ok) {
        tc_fence_after();
        for (int x = 0; x < rts; ++x) scores(x, 0);
        mma_commit(&bar->empty[0]);
      }
      for (int j = 0; j < tiles && ok; ++j) {
        const int iv = 2 * j + 1, ik = 2 * j + 2;
        const bool more = j + 1 < tiles;
        ok = wait_one(&bar->full[iv % S], (iv / S) & 1, abort, status);
        for (int x = 0; x < rts && ok; ++x) {
          ok = wait_one(&bar->p[x], j & 1, abort, status);
          if (!ok) break;
          tc_fence_after();
          values(x, iv, j > 0);
          if (x == rts - 1) mma_commit(&bar->empty[iv % S]);
          if (!more) {
            mma_commit(&bar->o[x]);
          } else {
            if (x == 0) ok = wait_one(&bar->full[ik % S], (ik / S) & 1, abort, status);
            if (!ok) break;
            tc_fence_after();
            scores(x, ik);
            if (x == rts - 1) mma_commit(&bar->empty[ik % S]);
          }
        }
      }
      drain_mmas(&bar->drain);
    }
    __syncwarp();
  } else if (go && warp / 4 < rts) {
    // ---- weights: this thread's row of tile x
    const int x = warp / 4, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t ts = lanes + C::tS + x * kT, to = lanes + C::tO + x * DP;
    float ref = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < tiles; ++j) {
      ok = __all_sync(0xffffffffu, wait_one(&bar->s[x], j & 1, abort, status));
      if (!ok) break;
      tc_fence_after();
      const int end = it.k1 - it.k0 - j * kT;         // keys of this tile
      uint32_t a[32], b[32];
      float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      auto most = [&](const uint32_t (&v)[32], int c0) {
        if (end >= kT) {
#pragma unroll
          for (int e = 0; e < 32; ++e) m[e & 3] = fmaxf(m[e & 3], __uint_as_float(v[e]));
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (c0 + e < end) m[e & 3] = fmaxf(m[e & 3], __uint_as_float(v[e]));
        }
      };
      tmem_ld32_async(ts, a);
      tmem_wait_ld(a);
      tmem_ld32_async(ts + 32, b);
      most(a, 0);
      tmem_wait_ld(b);
      tmem_ld32_async(ts + 64, a);
      most(b, 32);
      tmem_wait_ld(a);
      tmem_ld32_async(ts + 96, b);
      most(a, 64);
      tmem_wait_ld(b);
      tmem_ld32_async(ts, a);
      most(b, 96);
      const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
      const bool move = top > ref + 8.f;              // (-inf + 8 = -inf: the first tile)
      if (__any_sync(0xffffffffu, move)) {
        const float now = move ? top : ref, f = move ? exp2f(ref - now) : 1.f;
        ref = now;
        l *= f;
        tmem_wait_ld(a);
        if (j > 0) {                                  // (the scores' arrival: O is complete too)
          for (int c = 0; c < 16 * ks; c += 16) {
            float o[16];
            tmem_ld16(to + c, o);
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * f);
            tmem_st16_async(to + c, w);
          }
          tmem_wait_st();
        }
      }
      // all scores of a row are -inf, or NaN: no reference (the weights follow the scores)
      const float r = ref == -INFINITY ? 0.f : ref;
      const F2 minus_r(-r, -r);
      F2 sum[2] = {F2(0.f, 0.f), F2(0.f, 0.f)};
      auto weigh = [&](const uint32_t (&v)[32], int c0) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 x = add2(F2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), minus_r).get();
          float p0 = ex2(x.x), p1 = ex2(x.y);
          if (end < kT) {
            p0 = c0 + 2 * e < end ? p0 : 0.f;
            p1 = c0 + 2 * e + 1 < end ? p1 : 0.f;
          }
          sum[e & 1] = add2(sum[e & 1], F2(p0, p1));
          w[e] = pack_bf16(p0, p1);
        }
        tmem_st16_async(ts + c0 / 2, w);              // over scores that were read
      };
      tmem_wait_ld(a);
      tmem_ld32_async(ts + 32, b);
      weigh(a, 0);
      tmem_wait_ld(b);
      tmem_ld32_async(ts + 64, a);
      weigh(b, 32);
      tmem_wait_ld(a);
      tmem_ld32_async(ts + 96, b);
      weigh(a, 64);
      tmem_wait_ld(b);
      weigh(b, 96);
      l += sum[0].sum() + sum[1].sum();
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bar->p[x]);
    }
    if (ok) ok = __all_sync(0xffffffffu, wait_one(&bar->o[x], 0, abort, status));
    if (ok) {
      tc_fence_after();
      // sums through shared memory (the tile's queries have been read): 32 rows of 32
      // columns a warp at a time, so that rows are written in runs of 128 bytes
      float4* box = reinterpret_cast<float4*>(sm + C::oQ + x * C::kTile + (warp & 3) * 4096);
      const int row0 = x * kT + (warp & 3) * 32;
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
          const float4 v = box[r * 8 + (e ^ (r & 7))];
          if (row0 + r < it.nrows && c + 4 * e < d)
            *reinterpret_cast<float4*>(it.acc + (int64_t)(row0 + r) * d + c + 4 * e) = v;
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

template <int DP>
cudaError_t launch(const Params& q) {
  using C = Tc<DP>;
  static int smem_set[64];
  cudaError_t e = set_smem_limit_once((const void*)range_tc_kernel<DP>, (int)C::kSmem, smem_set);
  if (e != cudaSuccess) return e;
  const int rb = C::RT * kT;
  const dim3 grid((unsigned)(q.p.p_splits * ((q.p.all + rb - 1) / rb)), q.a.Hk);
  return launch_dependent(range_tc_kernel<DP>, grid, dim3(kThreads), C::kSmem, q.a.stream, q);
}

}  // namespace

cudaError_t launch_prefix_tc(const Params& q) {
  return q.p.dp == 64 ? launch<64>(q) : q.p.dp == 128 ? launch<128>(q) : launch<256>(q);
}

}  // namespace cache
}  // namespace dark
