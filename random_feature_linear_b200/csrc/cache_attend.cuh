// What the kernels of the cache attention share: the plan of a call (row counts, key
// ranges, workspace layout), the work items that a CTA index stands for, and the
// layout of partial results.
//
// Rows: the queries that read one key head are its G = H / Hk query heads of all
// sequences and tokens, row (b G + g) T + t; the G T rows of one sequence are
// consecutive. Keys: the prefix (one list of pages for all sequences, read once for
// all rows) and each sequence's own keys (its row of the page table). Both are cut into
// ranges; a range and a block of rows leave an unnormalised sum of values, the sum of
// weights and the reference exponent of every row, joined at the end.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace dark {
namespace cache {

constexpr int kKeyStep = 64;              // key ranges are multiples of this many keys

struct Plan {
  int rows, all;                          // G T rows of a sequence, B G T rows of a key head
  int dp;                                 // columns of the stored queries (d, padded)
  int mma;                                // bf16 with 16-byte rows: tensor cores
  int tc;                                 // the prefix by 128-row tiles (tcgen05)
  int share;                              // the prefix by blocks of share_rows() rows
  int p_splits, p_chunk;                  // ranges of the prefix, keys of a range
  int cap;                                // own ranges of all sequences, at most
  // byte offsets into the workspace
  size_t o_sched, o_y, o_y16, o_pacc, o_pml, o_oacc, o_oml, bytes;
};

// The cut of the own keys, written on the device from the sequences' lengths (one block
// of the first launch): int4 range[cap] = (sequence, first key, end, length), empty ones
// (0, 0, 0, 0) behind the last, then int off[B + 1] (ranges before sequence b), int len[B].
struct Params {
  CacheAttnArgs a;
  Plan p;
  int G;
  int box_rows;                           // rows of a tensor copy of the pools (0: none)
  long long stall;                        // testing stall of the tcgen05 kernel (0: none)
};

template <typename T>
__host__ __device__ inline T* at(const CacheAttnArgs& a, size_t off) {
  return reinterpret_cast<T*>(reinterpret_cast<char*>(a.ws) + off);
}

__device__ inline int4* sched_range(const Params& q) { return at<int4>(q.a, q.p.o_sched); }
__device__ inline int* sched_off(const Params& q) {
  return reinterpret_cast<int*>(sched_range(q) + q.p.cap);
}
__device__ inline int* sched_len(const Params& q) { return sched_off(q) + q.a.B + 1; }

// One CTA's work: keys [k0, k1) of a page list, rows [row0, row0 + nrows) of a key head.
struct Item {
  const int32_t* pages;
  int k0, k1;
  int row0, nrows;
  int len;                                // own keys of the sequence; -1: prefix
  float *acc, *ml;                        // partial sums [nrows][d], (exponent, weight) pairs
  bool any;
};

// The item of index x of key head `hk` with row blocks of `rb` rows: the prefix ranges
// first (if `prefix`), then the own ranges.
__device__ __forceinline__ Item item_of(const Params& q, int x, int hk, int rb, bool prefix,
                                        bool own) {
  const Plan& p = q.p;
  Item it;
  it.any = false;
  if (prefix) {
    const int nb = (p.all + rb - 1) / rb, n = p.p_splits * nb;
    if (x < n) {
      const int s = x / nb, blk = x % nb;
      it.pages = q.a.prefix_pages;
      it.k0 = s * p.p_chunk;
      it.k1 = it.k0 + p.p_chunk < q.a.prefix_len ? it.k0 + p.p_chunk : q.a.prefix_len;
      it.row0 = blk * rb;
      it.nrows = p.all - it.row0 < rb ? p.all - it.row0 : rb;
      it.len = -1;
      const size_t slot = ((size_t)hk * p.p_splits + s) * p.all + it.row0;
      it.acc = at<float>(q.a, p.o_pacc) + slot * q.a.d;
      it.ml = at<float>(q.a, p.o_pml) + slot * 2;
      it.any = it.k0 < it.k1;
      return it;
    }
    x -= n;
  }
  if (!own) return it;
  const int nb = (p.rows + rb - 1) / rb;
  const int r = x / nb, blk = x % nb;
  const int4 v = __ldcg(sched_range(q) + r);
  it.pages = q.a.table + (int64_t)v.x * q.a.max_pages;
  it.k0 = v.y;
  it.k1 = v.z;
  it.row0 = v.x * p.rows + blk * rb;
  it.nrows = p.rows - blk * rb < rb ? p.rows - blk * rb : rb;
  it.len = v.w;
  const size_t slot = ((size_t)hk * p.cap + r) * p.rows + blk * rb;
  it.acc = at<float>(q.a, p.o_oacc) + slot * q.a.d;
  it.ml = at<float>(q.a, p.o_oml) + slot * 2;
  it.any = it.k0 < it.k1;
  return it;
}

// Keys [0, limit) of the item's page list that its row `i` sees.
__device__ __forceinline__ int visible_keys(const Params& q, const Item& it, int i) {
  if (it.len < 0) return it.k1;
  if (!(q.a.flags & DARK_CAUSAL)) return it.len;
  const int t = (it.row0 + i) % q.a.T;
  const int lim = it.len - q.a.T + t + 1;
  return lim > 0 ? lim : 0;
}

// Row (of [page][d]) of key j of a page list for key head hk, or -1 where the list
// names no page of the cache.
__device__ __forceinline__ int64_t cache_row(const CacheAttnArgs& a, const int32_t* pages, int j,
                                             int hk) {
  const int pg = j / a.page, id = pages[pg];
  if (id < 0 || id >= a.pages) return -1;
  return ((int64_t)id * a.Hk + hk) * a.page + (j - pg * a.page);
}

}  // namespace cache
}  // namespace dark
