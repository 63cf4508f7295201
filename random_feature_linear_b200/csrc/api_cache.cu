// C ABI of the head norms with rotation, the paged cache and the exact mode's
// attention over it (declared in include/dark.h): argument validation on the host and
// launches on the caller's stream. Nothing here allocates device memory.
#include <math.h>
#include <string.h>

#include "common.cuh"
#include "internal.h"

namespace {

constexpr int kMaxD = 256, kMaxR = 256, kMaxM = 1024;
constexpr int64_t kMaxKeys = (int64_t)1 << 30;     // keys of one page list, tokens of a call

bool dtype_ok(dark_dtype t) { return t == DARK_F32 || t == DARK_BF16; }
size_t elt(dark_dtype t) { return t == DARK_BF16 ? 2 : 4; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
dark_status from_cuda(cudaError_t e) { return e == cudaSuccess ? DARK_OK : DARK_ERR_CUDA; }

bool rope_ok(const dark_rope* r) {
  return r->dims >= 0 && r->dims <= kMaxD && r->dims % 2 == 0 &&
         (r->interleaved == 0 || r->interleaved == 1);
}

// Element strides of a [B][H][L][d] tensor (null: contiguous). Results need a place of
// their own for every row, so a stride of 0 over more than one index is refused there.
bool take_strides(int64_t (&out)[3], const int64_t* s, int B, int H, int L, int d, bool written) {
  const int64_t c[3] = {(int64_t)H * L * d, (int64_t)L * d, d};
  const int n[3] = {B, H, L};
  for (int i = 0; i < 3; ++i) {
    out[i] = s ? s[i] : c[i];
    if (out[i] < 0 || (written && out[i] == 0 && n[i] > 1)) return false;
  }
  return true;
}

// Rows worked on in place: the same memory has to mean the same rows.
bool in_place_ok(const void* x, const int64_t (&xs)[3], const void* y, const int64_t (&ys)[3]) {
  return x != y || (xs[0] == ys[0] && xs[1] == ys[1] && xs[2] == ys[2]);
}

bool gamma_ok(const float* g, int heads, int H) {
  return g == nullptr || (aligned(g, 4) && (heads == 1 || heads == H));
}

// What the forward and backward of the head norms check alike; fills all but the rows.
dark_status norm_rope_args(dark::NormRopeArgs& a, const float* gamma_q, int heads_gq,
                           const float* gamma_k, int heads_gk, float eps, const dark_rope* rope,
                           const int32_t* positions, int64_t pos0, int B, int H, int Hk, int L,
                           int d, dark_dtype dtype, int* dev_status, void* stream) {
  memset(&a, 0, sizeof(a));
  if (!dtype_ok(dtype) || B < 1 || H < 1 || Hk < 0 || L < 1 || d < 1) return DARK_ERR_INVALID_ARG;
  if (d < 4 || d > kMaxD || d % 4 != 0 || (int64_t)B * L > kMaxKeys || (int64_t)H + Hk > 65535)
    return DARK_ERR_UNSUPPORTED;
  if (!gamma_ok(gamma_q, heads_gq, H) || !gamma_ok(gamma_k, heads_gk, Hk)) return DARK_ERR_INVALID_ARG;
  if ((gamma_q != nullptr || gamma_k != nullptr) && !(eps > 0.f && isfinite(eps)))
    return DARK_ERR_INVALID_ARG;
  if (rope != nullptr && (!rope_ok(rope) || rope->dims > d)) return DARK_ERR_INVALID_ARG;
  if (!aligned(positions, 4)) return DARK_ERR_INVALID_ARG;
  if (rope != nullptr) a.rope = *rope;
  a.dtype = dtype;
  a.eps = eps;
  a.B = B;
  a.L = L;
  a.d = d;
  a.positions = positions;
  a.pos0 = pos0;
  a.set[0].heads = H;
  a.set[0].gamma = gamma_q;
  a.set[0].gheads = heads_gq;
  a.set[0].rotate = 1;
  a.set[1].heads = Hk;
  a.set[1].gamma = Hk > 0 ? gamma_k : nullptr;
  a.set[1].gheads = heads_gk;
  a.set[1].rotate = 1;
  a.dev_status = dev_status;
  a.stream = (cudaStream_t)stream;
  return DARK_OK;
}

bool cache_ok(const dark_kv_cache* c) {
  return c != nullptr && c->k != nullptr && c->v != nullptr && c->k != c->v && dtype_ok(c->dtype) &&
         aligned(c->k, 16) && aligned(c->v, 16) && c->pages >= 1 && c->heads >= 1 &&
         c->page_size >= 1 && c->d >= 1;
}
bool cache_sizes_ok(const dark_kv_cache* c) {
  return c->d >= 4 && c->d <= kMaxD && c->d % 4 == 0 && c->heads <= 65535;
}

// Sizes of a cache-attention call that decide its workspace.
dark_status attention_sizes(dark::CacheAttnArgs& a, const dark_projection* proj,
                            const dark_kv_cache* c, int B, int H, int T, int prefix_len,
                            int max_pages) {
  memset(&a, 0, sizeof(a));
  if (proj == nullptr || proj->w == nullptr || !aligned(proj->w, 16) || !dtype_ok(proj->dtype) ||
      !cache_ok(c))
    return DARK_ERR_INVALID_ARG;
  if (proj->m < 1 || proj->r < 1 || proj->d < 1) return DARK_ERR_INVALID_ARG;
  if (proj->d != c->d || proj->dtype != c->dtype) return DARK_ERR_INVALID_ARG;
  if (B < 1 || H < 1 || T < 1 || prefix_len < 0 || max_pages < 1) return DARK_ERR_INVALID_ARG;
  if (!(proj->heads == 1 || proj->heads == H) || H % c->heads != 0) return DARK_ERR_INVALID_ARG;
  if (!cache_sizes_ok(c) || proj->m > kMaxM || proj->r > kMaxR) return DARK_ERR_UNSUPPORTED;
  // rows of all heads, keys of a list and the launches' grids stay inside 31 bits
  if ((int64_t)max_pages * c->page_size > kMaxKeys || prefix_len > kMaxKeys ||
      (int64_t)B * T > (1 << 20) || (int64_t)B * H * T > (1 << 24) || H > 65535)
    return DARK_ERR_UNSUPPORTED;
  a.heads_w = proj->heads;
  a.m = proj->m;
  a.r = proj->r;
  a.d = proj->d;
  a.dtype = proj->dtype;
  a.w = proj->w;
  a.kp = c->k;
  a.vp = c->v;
  a.pages = c->pages;
  a.Hk = c->heads;
  a.page = c->page_size;
  a.B = B;
  a.H = H;
  a.T = T;
  a.prefix_len = prefix_len;
  a.max_pages = max_pages;
  return DARK_OK;
}

}  // namespace

extern "C" {

dark_status dark_rope_init(dark_rope* rope, int dims, double base, double scale, int interleaved) {
  if (rope == nullptr || dims < 0 || dims > kMaxD || dims % 2 != 0) return DARK_ERR_INVALID_ARG;
  if (!(base > 0.0) || !isfinite(base) || !isfinite(scale)) return DARK_ERR_INVALID_ARG;
  memset(rope, 0, sizeof(*rope));
  rope->dims = dims;
  rope->interleaved = interleaved ? 1 : 0;
  const long double two_pi = 6.283185307179586476925286766559L;
  for (int i = 0; i < dims / 2; ++i) {
    const long double f = (long double)scale * powl((long double)base, -2.0L * i / dims) / two_pi;
    if (!isfinite((double)f)) return DARK_ERR_INVALID_ARG;
    // positions are whole numbers: whole turns a position change nothing
    long double part = f - floorl(f);
    part = floorl(part * 18446744073709551616.0L + 0.5L);
    rope->turns[i] = part >= 18446744073709551616.0L ? 0 : (uint64_t)part;
  }
  return DARK_OK;
}

dark_status dark_qk_norm_rope_fwd(const void* q, const int64_t* q_strides, const void* k,
                                  const int64_t* k_strides, void* q_out,
                                  const int64_t* q_out_strides, void* k_out,
                                  const int64_t* k_out_strides, const float* gamma_q, int heads_gq,
                                  const float* gamma_k, int heads_gk, float eps,
                                  const dark_rope* rope, const int32_t* positions, int64_t pos0,
                                  int B, int H, int Hk, int L, int d, dark_dtype dtype,
                                  int* dev_status, void* stream) {
  if (q == nullptr || q_out == nullptr) return DARK_ERR_INVALID_ARG;
  if (Hk > 0 && (k == nullptr || k_out == nullptr || k_out == q_out)) return DARK_ERR_INVALID_ARG;
  // a warp stores heads of q while it still fetches heads of k (and CTAs run in any order)
  if (Hk > 0 && (q_out == k || k_out == q)) return DARK_ERR_INVALID_ARG;
  dark::NormRopeArgs a;
  const dark_status st = norm_rope_args(a, gamma_q, heads_gq, gamma_k, heads_gk, eps, rope,
                                        positions, pos0, B, H, Hk, L, d, dtype, dev_status, stream);
  if (st != DARK_OK) return st;
  a.set[0].x = q;
  a.set[0].y = q_out;
  if (!aligned(q, elt(dtype)) || !aligned(q_out, elt(dtype)) ||
      !take_strides(a.set[0].xs, q_strides, B, H, L, d, false) ||
      !take_strides(a.set[0].ys, q_out_strides, B, H, L, d, true) ||
      !in_place_ok(q, a.set[0].xs, q_out, a.set[0].ys))
    return DARK_ERR_INVALID_ARG;
  if (Hk > 0) {
    a.set[1].x = k;
    a.set[1].y = k_out;
    if (!aligned(k, elt(dtype)) || !aligned(k_out, elt(dtype)) ||
        !take_strides(a.set[1].xs, k_strides, B, Hk, L, d, false) ||
        !take_strides(a.set[1].ys, k_out_strides, B, Hk, L, d, true) ||
        !in_place_ok(k, a.set[1].xs, k_out, a.set[1].ys))
      return DARK_ERR_INVALID_ARG;
  }
  return from_cuda(dark::launch_norm_rope(a));
}

size_t dark_qk_norm_rope_bwd_workspace_bytes(int B, int H, int Hk, int L, int d) {
  if (B < 1 || H < 1 || Hk < 0 || L < 1 || d < 4 || d > kMaxD || d % 4 != 0 ||
      (int64_t)B * L > kMaxKeys || (int64_t)H + Hk > 65535)
    return 0;
  return dark::norm_rope_bwd_workspace_bytes(B, H, Hk, L, d);
}

dark_status dark_qk_norm_rope_bwd(const void* q, const int64_t* q_strides, const void* k,
                                  const int64_t* k_strides, const void* dq_out,
                                  const int64_t* dq_out_strides, const void* dk_out,
                                  const int64_t* dk_out_strides, void* dq,
                                  const int64_t* dq_strides, void* dk, const int64_t* dk_strides,
                                  const float* gamma_q, int heads_gq, const float* gamma_k,
                                  int heads_gk, float* dgamma_q, float* dgamma_k, float eps,
                                  const dark_rope* rope, const int32_t* positions, int64_t pos0,
                                  int B, int H, int Hk, int L, int d, dark_dtype dtype, void* ws,
                                  size_t ws_bytes, int* dev_status, void* stream) {
  if (q == nullptr || dq_out == nullptr || dq == nullptr || ws == nullptr || !aligned(ws, 256))
    return DARK_ERR_INVALID_ARG;
  if (Hk > 0 && (k == nullptr || dk_out == nullptr || dk == nullptr || dk == dq))
    return DARK_ERR_INVALID_ARG;
  if (Hk > 0 && (dq == k || dq == dk_out || dk == q || dk == dq_out)) return DARK_ERR_INVALID_ARG;
  dark::NormRopeArgs a;
  const dark_status st = norm_rope_args(a, gamma_q, heads_gq, gamma_k, heads_gk, eps, rope,
                                        positions, pos0, B, H, Hk, L, d, dtype, dev_status, stream);
  if (st != DARK_OK) return st;
  // a weight and its gradient come together
  if ((gamma_q == nullptr) != (dgamma_q == nullptr) || !aligned(dgamma_q, 4)) return DARK_ERR_INVALID_ARG;
  if (Hk <= 0 && dgamma_k != nullptr) return DARK_ERR_INVALID_ARG;       // nothing would write it
  if (Hk > 0 && (((gamma_k == nullptr) != (dgamma_k == nullptr)) || !aligned(dgamma_k, 4) ||
                 (dgamma_k != nullptr && dgamma_k == dgamma_q)))
    return DARK_ERR_INVALID_ARG;
  if (ws_bytes < dark_qk_norm_rope_bwd_workspace_bytes(B, H, Hk, L, d)) return DARK_ERR_INVALID_ARG;
  a.part = (float*)((char*)ws + dark::kWsHeader);
  const size_t e = elt(dtype);
  a.set[0].x = q;
  a.set[0].g = dq_out;
  a.set[0].y = dq;
  a.set[0].dgamma = dgamma_q;
  if (!aligned(q, e) || !aligned(dq_out, e) || !aligned(dq, e) ||
      !take_strides(a.set[0].xs, q_strides, B, H, L, d, false) ||
      !take_strides(a.set[0].gs, dq_out_strides, B, H, L, d, false) ||
      !take_strides(a.set[0].ys, dq_strides, B, H, L, d, true) ||
      !in_place_ok(dq_out, a.set[0].gs, dq, a.set[0].ys) ||
      !in_place_ok(q, a.set[0].xs, dq, a.set[0].ys))
    return DARK_ERR_INVALID_ARG;
  if (Hk > 0) {
    a.set[1].x = k;
    a.set[1].g = dk_out;
    a.set[1].y = dk;
    a.set[1].dgamma = dgamma_k;
    if (!aligned(k, e) || !aligned(dk_out, e) || !aligned(dk, e) ||
        !take_strides(a.set[1].xs, k_strides, B, Hk, L, d, false) ||
        !take_strides(a.set[1].gs, dk_out_strides, B, Hk, L, d, false) ||
        !take_strides(a.set[1].ys, dk_strides, B, Hk, L, d, true) ||
        !in_place_ok(dk_out, a.set[1].gs, dk, a.set[1].ys) ||
        !in_place_ok(k, a.set[1].xs, dk, a.set[1].ys))
      return DARK_ERR_INVALID_ARG;
  }
  return from_cuda(dark::launch_norm_rope_bwd(a));
}

dark_status dark_kv_append(const dark_kv_cache* cache, const void* k, const int64_t* k_strides,
                           const void* v, const int64_t* v_strides, int B, int T,
                           const int32_t* page_table, int max_pages, const int32_t* lens,
                           const int32_t* new_lens, const float* gamma_k, int heads_gk, float eps,
                           const dark_rope* rope, const int32_t* positions, int64_t pos0,
                           int* dev_status, void* stream) {
  if (!cache_ok(cache) || k == nullptr || v == nullptr || page_table == nullptr || lens == nullptr ||
      max_pages < 1)
    return DARK_ERR_INVALID_ARG;
  if (!aligned(page_table, 4) || !aligned(lens, 4) || !aligned(new_lens, 4)) return DARK_ERR_INVALID_ARG;
  const int Hk = cache->heads, d = cache->d;
  if (!cache_sizes_ok(cache) || (int64_t)max_pages * cache->page_size > kMaxKeys)
    return DARK_ERR_UNSUPPORTED;
  dark::NormRopeArgs a;
  const dark_status st = norm_rope_args(a, gamma_k, heads_gk, nullptr, 1, eps, rope, positions, pos0,
                                        B, Hk, Hk, T, d, cache->dtype, dev_status, stream);
  if (st != DARK_OK) return st;
  const size_t e = elt(cache->dtype);
  a.set[0].x = k;
  a.set[0].y = cache->k;
  a.set[1].x = v;
  a.set[1].y = cache->v;
  a.set[1].rotate = 0;
  if (!aligned(k, e) || !aligned(v, e) || !take_strides(a.set[0].xs, k_strides, B, Hk, T, d, false) ||
      !take_strides(a.set[1].xs, v_strides, B, Hk, T, d, false))
    return DARK_ERR_INVALID_ARG;
  a.lens = lens;
  a.new_lens = new_lens;
  a.table = page_table;
  a.max_pages = max_pages;
  a.pages = cache->pages;
  a.page = cache->page_size;
  return from_cuda(dark::launch_norm_rope(a));
}

size_t dark_cache_attention_workspace_bytes(const dark_projection* proj, const dark_kv_cache* cache,
                                            int B, int H, int T, int prefix_len, int max_pages) {
  dark::CacheAttnArgs a;
  if (attention_sizes(a, proj, cache, B, H, T, prefix_len, max_pages) != DARK_OK) return 0;
  return dark::cache_attention_workspace_bytes(a);
}

dark_status dark_cache_attention_fwd(const dark_projection* proj, const dark_kv_cache* cache,
                                     const void* q, const int64_t* q_strides, void* out,
                                     const int64_t* out_strides, int B, int H, int T,
                                     const int32_t* prefix_pages, int prefix_len,
                                     const int32_t* page_table, int max_pages, const int32_t* lens,
                                     int flags, void* ws, size_t ws_bytes, int* dev_status,
                                     void* stream) {
  dark::CacheAttnArgs a;
  const dark_status st = attention_sizes(a, proj, cache, B, H, T, prefix_len, max_pages);
  if (st != DARK_OK) return st;
  if (q == nullptr || out == nullptr || page_table == nullptr || lens == nullptr ||
      (prefix_len > 0 && prefix_pages == nullptr))
    return DARK_ERR_INVALID_ARG;
  if (flags & ~(DARK_CAUSAL | DARK_EXACT)) return DARK_ERR_INVALID_ARG;
  const size_t e = elt(proj->dtype);
  if (!aligned(q, e) || !aligned(out, e) || !aligned(page_table, 4) || !aligned(lens, 4) ||
      !aligned(prefix_pages, 4) || !take_strides(a.qs, q_strides, B, H, T, a.d, false) ||
      !take_strides(a.os, out_strides, B, H, T, a.d, true))
    return DARK_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned(ws, 256) || ws_bytes < dark::cache_attention_workspace_bytes(a))
    return DARK_ERR_INVALID_ARG;
  a.q = q;
  a.out = out;
  a.prefix_pages = prefix_pages;
  a.table = page_table;
  a.lens = lens;
  a.flags = flags;
  a.ws = ws;
  a.dev_status = dev_status;
  a.stream = (cudaStream_t)stream;
  return from_cuda(dark::launch_cache_attention(a));
}

}  // extern "C"
