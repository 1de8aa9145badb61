// Declarations shared by the serving operators (rotary.cu, kv_cache.cu, paged_attn*.cu):
// views of heads, the cache as the kernels see it, the argument rules, and the device
// arithmetic they have in common.
#pragma once

#include <cuda_fp8.h>

#include "api_internal.cuh"

namespace lgb {

// A view [tokens x heads x head_dim] of bf16.
struct HeadsView {
  const bf16* x;
  long long ts, hs;
};
struct HeadsOut {
  bf16* y;
  long long ts, hs;
};

struct RotaryArgs {
  const float* cos;
  const float* sin;
  const int* pos;
  int npos;
  int half;
};

struct CacheArgs {
  void* k;
  void* v;
  float* ks;
  float* vs;
  long long n_pages;
  int page_shift;            // page_size = 1 << page_shift
  int heads;
};

inline lora_status_t check_heads_in(const lora_heads_t* h) {
  if (h->heads < 1 || h->token_stride < 0 || h->head_stride < 0) return LORA_ERR_INVALID_ARG;
  if (h->heads > 65535) return LORA_ERR_UNSUPPORTED;
  if (!aligned(h->data, 16) || h->token_stride % 8 || h->head_stride % 8) return LORA_ERR_ALIGNMENT;
  return LORA_OK;
}
// Rows must not overlap: one of the two strides steps over everything the other spans.
inline lora_status_t check_heads_out(const lora_heads_t* h, int64_t M, int head_dim) {
  LGB_TRY(check_heads_in(h));
  const int64_t ts = h->token_stride, hs = h->head_stride;
  const bool heads_apart = h->heads == 1 || hs >= head_dim, tokens_apart = M <= 1 || ts >= head_dim;
  const bool nested = h->heads == 1 || M <= 1 || ts >= (h->heads - 1) * hs + head_dim || hs >= (M - 1) * ts + head_dim;
  return heads_apart && tokens_apart && nested ? LORA_OK : LORA_ERR_INVALID_ARG;
}
inline lora_status_t check_rotary(const lora_rotary_t* r, int head_dim) {
  if (!r->cos || !r->sin || r->n_pos < 1 || r->rot_dim < 2 || r->rot_dim % 2 || r->rot_dim > head_dim ||
      (r->layout != LORA_ROTARY_HALF && r->layout != LORA_ROTARY_INTERLEAVED))
    return LORA_ERR_INVALID_ARG;
  if (r->n_pos > kMaxExtent) return LORA_ERR_UNSUPPORTED;
  if (!aligned(r->cos, 16) || !aligned(r->sin, 16) || !aligned(r->pos, 4)) return LORA_ERR_ALIGNMENT;
  return LORA_OK;
}
inline lora_status_t check_cache(const lora_kv_cache_t* c) {
  if (!c || !c->k || !c->v || c->n_pages < 1 || c->heads < 1 || c->format < LORA_KV_BF16 || c->format > LORA_KV_INT8)
    return LORA_ERR_INVALID_ARG;
  if (c->format != LORA_KV_BF16 && (!c->k_scale || !c->v_scale)) return LORA_ERR_INVALID_ARG;
  const int ps = c->page_size, d = c->head_dim;
  if (ps < 16 || ps > 256 || (ps & (ps - 1)) || (d != 64 && d != 128 && d != 256)) return LORA_ERR_UNSUPPORTED;
  if (c->heads > 65535 || c->n_pages > kMaxExtent / (static_cast<int64_t>(c->heads) * ps)) return LORA_ERR_UNSUPPORTED;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))
    return LORA_ERR_ALIGNMENT;
  return LORA_OK;
}
inline lora_status_t check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (!ws) return LORA_ERR_INVALID_ARG;
  if (!aligned(ws, 256)) return LORA_ERR_ALIGNMENT;
  return ws_bytes < need ? LORA_ERR_WORKSPACE : LORA_OK;
}
inline RotaryArgs rotary_args(const lora_rotary_t* r) {
  return RotaryArgs{r->cos, r->sin, r->pos, static_cast<int>(r->n_pos), r->rot_dim / 2};
}
inline CacheArgs cache_args(const lora_kv_cache_t* c) {
  int shift = 4;
  while ((1 << shift) < c->page_size) ++shift;
  return CacheArgs{c->k, c->v, c->k_scale, c->v_scale, c->n_pages, shift, c->heads};
}

// Heads each thread group (of `lanes` threads) walks: up to eight, as many as leave the GPU
// some two rounds of its resident threads, so that the last round's idle part is small;
// the table entries of a token are loaded once for them.  kHeadBatch: heads whose loads the
// cache kernels issue together.
constexpr int kHeadBatch = 4;
inline int heads_per_group(int64_t M, int lanes, int heads) {
  const int64_t want = static_cast<int64_t>(num_sms()) * 2048 * 2;     // threads
  int hp = 8;
  while (hp > 1 && M * lanes * ceil_div(heads, hp) < want) hp >>= 1;
  return hp;
}

// ---------------------------------------------------------------- device arithmetic

__device__ __forceinline__ int checked_position(const RotaryArgs& r, int pos, unsigned* status) {
  if (pos >= 0 && pos < r.npos) return pos;
  atomicOr(status, kStatusInput);
  return 0;
}
// a cos - b sin and b cos + a sin with every product and sum rounded on its own: no
// contraction, so the value does not depend on which of the two products is fused.
__device__ __forceinline__ void turn(float a, float b, float c, float s, float& ya, float& yb) {
  ya = __fadd_rn(__fmul_rn(a, c), -__fmul_rn(b, s));
  yb = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}
__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(v[e] << 16);
    x[2 * e + 1] = __uint_as_float(v[e] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void load8f(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// The sequence that owns row r: the last b with cu[b] <= r, or -1 where none does.
__device__ __forceinline__ int owner_of(const int* cu, int n, long long r) {
  if (r < __ldg(cu) || r >= __ldg(cu + n)) return -1;
  int lo = 0, hi = n;                       // cu[lo] <= r < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid) <= r) lo = mid; else hi = mid;
  }
  return lo;
}

}  // namespace lgb
