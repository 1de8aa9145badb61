// Attention of new tokens over the paged cache (lora_paged_attention);
// include/lora_gb300.h is the contract.
//
// One warp per (token, query head): each lane holds head_dim / 32 features of q and of
// the running output, and the warp walks the visible positions with an online softmax.
#include "serve.cuh"

namespace lgb {

struct AttnParams {
  HeadsView q;
  int hq, group;
  long long M;
  CacheArgs cache;
  const int* table;
  long long max_pages;
  const int* kv_len;
  const int* cu_q;
  int n_seqs;
  float scale;
  int causal;
  long long window;
  bf16* out;
  float* lse;
  unsigned* status;
};

template <int D, int FMT>
__device__ __forceinline__ void load_features(const void* base, const float* scales, long long row, int lane,
                                              float (&x)[D / 32]) {
  const float scale = FMT == LORA_KV_BF16 ? 1.0f : __ldg(scales + row);
#pragma unroll
  for (int e = 0; e < D / 32; ++e) {
    const long long at = row * D + e * 32 + lane;
    if (FMT == LORA_KV_BF16)
      x[e] = __bfloat162float(static_cast<const bf16*>(base)[at]);
    else if (FMT == LORA_KV_INT8)
      x[e] = scale * static_cast<float>(static_cast<const int8_t*>(base)[at]);
    else
      x[e] = scale * __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(base)[at], __NV_E4M3)));
  }
}

template <int D, int FMT>
__global__ void __launch_bounds__(256) paged_attn_kernel(const __grid_constant__ AttnParams p) {
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < p.n_seqs; b += 256) {
      const int q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1);
      if (q0 < 0 || q1 < q0 || q1 > p.M) atomicOr(p.status, kStatusInput);
    }
  const int lane = threadIdx.x & 31;
  const long long warps = static_cast<long long>(gridDim.x) * 8;
  for (long long w = blockIdx.x * 8ll + (threadIdx.x >> 5); w < p.M * p.hq; w += warps) {
    const long long m = w / p.hq;
    const int h = static_cast<int>(w - m * p.hq);
    const int b = owner_of(p.cu_q, p.n_seqs, m);
    if (b < 0) continue;
    const long long q0 = max(0, __ldg(p.cu_q + b)), q1 = min(static_cast<long long>(__ldg(p.cu_q + b + 1)), p.M);
    long long kv = __ldg(p.kv_len + b);
    const long long most = p.max_pages << p.cache.page_shift;
    if (kv < 0 || kv > most) {
      atomicOr(p.status, kStatusInput);
      kv = kv < 0 ? 0 : most;
    }
    const long long pos = kv - (q1 - q0) + (m - q0);
    const long long hi = p.causal ? min(kv, pos + 1) : kv;
    const long long lo = p.window > 0 ? max(0ll, pos - p.window + 1) : 0;
    float q[D / 32], o[D / 32] = {};
    const bf16* qr = p.q.x + m * p.q.ts + h * p.q.hs;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) q[e] = __bfloat162float(qr[e * 32 + lane]);
    float top = -INFINITY, sum = 0.0f;
    for (long long j = lo; j < hi; ++j) {
      long long page = __ldg(p.table + b * p.max_pages + (j >> p.cache.page_shift));
      if (page < 0 || page >= p.cache.n_pages) {
        atomicOr(p.status, kStatusInput);
        page = 0;
      }
      const long long row = ((page * p.cache.heads + h / p.group) << p.cache.page_shift) +
                            (j & ((1 << p.cache.page_shift) - 1));
      float x[D / 32];
      load_features<D, FMT>(p.cache.k, p.cache.ks, row, lane, x);
      float s = 0.0f;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) s += q[e] * x[e];
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      s *= p.scale;
      const float next = fmaxf(top, s);
      const float old = top == -INFINITY ? 0.0f : __expf(top - next);
      const float wgt = __expf(s - next);
      load_features<D, FMT>(p.cache.v, p.cache.vs, row, lane, x);
#pragma unroll
      for (int e = 0; e < D / 32; ++e) o[e] = o[e] * old + wgt * x[e];
      sum = sum * old + wgt;
      top = next;
    }
    bf16* out = p.out + (m * p.hq + h) * D;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) out[e * 32 + lane] = __float2bfloat16_rn(hi > lo ? o[e] / sum : 0.0f);
    if (p.lse != nullptr && lane == 0) p.lse[m * p.hq + h] = hi > lo ? top + __logf(sum) : -INFINITY;
  }
}

typedef void (*AttnKernel)(const AttnParams);
template <int D>
static AttnKernel attn_of(int fmt) {
  return fmt == LORA_KV_BF16 ? paged_attn_kernel<D, LORA_KV_BF16>
                             : fmt == LORA_KV_FP8 ? paged_attn_kernel<D, LORA_KV_FP8>
                                                  : paged_attn_kernel<D, LORA_KV_INT8>;
}

}  // namespace lgb

using namespace lgb;

extern "C" size_t lora_paged_attention_workspace_bytes(int64_t M, int64_t n_seqs, int heads_q,
                                                       const lora_kv_cache_t* cache) {
  if (M < 0 || M > kMaxExtent || n_seqs < 1 || n_seqs > kMaxExtent || heads_q < 1 || check_cache(cache) != LORA_OK ||
      heads_q % cache->heads)
    return 0;
  return kWsHeader;
}

extern "C" lora_status_t lora_paged_attention(int64_t M, int heads_q, const lora_heads_t* q,
                                              const lora_kv_cache_t* cache, const lora_paged_batch_t* batch,
                                              float scale, int causal, int64_t window, void* out, float* lse, void* ws,
                                              size_t ws_bytes, cudaStream_t stream) {
  NvtxRange nvtx_range("lora_paged_attention");
  if (M < 0 || !q || (M > 0 && (!q->data || !out)) || !batch || !batch->page_table || !batch->kv_len ||
      !batch->cu_q || batch->n_seqs < 1 || batch->max_pages < 1 || window < 0 || !std::isfinite(scale))
    return LORA_ERR_INVALID_ARG;
  LGB_TRY(check_cache(cache));
  if (heads_q < 1 || heads_q % cache->heads || q->heads != heads_q) return LORA_ERR_INVALID_ARG;
  if (M > kMaxExtent || batch->n_seqs > kMaxExtent || batch->max_pages > kMaxExtent / cache->page_size)
    return LORA_ERR_UNSUPPORTED;
  LGB_TRY(check_heads_in(q));
  if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(batch->page_table, 4) || !aligned(batch->kv_len, 4) ||
      !aligned(batch->cu_q, 4))
    return LORA_ERR_ALIGNMENT;
  LGB_TRY(check_ws(ws, ws_bytes, lora_paged_attention_workspace_bytes(M, batch->n_seqs, heads_q, cache)));
  if (M == 0) return LORA_OK;
  AttnParams p;
  p.q = HeadsView{static_cast<const bf16*>(q->data), q->token_stride, q->head_stride};
  p.hq = heads_q;
  p.group = heads_q / cache->heads;
  p.M = M;
  p.cache = cache_args(cache);
  p.table = batch->page_table;
  p.max_pages = batch->max_pages;
  p.kv_len = batch->kv_len;
  p.cu_q = batch->cu_q;
  p.n_seqs = static_cast<int>(batch->n_seqs);
  p.scale = scale;
  p.causal = causal != 0;
  p.window = window;
  p.out = static_cast<bf16*>(out);
  p.lse = lse;
  p.status = static_cast<unsigned*>(ws);
  const int D = cache->head_dim;
  const AttnKernel f = D == 64 ? attn_of<64>(cache->format) : D == 128 ? attn_of<128>(cache->format)
                                                                      : attn_of<256>(cache->format);
  const int64_t blocks = ceil_div(M * heads_q, 8);
  return launch_counted(f, dim3(static_cast<unsigned>(blocks < 65535 ? blocks : 65535)), dim3(256), 0, LORA_KIND_ATTN,
                        stream, p);
}
