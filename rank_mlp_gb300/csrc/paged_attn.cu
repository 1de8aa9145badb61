// lora_paged_attention: arguments, workspace and the choice of kernel;
// include/lora_gb300.h is the contract, paged_attn.cuh says how the work is shared out.
#include "paged_attn.cuh"

namespace lgb {

// Which kernel: the one whose tiles the rows fill.  A call's lengths are on the device, so
// the rule takes the mean number of query rows that share a cache head.  Returns the row
// halves of the tcgen05 kernel, or 0 for the few-row kernel.  Measured with 64 sequences of
// 4096 positions, eight cache heads of 128 features (us, single calls on cold caches):
//   rows of a cache head        4    16    20   128   132   256
//   bf16  few-row kernel      186   188   341  1265  1405  2490
//         one row half        186   188   190   199   353   359
//         two row halves      191   195   197   209   227   238
//   fp8   few-row kernel      151   156   281  1067  1195  2103
//         one row half        261   281   282   291   525   550
//         two row halves      264   275   275   285   338   353
// (bf16 with few rows: either; the few-row kernel keeps more bits of the weights.)  The mean
// counts idle sequences too, so a chunk among many of them, or among many single tokens, can
// go to the few-row kernel: right, but slower by the columns to the right.
// head_dim 256 has one half: two outputs would fill the tensor memory.
static int row_halves(int64_t M, int64_t n_seqs, int group, int head_dim) {
  if (M * group <= kFewRows * n_seqs) return 0;
  return head_dim == 256 || M * group <= 128 * n_seqs ? 1 : 2;
}

// Workspace: header, the parts' descriptors, maxima and sums, outputs.  It is the same for
// every call over a cache, that of the kernel with the larger tiles: a decode step that a
// graph has recorded and the prefills between its replays share one workspace.
static int largest_halves(int head_dim) { return head_dim == 256 ? 1 : 2; }
static void carve_parts(Carve& c, int halves, int head_dim, AttnParams& p) {
  const int64_t ctas = halves ? kMaxManyCtas : kMaxFewCtas, rows = 2 * ctas * (halves ? 128 * halves : kFewRows);
  c.take(kWsHeader);
  p.join = c.take_n<JoinDesc>(ctas);
  p.part_ml = c.take_n<float2>(rows);
  p.part_o = c.take_n<float>(rows * head_dim);
}

}  // namespace lgb

using namespace lgb;

extern "C" size_t lora_paged_attention_workspace_bytes(int64_t M, int64_t n_seqs, int heads_q,
                                                       const lora_kv_cache_t* cache) {
  if (M < 0 || n_seqs < 1 || n_seqs > kMaxExtent || heads_q < 1 || M > kMaxExtent / heads_q || check_cache(cache) != LORA_OK ||
      heads_q % cache->heads)
    return 0;
  AttnParams p;
  Carve c(nullptr);
  carve_parts(c, largest_halves(cache->head_dim), cache->head_dim, p);
  return c.off;
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
  if (M > kMaxExtent / heads_q || batch->n_seqs > kMaxExtent || batch->max_pages > kMaxExtent / cache->page_size)
    return LORA_ERR_UNSUPPORTED;
  LGB_TRY(check_heads_in(q));
  if ((M > 1 && q->token_stride == 0) || (heads_q > 1 && q->head_stride == 0)) return LORA_ERR_UNSUPPORTED;
  if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(batch->page_table, 4) || !aligned(batch->kv_len, 4) ||
      !aligned(batch->cu_q, 4))
    return LORA_ERR_ALIGNMENT;
  LGB_TRY(check_ws(ws, ws_bytes, lora_paged_attention_workspace_bytes(M, batch->n_seqs, heads_q, cache)));
  if (M == 0) return LORA_OK;
  AttnParams p;
  std::memset(static_cast<void*>(&p), 0, sizeof(p));
  // the stride of an extent of one is never taken; the tensor map wants one all the same
  p.q = HeadsView{static_cast<const bf16*>(q->data), M > 1 ? q->token_stride : 8, heads_q > 1 ? q->head_stride : 8};
  p.hq = heads_q;
  p.group = heads_q / cache->heads;
  p.M = static_cast<int>(M);
  p.cache = cache_args(cache);
  p.table = batch->page_table;
  p.max_pages = batch->max_pages;
  p.kv_len = batch->kv_len;
  p.cu_q = batch->cu_q;
  p.n_seqs = static_cast<int>(batch->n_seqs);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.causal = causal != 0;
  p.window = window > kMaxExtent ? 0 : static_cast<int>(window);
  p.out = static_cast<bf16*>(out);
  p.lse = lse;
  p.status = static_cast<unsigned*>(ws);
  p.timeout_ns = wait_timeout_ns();
  p.inject_stall = take_expiry();
  Carve c(ws);
  const int halves = row_halves(M, batch->n_seqs, p.group, cache->head_dim);
  carve_parts(c, halves, cache->head_dim, p);        // (never more than the largest)
  return halves ? launch_attn_many(p, halves, cache->head_dim, cache->format, stream)
                : launch_attn_few(p, cache->head_dim, cache->format, stream);
}
