/*
 * lora_gb300.h -- C ABI of the GB300 (sm_103a) LoRA block-projection library.
 *
 * What is computed
 * ----------------
 * A LoRA linear with frozen base weight W [out x in] and adapter A [r x in],
 * B [out x r], scale s:
 *
 *     y = x W^T + s (x A^T) B^T                                               (1)
 *
 * ("Model Patches and Kernels", opake user guide, section "Fused LoRA operations",
 * row opake_lora_w: x @ W.T + x @ A @ B * s, written here in the PEFT layout with
 * A stored [r x in] and B stored [out x r]; s = alpha / r.)
 *
 * The gated MLP (same section, row opake_lora_mlp: gate + up + activation + down in
 * one call; activations from the same page, "Activation functions" table):
 *
 *     g = (1) with gate,  u = (1) with up,  h = act(g) * u,  y = (1) of h with down
 *     act = silu (SwiGLU), or GELU (GeGLU): exact (erf) or its tanh approximation
 *
 * The attention projections (row opake_lora_qkv: q, k, v share the input x; the
 * axolotl "monkeypatch.lora_kernels" reference, original_apply_qkv returning
 * (query, key, value) and original_apply_o for the output projection): q, k, v and
 * o are each (1); o's input is the attention output, which this library does not
 * compute.
 *
 * Backward computes the gradient of <dy, y> with respect to x and every A and B.
 * W is frozen and gets no gradient ("Model Patches and Kernels", section "Fused
 * linear cross-entropy": a frozen weight's gradient is skipped).  Adapters have no
 * dropout and no bias (axolotl apply_lora_kernel_patches note; MLP fusion is
 * bias-free per opake).
 *
 * Conventions (all entry points)
 * ------------------------------
 * - Tensors are bf16, row-major, dense (row stride = number of columns), in device
 *   memory, token-major for activations: x [M x in], y [M x out]; M = batch * seq.
 *   W [out x in], A [r x in], B [out x r], dA [r x in], dB [out x r].
 * - The caller owns and allocates every buffer, including `saved` and `ws`; the
 *   library allocates no memory and never synchronises (lora_poll_status and
 *   lora_trace_read aside).  All work is enqueued on `stream`, in order.  Kernels are
 *   launched with programmatic dependent launch (each waits for the previous work on
 *   the stream before it touches memory; environment LORA_PDL=0 turns the attribute
 *   off), so stream order holds as usual for the caller's own work around the calls.
 * - Gradient outputs (dx, dA, dB) are overwritten, not accumulated.
 * - Alignment: every pointer 16-byte aligned (`ws` and `saved` 256-byte aligned);
 *   every feature size (in, out, h, i, n_q, n_kv) a multiple of 8.  A and B need no
 *   alignment beyond their element size.  Violations return LORA_ERR_ALIGNMENT.
 * - Rank limits: 1 <= r, and (number of adapters sharing one input) * r <= 256,
 *   i.e. r <= 128 for the MLP's gate/up pair and r <= 85 for q/k/v; otherwise
 *   LORA_ERR_UNSUPPORTED.  Size limits: M and every feature size at most 2^31 - 1
 *   (32-bit row, column and tile indices); otherwise LORA_ERR_UNSUPPORTED.
 * - Every argument error returns before anything is enqueued.  No entry point
 *   aborts, throws or prints.
 * - `ws` must hold lora_*_workspace_bytes(...) bytes; its first 256 bytes hold the
 *   status word that kernels set asynchronously (zero them before first use;
 *   lora_poll_status reads and clears it).  `saved` must hold lora_*_saved_bytes(...)
 *   and is an opaque blob written by forward and read by backward.
 * - M == 0 is allowed: forward enqueues nothing, backward zero-fills dA and dB.
 * - Calls that share a `ws` must not overlap on the GPU (same stream is safe).
 */
#ifndef LORA_GB300_H
#define LORA_GB300_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  LORA_ACT_SWIGLU = 0,      /* silu(g) * u */
  LORA_ACT_GEGLU_TANH = 1,  /* gelu_tanh(g) * u, 0.5 g (1 + tanh(sqrt(2/pi)(g + 0.044715 g^3))) */
  LORA_ACT_GEGLU_ERF = 2    /* gelu(g) * u, 0.5 g (1 + erf(g / sqrt 2)) */
} lora_act_t;

typedef enum {
  LORA_OK = 0,
  LORA_ERR_INVALID_ARG = 1,   /* NULL pointer, negative size, bad enum, non-finite s */
  LORA_ERR_ALIGNMENT = 2,     /* pointer or feature size violates the alignment rules */
  LORA_ERR_UNSUPPORTED = 3,   /* rank or size beyond the limits above */
  LORA_ERR_WORKSPACE = 4,     /* ws_bytes below the workspace query */
  LORA_ERR_CUDA = 5,          /* a CUDA runtime call or kernel launch failed */
  LORA_ERR_TIMEOUT = 6,       /* a kernel's bounded wait expired (read by lora_poll_status) */
  LORA_ERR_DEVICE_INPUT = 7   /* a value in device memory was out of range: a RoPE position
                                 outside [0, n_pos) (position 0 was used in its place), or a
                                 cache slot, page or length (see those calls); read by
                                 lora_poll_status */
} lora_status_t;

/* One frozen base weight and its adapter: device pointers, bf16, row-major.
 * W [out x in], A [r x in], B [out x r]. */
typedef struct {
  const void* W;
  const void* A;
  const void* B;
} lora_linear_t;

/* Gradient outputs of one adapter: dA [r x in], dB [out x r], bf16, overwritten. */
typedef struct {
  void* dA;
  void* dB;
} lora_grads_t;

/* ---------------------------------------------------------------- single linear
 * (1) for one projection ("opake_lora_w").  saved holds the rank-r projection x A^T
 * and the adapter packed for backward; pass NULL for inference. */
size_t lora_linear_saved_bytes(int64_t M, int64_t in, int64_t out, int r);
size_t lora_linear_workspace_bytes(int64_t M, int64_t in, int64_t out, int r);
lora_status_t lora_linear_forward(int64_t M, int64_t in, int64_t out, int r, float s,
                                  const void* x, lora_linear_t lin, void* y, void* saved,
                                  void* ws, size_t ws_bytes, cudaStream_t stream);
/* dx [M x in] = dy W + s (dy B) A;  dA = s (dy B)^T x;  dB = s dy^T (x A^T).
 * x is the forward input again; saved is what forward wrote, including the adapter
 * packed as this call's operands (with the forward's s): lin must be the forward's
 * (its W is read here, its A and B only checked), and s the same, as autograd uses the
 * tensors a forward saved. */
lora_status_t lora_linear_backward(int64_t M, int64_t in, int64_t out, int r, float s,
                                   const void* x, lora_linear_t lin, const void* saved,
                                   const void* dy, void* dx, lora_grads_t grads,
                                   void* ws, size_t ws_bytes, cudaStream_t stream);

/* Forward of the single linear (inference: nothing is saved) that allocates nothing
 * and takes no workspace.  The pages have no counterpart; it exists for callers that
 * cannot allocate device memory where they run this projection -- a plugin inside a
 * host framework that owns all device memory and passes the plugin only its input and
 * output buffers, or a latency-critical loop that must never call cudaMalloc (which
 * can synchronise the device).  Scratch comes from a fixed 32 MiB array inside the
 * library, which every GPU that loads the library holds until the process exits.
 * - Problems whose forward needs more than 32 MiB of scratch (the forward's share of
 *   lora_linear_workspace_bytes(M, in, out, r), which also counts the backward's) are
 *   rejected with LORA_ERR_WORKSPACE before anything is enqueued; other argument rules
 *   are those of lora_linear_forward with saved == NULL, and so is the result, up to
 *   the order of the f32 sums (this call always gives each 256 x 256 output tile to
 *   one CTA pair).
 * - Asynchronous errors (an expired bounded wait) set the status word at the front of
 *   the array; lora_poll_status(NULL, stream) reads and clears it.  It stays set across
 *   calls until polled.
 * - The first call on a device, and the first after the device's context was
 *   destroyed and created again (cudaDeviceReset), looks up the array's device address;
 *   make that first call before any stream capture.
 * - Every call on a device shares the one array and leaves its contents behind; calls
 *   whose GPU work overlaps (other streams, other threads) race and corrupt each
 *   other's results.  Calls in order on one stream are safe. */
lora_status_t lora_linear_forward_noalloc(int64_t M, int64_t in, int64_t out, int r, float s,
                                          const void* x, lora_linear_t lin, void* y,
                                          cudaStream_t stream);

/* ---------------------------------------------------------------- gated MLP
 * x [M x h] -> y [M x h] through gate/up [i x h] and down [h x i] ("opake_lora_mlp").
 * saved (NULL for inference) receives g, u, h and the rank-r projections for
 * backward (x [A_g; A_u]^T also transposed, for the backward's single pass over dg, du
 * when r <= 16), and the adapters packed as the backward's operands. */
size_t lora_mlp_saved_bytes(int64_t M, int64_t h, int64_t i, int r);
size_t lora_mlp_workspace_bytes(int64_t M, int64_t h, int64_t i, int r);
lora_status_t lora_mlp_forward(int64_t M, int64_t h, int64_t i, int r, float s, lora_act_t act,
                               const void* x, lora_linear_t gate, lora_linear_t up,
                               lora_linear_t down, void* y, void* saved,
                               void* ws, size_t ws_bytes, cudaStream_t stream);
/* Gradients of <dy, y>: dx [M x h] and dA/dB of gate, up and down.  Needs the
 * forward's x and saved blob (the activation and its derivative are recomputed from
 * the saved g, u).  The adapters enter as the forward packed them into saved (with its
 * s), as autograd uses the tensors a forward saved: gate, up and down must be the
 * forward's (their W is read here; their A and B only checked), and s the same. */
lora_status_t lora_mlp_backward(int64_t M, int64_t h, int64_t i, int r, float s, lora_act_t act,
                                const void* x, lora_linear_t gate, lora_linear_t up,
                                lora_linear_t down, const void* saved, const void* dy,
                                void* dx, lora_grads_t d_gate, lora_grads_t d_up,
                                lora_grads_t d_down, void* ws, size_t ws_bytes,
                                cudaStream_t stream);

/* Per-example adapter gradients, for DP-SGD (the opake use case: per-example
 * gradients by vmap(grad) before clipping; "Model Patches and Kernels").  The M tokens
 * are n_examples examples of seq = M / n_examples consecutive tokens (M must be a
 * multiple of n_examples; token t belongs to example t / seq).  Writes dx as
 * lora_mlp_backward does, and for each adapter the gradient of every example on its
 * own: d_*.dA [n_examples x r x in], d_*.dB [n_examples x out x r] (bf16, example-major).
 * sq_norms (NULL or float [n_examples]) receives each example's squared L2 norm over
 * all six adapter gradients, summed from the bf16 results in a fixed order.  ws must
 * hold lora_mlp_per_example_workspace_bytes(M, h, i, r, n_examples). */
size_t lora_mlp_per_example_workspace_bytes(int64_t M, int64_t h, int64_t i, int r, int64_t n_examples);
lora_status_t lora_mlp_backward_per_example(int64_t M, int64_t h, int64_t i, int r, float s, lora_act_t act,
                                            int64_t n_examples, const void* x, lora_linear_t gate,
                                            lora_linear_t up, lora_linear_t down, const void* saved,
                                            const void* dy, void* dx, lora_grads_t d_gate,
                                            lora_grads_t d_up, lora_grads_t d_down, float* sq_norms,
                                            void* ws, size_t ws_bytes, cudaStream_t stream);

/* Rotary position embedding of q and k ("Model Patches and Kernels", section "Rotary
 * position embeddings (RoPE)": q and k rotated together, GQA head counts; RoFormer's
 * position encoding).  Every head (head_dim features) of q and k is rotated pair by
 * pair, the pair being features (c, c + head_dim/2) of the head:
 *   q'[c] = q[c] cos - q[c + d/2] sin,  q'[c + d/2] = q[c + d/2] cos + q[c] sin,
 * with cos, sin = cos[pos[m]][c], sin[pos[m]][c] for token m.  The tables are the
 * caller's (lora_rope_table fills RoFormer's p * base^(-2c/d); scaled variants are
 * any other table).  Device pointers: cos, sin f32 [n_pos x head_dim/2] row-major,
 * 16-byte aligned; pos int32 [M], 4-byte aligned.  head_dim is 64, 128 or 256 and
 * divides n_q and n_kv.  A position outside [0, n_pos) is read as 0 and reported by
 * lora_poll_status as LORA_ERR_DEVICE_INPUT. */
typedef struct {
  const float* cos;
  const float* sin;
  const int32_t* pos;
  int64_t n_pos;
  int head_dim;
} lora_rope_t;

/* Fills cos/sin [n_pos x head_dim/2] (f32, device, 16-byte aligned) with the cosine
 * and sine of p * base^(-2c/head_dim), computed in double and rounded once.
 * head_dim even and >= 2, n_pos >= 1, base > 0, else LORA_ERR_INVALID_ARG. */
lora_status_t lora_rope_table(float* cos, float* sin, int64_t n_pos, int head_dim, double base,
                              cudaStream_t stream);

/* ---------------------------------------------------------------- Q/K/V + O
 * q = (1)(x; q) [M x n_q], k, v = (1)(x; k or v) [M x n_kv] ("opake_lora_qkv"), and
 * yo = (1)(o_in; o) [M x h] with W_o [h x n_q] ("original_apply_o").  Attention runs
 * between the two halves in a real block, so either half may be skipped: x == NULL
 * skips q/k/v, o_in == NULL skips O.  bias_qkv is NULL or the frozen base-layer
 * biases of q, k and v, bf16 [n_q + 2 n_kv] (q's, then k's, then v's), 16-byte
 * aligned, added to q, k, v ("Fused LoRA operations": QKV fusion supports optional
 * frozen base-layer biases); a frozen bias gets no gradient, so backward does not
 * take it.  rope is NULL or the rotary embedding applied to q and k after the bias,
 * in the projection's epilogue (lora_rope_t above; ignored when x == NULL).  saved
 * (NULL for inference) receives the rank-r projections (also transposed where the
 * backward's single passes read them) and the adapters packed for backward. */
size_t lora_qkvo_saved_bytes(int64_t M, int64_t h, int64_t n_q, int64_t n_kv, int r);
size_t lora_qkvo_workspace_bytes(int64_t M, int64_t h, int64_t n_q, int64_t n_kv, int r);
lora_status_t lora_qkvo_forward(int64_t M, int64_t h, int64_t n_q, int64_t n_kv, int r, float s,
                                const void* x, lora_linear_t q, lora_linear_t k,
                                lora_linear_t v, void* yq, void* yk, void* yv,
                                const void* o_in, lora_linear_t o, void* yo,
                                const void* bias_qkv, const lora_rope_t* rope, void* saved,
                                void* ws, size_t ws_bytes, cudaStream_t stream);
/* Gradients of <dyq, q> + <dyk, k> + <dyv, v> (dx = their sum over the three
 * projections, and dA/dB of q, k, v) and of <dyo, yo> (do_in and dA/dB of o).
 * x == NULL skips the q/k/v half, o_in == NULL the O half.  With rope (the one the
 * forward used), dyq and dyk are gradients of the rotated q and k: they are turned
 * back by the transpose rotation (into the workspace) before the projections'
 * backward.  The adapters enter as the forward packed them into saved (with its s):
 * q, k, v, o must be the forward's (their W is read here; their A and B only
 * checked), and s the same. */
lora_status_t lora_qkvo_backward(int64_t M, int64_t h, int64_t n_q, int64_t n_kv, int r, float s,
                                 const void* x, lora_linear_t q, lora_linear_t k,
                                 lora_linear_t v, const void* o_in, lora_linear_t o,
                                 const void* saved, const lora_rope_t* rope,
                                 const void* dyq, const void* dyk,
                                 const void* dyv, void* dx, const void* dyo, void* do_in,
                                 lora_grads_t d_q, lora_grads_t d_k, lora_grads_t d_v,
                                 lora_grads_t d_o, void* ws, size_t ws_bytes,
                                 cudaStream_t stream);

/* ---------------------------------------------------------------- serving: rotary, cache, attention
 * What stands between the Q/K/V and the O projection when a tuned model answers: the
 * rotation of q and k, a paged cache of K and V, and the attention of the new tokens
 * over it.  Tensors of heads are views, so that q, k and v can be slices of one buffer.
 *
 * lora_heads_t: bf16 [M x heads x head_dim], feature stride 1, the other strides in
 * elements, not negative and multiples of 8; data 16-byte aligned.  An output's rows must
 * not overlap. */
typedef struct {
  void* data;
  int64_t heads;
  int64_t token_stride;
  int64_t head_stride;
} lora_heads_t;

/* Rotary positions of the first rot_dim features of a head; the others pass through.
 * The pair (a, b) that table column c turns is (x[c], x[c + rot_dim/2]) in the half
 * layout and (x[2c], x[2c + 1]) in the interleaved one:
 *   a' = a cos - b sin,   b' = b cos + a sin,   cos, sin = cos[pos[m]][c], sin[pos[m]][c].
 * Tables f32 [n_pos x rot_dim/2], 16-byte aligned; pos int32 [M].  rot_dim even, at
 * least 2, at most head_dim (multiples of 16 are fastest).  A position outside
 * [0, n_pos) is read as 0 and reported by lora_poll_status as LORA_ERR_DEVICE_INPUT.
 * (lora_rope_t, the rotation inside the Q/K/V projection, is the half layout with
 * rot_dim == head_dim.) */
typedef enum { LORA_ROTARY_HALF = 0, LORA_ROTARY_INTERLEAVED = 1 } lora_rotary_layout_t;
typedef struct {
  const float* cos;
  const float* sin;
  const int32_t* pos;
  int64_t n_pos;
  int rot_dim;
  int layout;               /* lora_rotary_layout_t */
} lora_rotary_t;

/* yq = rotated q, yk = rotated k (k->data NULL: only q) in one launch; head_dim a
 * multiple of 8, at most 1024.  inverse != 0 turns back by the same angles: the
 * gradient of q and k from that of yq and yk.  Products and sums are f32, each rounded,
 * and the result is rounded to bf16 once.  y may be x itself (same data and strides);
 * any other overlap is undefined.  ws: at least 256 bytes (the status word). */
lora_status_t lora_rotary(int64_t M, int head_dim, const lora_heads_t* q, const lora_heads_t* yq,
                          const lora_heads_t* k, const lora_heads_t* yk, const lora_rotary_t* rot,
                          int inverse, void* ws, size_t ws_bytes, cudaStream_t stream);

/* lora_rope_table for long contexts: cos, sin [n_pos x rot_dim/2] of p * w_c, times a
 * magnitude, where w_c = base^(-2c/rot_dim) is changed by `kind`:
 *   LINEAR      w_c / factor (position interpolation)
 *   NTK         base becomes base * factor^(rot_dim / (rot_dim - 2)); rot_dim >= 4
 *   YARN        (1 - g_c) w_c + g_c w_c / factor, g_c rising from 0 to 1 between the
 *               columns that turn `high` and `low` times in original_len positions
 *               (rounded outwards); 0 < low < high (the method's own choice: 1, 32)
 *   WAVELENGTH  wavelengths below original_len / high keep w_c, those above
 *               original_len / low take w_c / factor, between them a linear blend in
 *               original_len / wavelength; 0 < low < high
 * factor >= 1.  magnitude multiplies cos and sin; 0 stands for 1, and with YARN for
 * 0.1 ln(factor) + 1.  Computed in double and rounded once. */
typedef enum {
  LORA_ROPE_PLAIN = 0, LORA_ROPE_LINEAR = 1, LORA_ROPE_NTK = 2, LORA_ROPE_YARN = 3, LORA_ROPE_WAVELENGTH = 4
} lora_rope_kind_t;
typedef struct {
  int kind;                 /* lora_rope_kind_t */
  double factor;
  double original_len;
  double low, high;
  double magnitude;
} lora_rope_scaling_t;
lora_status_t lora_rope_table_scaled(float* cos, float* sin, int64_t n_pos, int rot_dim, double base,
                                     const lora_rope_scaling_t* scaling, cudaStream_t stream);

/* A paged cache of K and V: pages [n_pages x heads x page_size x head_dim] of bf16, or
 * of 8-bit codes (e4m3 or int8) with a scale for each row, f32 [n_pages x heads x
 * page_size] (NULL for bf16).  page_size 16, 32, 64, 128 or 256; head_dim 64, 128 or
 * 256; pages and scales 16-byte aligned.  n_pages * heads * page_size is at
 * most 2^31 - 1 rows.  Slot number s is row s % page_size of page s / page_size.
 *
 * A row x is stored as codes rn(x * (1 / scale)) with scale = max(amax|x| * (1/Q),
 * the smallest normal f32), Q = 127 for int8 and 448 for e4m3 (all in f32, ties to even).
 * A row that holds an infinity or a NaN is stored as scale NaN and codes 0. */
typedef enum { LORA_KV_BF16 = 0, LORA_KV_FP8 = 1, LORA_KV_INT8 = 2 } lora_kv_format_t;
typedef struct {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int64_t n_pages;
  int page_size;
  int heads;
  int head_dim;
  int format;               /* lora_kv_format_t */
} lora_kv_cache_t;

/* Writes token m's k and v (views with the cache's heads) to slot slots[m] (int64 [M]) in the
 * cache's format.  With rot, k is rotated first, and q (NULL or data NULL: none) into yq
 * in the same launch; the rotated k is not rounded before it is quantised.  A negative
 * slot is skipped (padding); one past the cache is skipped and reported
 * (LORA_ERR_DEVICE_INPUT).  The slots of a call must differ from each other.  q needs
 * rot.  yq may be q itself.  ws: at least 256 bytes. */
lora_status_t lora_kv_append(int64_t M, const lora_kv_cache_t* cache, const lora_heads_t* k,
                             const lora_heads_t* v, const int64_t* slots, const lora_heads_t* q,
                             const lora_heads_t* yq, const lora_rotary_t* rot, void* ws, size_t ws_bytes,
                             cudaStream_t stream);

/* Reads sequences back: row cu_kv[b] + i of k and v (bf16 [total x heads x head_dim],
 * dense) is position i of sequence b, 0 <= i < cu_kv[b+1] - cu_kv[b].  cu_kv int32
 * [n_seqs + 1], rising from 0 to total; page_table int32 [n_seqs x max_pages], entry
 * [b][i / page_size] the page of position i.  A page outside the cache, a position past
 * the table and a row that cu_kv does not cover read as 0 and are reported
 * (LORA_ERR_DEVICE_INPUT).  ws: at least 256 bytes. */
lora_status_t lora_kv_read(int64_t n_seqs, int64_t total, const lora_kv_cache_t* cache,
                           const int32_t* page_table, int64_t max_pages, const int32_t* cu_kv, void* k,
                           void* v, void* ws, size_t ws_bytes, cudaStream_t stream);

/* The sequences of a call: sequence b owns query rows [cu_q[b], cu_q[b+1]) of M (cu_q int32
 * [n_seqs + 1], not falling, inside [0, M]) and kv_len[b] cached positions (int32), its
 * new tokens' own among them; page_table as above.  All on the device: a step can be
 * captured in a graph and its lengths changed between replays. */
typedef struct {
  int64_t n_seqs;
  const int32_t* page_table;
  int64_t max_pages;
  const int32_t* kv_len;
  const int32_t* cu_q;
} lora_paged_batch_t;

/* Attention of new tokens over the cache.  Token i of sequence b's n_b = cu_q[b+1] -
 * cu_q[b] stands at position p = kv_len[b] - n_b + i and sees the positions j <
 * kv_len[b] with j <= p (causal != 0) and p - j < window (window > 0; 0: no window).
 * Query head g reads cache head g / (heads_q / heads):
 *   out = sum_j e^(s_j - max s) v_j / sum_j e^(s_j - max s),  s_j = scale * <q, k_j>.
 * out bf16 [M x heads_q x head_dim], dense (the O projection's input); lse f32 [M x
 * heads_q] or NULL receives ln sum_j e^(s_j).  A token that sees nothing (kv_len 0, or
 * p < 0) gets out 0 and lse -inf.  Rows of M that no sequence owns are not written.
 * q is a view (of strides above 0); heads_q is a multiple of the cache's heads, and
 * M * heads_q at most 2^31 - 1.
 * Scores, maxima, sums and the accumulated output are f32; the weights e^(...) are rounded
 * to the matrix units' 16 bits before they multiply V, and the result is rounded once.  With a
 * bf16 cache the weights are bf16; few query rows carry them in two parts, 16 bits of
 * significand.  With an 8-bit cache they are f16, and many query rows may also have V, code
 * times scale, rounded to f16's 11 bits; a weight whose product with its V's scale is below
 * 2^-14 of the row's largest such product is rounded to 2^-24 of that.
 * What lies past kv_len in a page is not looked at, whatever bits it holds, and neither are
 * the table entries and pages that lie wholly before the window of a sequence's first new
 * token (they may have been released).  Any other page outside the cache is read as page 0,
 * and a length past the table or a query range outside M is cut to it, each reported by
 * lora_poll_status (LORA_ERR_DEVICE_INPUT).  An infinity or NaN in a position of a sequence's
 * own V in a bf16 cache (kv_len's inside; in an e4m3 one a NaN code, which lora_kv_append
 * never writes) may also reach tokens of that sequence that do not see the position.
 * ws: lora_paged_attention_workspace_bytes, the same for every M, n_seqs and heads_q over a
 * cache (0 for arguments that the call refuses): steps of any size can share one. */
size_t lora_paged_attention_workspace_bytes(int64_t M, int64_t n_seqs, int heads_q, const lora_kv_cache_t* cache);
lora_status_t lora_paged_attention(int64_t M, int heads_q, const lora_heads_t* q, const lora_kv_cache_t* cache,
                                   const lora_paged_batch_t* batch, float scale, int causal, int64_t window,
                                   void* out, float* lse, void* ws, size_t ws_bytes, cudaStream_t stream);

/* ---------------------------------------------------------------- the rest of a training step
 * What a step runs around the block's projections: the norms before them, the loss behind
 * the last block, and the clipping of the adapters' gradients.
 *
 * RMS norm, with the residual's addition before it.  A row is one token's head of the views
 * (heads == 1: one token), `dim` features:
 *   s = x + residual, rounded to bf16 (residual NULL or data NULL: s = x)
 *   rstd = (mean s^2 + eps)^(-1/2),   y = s * rstd * (weight + offset)
 * The norm is of s as it is rounded.  f32 arithmetic; y is rounded once.
 * - sum receives s (required with a residual; NULL or data NULL without one).  It may be x or
 *   the residual itself; any other overlap of an output with an input is undefined, but that
 *   without a residual a dense x may be y.
 * - weight bf16 [dim]; offset is added to it in f32 (1 for weights stored around zero).
 * - y dense [M x heads x dim]: bf16 (LORA_NORM_BF16), or e4m3 codes with a scale for each row
 *   (LORA_NORM_FP8): scale = max(amax|y| * (1/448), the smallest normal f32), codes =
 *   rn(y * (1 / scale)) of the y that was not rounded; a row whose y holds an infinity or a
 *   NaN gets the scale NaN and codes 0.  Codes are 8-byte aligned.  y_scale f32 [M x heads], NULL
 *   with LORA_NORM_BF16.
 * - rstd f32 [M x heads], or NULL (inference).  Where it leaves f32's range (eps 0 and a row of zeros, or of values
 *   below 2.9e-39) it is infinite, and y infinite or NaN.
 * dim a multiple of 8, at most 32768.  M * heads at most 2^31 - 1.  ws: at least 256 bytes. */
typedef enum { LORA_NORM_BF16 = 0, LORA_NORM_FP8 = 1 } lora_norm_format_t;
lora_status_t lora_rms_norm(int64_t M, int dim, const lora_heads_t* x, const lora_heads_t* residual,
                            const void* weight, float offset, float eps, int format, const lora_heads_t* sum,
                            void* y, float* y_scale, float* rstd, void* ws, size_t ws_bytes, cudaStream_t stream);

/* Gradients of <dy, y> + <ds, s>, s and rstd the forward's (s its sum, or x without a residual):
 *   dx = ds + rstd * (g - s * rstd^2 * mean(g * s)),  g = dy * (weight + offset)
 *   dweight = sum over the rows of dy * s * rstd
 * dx, dense bf16 [M x heads x dim], is the gradient of x and of the residual.  ds NULL or
 * data NULL: none.  dweight bf16 [dim], or NULL (a frozen weight's gradient is skipped); its
 * f32 sums run in an order that depends on the sizes and the device alone.  dx may be dy or ds where
 * they are dense.  M == 0 sets dweight to zero.  ws: lora_rms_norm_workspace_bytes (0 for
 * sizes that the calls refuse). */
size_t lora_rms_norm_workspace_bytes(int64_t M, int64_t heads, int dim);
lora_status_t lora_rms_norm_backward(int64_t M, int dim, const lora_heads_t* dy, const lora_heads_t* s,
                                     const void* weight, float offset, const float* rstd, const lora_heads_t* ds,
                                     void* dx, void* dweight, void* ws, size_t ws_bytes, cudaStream_t stream);

/* Cross entropy of a frozen head, from the hidden rows to the loss and their gradient without
 * keeping the logits ("Model Patches and Kernels", section "Fused linear cross-entropy":
 * logit scaling, softcap; "Cross-entropy": label smoothing; a frozen weight's gradient is
 * skipped).  x bf16 [M x h], W bf16 [vocab x h], labels int64 [M]:
 *   z = logit_scale * x W^T,   z' = softcap * tanh(z / softcap)  (softcap 0: z' = z)
 *   lse_m = ln sum_v e^(z'_v),   loss_m = lse_m - (1 - smoothing) z'_y - smoothing * mean_v z'_v
 *   total = sum_m loss_m, divided for LORA_LOSS_MEAN by the number of labelled tokens (by 1 if
 *   there is none)
 *   dx = the gradient of total with respect to x
 * A token whose label is ignore_index has no part in it: its loss, lse and dx row are 0 and its
 * x is not used.  So has one whose label is outside [0, vocab), which is reported
 * (LORA_ERR_DEVICE_INPUT).  loss, lse f32 [M], or NULL; total f32 [1]; dx bf16 [M x h], or
 * NULL (the loss alone).  dx may not overlap x or W.
 * Logits, their exponentials and all sums are f32.  The matrix units sum up to 1024 features of a logit and
 * cut what falls below the last place (1e-6 of a logit whose products have one sign); such parts join
 * in f32.  A cap costs a logit 24 units of 2^-24 of itself at most.  For dx the weights of all but the label's word are rounded to bf16 on their way to the
 * product with W, and scaled so that their sum stays what it was; the label's stays f32.
 * Tokens are taken in pieces of up to 1 GiB of such weights (256 tokens at least) and as much of f32 sums, which live
 * in the workspace: a piece has a bf16 number for every logit.  With dx 4096 tokens x 4096 x 131,072 words take
 * 1.2 GiB, 2048 x 4096 x 50,257 327 MiB, 64 x 896 x 32,000 49 MiB; the loss alone 64, 22 and 0.6 MiB.  A label
 * more than 100 below its row's largest logit makes its piece take both products again.  h a multiple of 8; vocab at most 2^24; x, W, dx 16-byte aligned.  logit_scale finite, not 0;
 * softcap finite, >= 0; 0 <= smoothing < 1.
 * ws: lora_linear_ce_workspace_bytes (0 for sizes or options that the call refuses), which
 * grows with M by x's own size and the pieces. */
typedef enum { LORA_LOSS_SUM = 0, LORA_LOSS_MEAN = 1 } lora_loss_reduction_t;
typedef struct {
  float logit_scale;
  float softcap;
  float smoothing;
  int reduction;            /* lora_loss_reduction_t */
  int64_t ignore_index;
} lora_ce_t;
size_t lora_linear_ce_workspace_bytes(int64_t M, int64_t h, int64_t vocab, const lora_ce_t* opts, int want_dx);
lora_status_t lora_linear_ce(int64_t M, int64_t h, int64_t vocab, const void* x, const void* W,
                             const int64_t* labels, const lora_ce_t* opts, float* loss, float* lse, float* total,
                             void* dx, void* ws, size_t ws_bytes, cudaStream_t stream);

/* y_m = g[m * g_stride] * x_m, rounded once: rows of bf16 [M x h], factors f32 (g_stride 1: one a row, 0:
 * one for all).  What autograd does with lora_linear_ce's dx when the loss's own gradient arrives.
 * y may be x.  h a multiple of 8, x and y 16-byte aligned.  ws: at least 256 bytes. */
lora_status_t lora_scale_rows(int64_t M, int64_t h, const void* x, const float* g, int g_stride, void* y, void* ws,
                              size_t ws_bytes, cudaStream_t stream);

/* A tensor of a list: count elements, one after the other, aligned to their own size.  The
 * list itself is host memory and is copied by the call (into the launch, so that a captured
 * call keeps it). */
typedef enum { LORA_BF16 = 0, LORA_F32 = 1 } lora_dtype_t;
typedef struct {
  void* data;               /* may be NULL where count is 0 */
  int64_t count;
  int dtype;                /* lora_dtype_t */
} lora_tensor_t;

/* The norm of all tensors of a list together: (sum g^2)^(1/2) (LORA_GRAD_NORM_2) or max |g|
 * (LORA_GRAD_NORM_INF; a NaN if there is one), f32 [1], 0 for a list of nothing.  Squares and their
 * sums are f32, in short chains whose order depends on the counts and the tensors' alignment
 * alone: the first kind is infinite beyond 1.8e19, and elements below 1e-23 count as zero.
 * lora_clip_grads: out_i = g_i * min(1, max_norm / (norm + 1e-6)), rounded once to its type;
 * norm receives the norm before it.  A norm that is not finite goes into the factor as it is:
 * infinite gives 0 (and NaN for an infinite element), NaN gives NaN.  out: NULL (in place, and
 * nothing is written where the factor is 1) or a list like grads (counts and types), whose
 * tensors overlap no other tensor of grads or out but may be the same one of grads.
 * max_norm > 0 (infinity: out is a copy).  Neither synchronises.  n at most 2^20 tensors.
 * ws: lora_grad_norm_workspace_bytes(n) (0 for n that the calls refuse). */
typedef enum { LORA_GRAD_NORM_2 = 0, LORA_GRAD_NORM_INF = 1 } lora_grad_norm_t;
size_t lora_grad_norm_workspace_bytes(int64_t n);
lora_status_t lora_grad_norm(int64_t n, const lora_tensor_t* grads, int norm_type, float* norm, void* ws,
                             size_t ws_bytes, cudaStream_t stream);
lora_status_t lora_clip_grads(int64_t n, const lora_tensor_t* grads, const lora_tensor_t* out, int norm_type,
                              float max_norm, float* norm, void* ws, size_t ws_bytes, cudaStream_t stream);

/* DP-SGD's clipped sum of per-example gradients (those of lora_mlp_backward_per_example and
 * whatever else belongs to the same examples): each tensor of grads holds n_examples gradients
 * of count / n_examples elements, example-major, and
 *   out_i = scale * sum_e c_e g_i[e],   c_e = min(1, max_norm / (sum_i |g_i[e]|^2)^(1/2))
 * out: n tensors of f32, of count / n_examples elements each, that overlap nothing else.
 * sq_norms f32 [n_examples] holds the examples' squared norms: norms_given != 0 reads them (as
 * lora_mlp_backward_per_example gives them, added over its calls), else the call writes them.
 * Sums are f32, in a fixed order of the examples; squares too, so that elements below 1e-23 count as zero in a
 * norm and one beyond 1.8e19 is infinite.  An example whose norm is not finite makes the sums NaN where its factor or its elements do.
 * max_norm > 0, scale finite; n_examples at most 65535.
 * ws: lora_clip_examples_workspace_bytes(n, n_examples) (0 for what the call refuses). */
size_t lora_clip_examples_workspace_bytes(int64_t n, int64_t n_examples);
lora_status_t lora_clip_examples(int64_t n, const lora_tensor_t* grads, int64_t n_examples, const lora_tensor_t* out,
                                 float max_norm, float scale, float* sq_norms, int norms_given, void* ws,
                                 size_t ws_bytes, cudaStream_t stream);

/* ---------------------------------------------------------------- status, counters
 * lora_poll_status: synchronises `stream`, reads the asynchronous status word in
 * ws, clears it, and returns LORA_OK, LORA_ERR_TIMEOUT or LORA_ERR_DEVICE_INPUT
 * (timeout first when both are set; LORA_ERR_CUDA if the synchronisation itself
 * fails).  ws == NULL reads and clears the status word of the current device's
 * lora_linear_forward_noalloc scratch instead (the word that call's kernels set). */
lora_status_t lora_poll_status(void* ws, cudaStream_t stream);
const char* lora_status_string(lora_status_t status);
/* Kernels this library has launched in this process (all entry points). */
uint64_t lora_launch_count(void);

/* ---------------------------------------------------------------- bounded waits
 * Every wait inside the GEMM kernels (a pipeline stage, an accumulator buffer) is
 * bounded.  When one runs out, the kernel stops issuing work, lets its own copies and
 * MMAs in flight finish, frees its tensor memory and exits; the status word in `ws`
 * then reads LORA_ERR_TIMEOUT (see lora_poll_status) and that call's outputs are
 * undefined.  The CUDA context stays usable.  The pages define no such mechanism.
 *
 * lora_set_wait_timeout: the limit in nanoseconds for launches enqueued after the
 * call, process-wide (all devices, all threads).  0 restores the default of 2 s.
 * Accepted range 1 ms .. 60 s, else LORA_ERR_INVALID_ARG.  A limit shorter than
 * the slowest tile of a workload (tens of microseconds for the shapes here, longer
 * when the GPU is time-sliced with other processes) makes healthy calls fail.
 * The limit is wall-clock time (the GPU's nanosecond timer), whatever the SM clock.
 * lora_wait_timeout: the current limit in nanoseconds. */
lora_status_t lora_set_wait_timeout(uint64_t ns);
uint64_t lora_wait_timeout(void);

/* ---------------------------------------------------------------- split tail
 * The projection GEMMs deal whole 256 x 256 output tiles round-robin to pairs of SMs.
 * When the last wave would leave pairs idle, the tiles of that wave (all tiles, when
 * there are fewer than pairs) can each be cut into 2 to 4 equal k-ranges computed by
 * different pairs; the last piece of a tile to finish adds the others' f32 partial
 * sums, in a fixed order, before the epilogue, so results stay deterministic for a
 * given device and mode (and match the whole-tile schedule up to the order of the f32
 * sums).  The partial sums live in the call's workspace (the size queries include
 * them).  Not from the pages: a scheduling choice of this library.
 *
 * lora_set_split_tail: 0 (default) cuts the tail into the number of pieces (2 to 4)
 * for which a cost model of the partial sums expects the launch to gain most, if at
 * least 2%; 1 never cuts; 2, 3 or 4 cuts every tail into that many pieces whenever the
 * launch allows it (every group with the same k-extent, at least 8 k-blocks per tile
 * and two per piece, a tail of at most 128 tiles).  Process-wide, for launches enqueued
 * after the call; the environment variable LORA_SPLIT_TAIL=1..4 sets the initial mode.
 * Other values return LORA_ERR_INVALID_ARG.  lora_split_tail: the current mode. */
lora_status_t lora_set_split_tail(int mode);
int lora_split_tail(void);

/* Test hook for the failure path (no counterpart in the pages): the next `launches`
 * GEMM or paged-attention launches (0 .. 64; 0 cancels) each leave the first pipeline stage of every
 * CTA's first tile unfilled, so the waits on it expire after the wait limit and the
 * call reports LORA_ERR_TIMEOUT through the status word.  Nothing faults, traps or
 * hangs: the waits are the bounded ones above.  Returns LORA_ERR_INVALID_ARG out of
 * range. */
lora_status_t lora_test_expire_waits(int launches);

/* Launch tracing, for measurement.  lora_trace_enable(n) makes every later launch (of
 * the kinds lora_trace_kinds selects; all by default) record a pair of CUDA events
 * around itself on its stream, keeping the first n launches (0 disables and frees
 * the events).  lora_trace_read synchronises the
 * recorded events, fills kind[] and ms[] (kernel kinds below) for up to `max`
 * launches, and restarts the trace; it returns the number filled or -1 on error. */
enum {
  LORA_KIND_PACK = 0,        /* adapter packing */
  LORA_KIND_REDUCE = 1,      /* split-K sums of the rank-r products; per-example norms */
  LORA_KIND_RANK_PROJ = 2,   /* token-major rank-r projections (x A^T, dy B, dg B) */
  LORA_KIND_RANK_GRAD = 3,   /* reductions over tokens (dA, dB) */
  LORA_KIND_GATE_UP = 4,     /* gate/up GEMM with the activation epilogue */
  LORA_KIND_PROJ = 5,        /* plain projection GEMM (down, q/k/v, o) */
  LORA_KIND_ACT_BWD = 6,     /* dh GEMM with the activation-derivative epilogue */
  LORA_KIND_DGRAD = 7,       /* input-gradient GEMM (dx, d o_in) */
  LORA_KIND_ROPE = 8,        /* RoPE transpose rotation of dy_q, dy_k; RoPE tables; lora_rotary */
  LORA_KIND_CACHE = 9,       /* cache writes and reads */
  LORA_KIND_ATTN = 10,       /* attention over the cache, and the joining of its split sums */
  LORA_KIND_NORM = 11,       /* RMS norm and its gradient */
  LORA_KIND_LOSS = 12,       /* the linear cross entropy: its GEMMs and what stands between them */
  LORA_KIND_CLIP = 13        /* gradient norms and clipping */
};
lora_status_t lora_trace_enable(int capacity);
int lora_trace_read(int* kind, float* ms, int max);
/* Restricts tracing to the kinds whose bit is set in mask (bit k: kind k; all by
 * default).  Events between two launches serialise them, so tracing only the kernel
 * being measured keeps the others' overlap (programmatic dependent launch) intact. */
void lora_trace_kinds(unsigned mask);

#ifdef __cplusplus
}
#endif

#endif /* LORA_GB300_H */
