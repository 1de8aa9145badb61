// The paged K/V cache: writing tokens into it, rotated and quantised on the way
// (lora_kv_append), and reading sequences back (lora_kv_read); include/lora_gb300.h is
// the contract.
//
// Both move every byte once and are bounded by memory (small calls by the launch).  A row
// (one token's head) belongs to head_dim / 8 neighbouring lanes, 8 features each, so its
// maximum takes log2(head_dim / 8) shuffles and its codes leave as one contiguous piece;
// a lane group walks several heads of its token with the same slot, position, cos and
// sin.  Measured: writing 8192 tokens of 8 + 8 heads of 128 features into an fp8 cache, 32
// query heads turned beside them: 190 MB in 42.6 us (4.4 TB/s, 65% of a copy's rate; the
// rounding that the plain form takes, product by product, keeps it at the instructions), bf16
// 40.5 us; reading back 24,000 int8 positions: 151 MB in 28.1 us (5.4 TB/s, 79%); 64 tokens
// into an int8 cache 2.5 us in a graph.
#include "serve.cuh"

namespace lgb {

struct AppendParams {
  HeadsView k, v, q;
  HeadsOut yq;
  int hk, hq;                // the heads of a call, in order: k's, v's, q's
  long long M;
  const long long* slots;
  CacheArgs cache;
  RotaryArgs rot;
  int rotate, interleaved;
  int per_group, groups;     // heads a lane group walks; such groups of heads
  unsigned* status;
};

// The lane's cos and sin by feature, with the sign that the second product takes:
// y = x cos + partner * ssn.  Features that do not turn have a cleared bit in `turned`.
struct LaneTurn {
  float c[8], s[8];
  unsigned turned;
};

// VEC: rot_dim is a multiple of 16, a lane's 8 features turn together or not at all.
template <bool VEC>
__device__ __forceinline__ void load_turn(const AppendParams& p, int at, int f0, LaneTurn& t) {
  const int half = p.rot.half;
  t.turned = 0;
  if (f0 >= 2 * half) return;
  const long long tab = static_cast<long long>(checked_position(p.rot, at, p.status)) * half;
  const float* cos = p.rot.cos + tab;
  const float* sin = p.rot.sin + tab;
  if (VEC && !p.interleaved) {
    const bool second = f0 >= half;
    load8f(cos + (second ? f0 - half : f0), t.c);
    load8f(sin + (second ? f0 - half : f0), t.s);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (!second) t.s[e] = -t.s[e];
    t.turned = 0xFFu;
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int f = f0 + e;
    if (f >= 2 * half) continue;
    const int col = p.interleaved ? f / 2 : (f < half ? f : f - half);
    const bool second = p.interleaved ? (f & 1) : f >= half;
    t.c[e] = __ldg(cos + col);
    t.s[e] = second ? __ldg(sin + col) : -__ldg(sin + col);
    t.turned |= 1u << e;
  }
}

// The lane's 8 features [f0, f0 + 8) of row x (own: as loaded) rotated in f32, not rounded.
// Whole warps call it: in the half layout a lane's partners come from another lane of the
// row, `from`.
template <bool VEC>
__device__ __forceinline__ void turn_piece(const AppendParams& p, uint4 own, const bf16* x, int f0, int from,
                                           const LaneTurn& t, bool rotate, float (&y)[8]) {
  unpack8(own, y);
  float o[8];
  if (p.interleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = y[e ^ 1];
  } else if (VEC) {
    uint4 w;
    w.x = __shfl_sync(0xffffffffu, own.x, from);
    w.y = __shfl_sync(0xffffffffu, own.y, from);
    w.z = __shfl_sync(0xffffffffu, own.z, from);
    w.w = __shfl_sync(0xffffffffu, own.w, from);
    unpack8(w, o);
  } else if (rotate) {
    const int half = p.rot.half;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int f = f0 + e;
      o[e] = (t.turned >> e) & 1u ? __bfloat162float(x[f < half ? f + half : f - half]) : 0.0f;
    }
  }
  if (!rotate || !t.turned) return;
  // (scalar on purpose: as packed f32x2 operations the compiler joins the product and the sum)
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (VEC || ((t.turned >> e) & 1u)) y[e] = __fadd_rn(__fmul_rn(y[e], t.c[e]), __fmul_rn(o[e], t.s[e]));
}

// Four heads' pieces in flight a lane, and blocks an SM: 8192 tokens took 44.4, 40.5 and 55.9
// us with 5, 6 and 7 blocks (bf16; at 7 the pieces spill), 49.4, 44.9, 42.6 and 57.7 us with 5
// to 8 (fp8).
constexpr int kAppendThreads = 128;

template <int D, int FMT, bool VEC>
__global__ void __launch_bounds__(kAppendThreads, FMT == LORA_KV_BF16 ? 6 : 7) append_kernel(const __grid_constant__ AppendParams p) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int L = D / 8;                       // lanes of a row
  const int f0 = (threadIdx.x % L) * 8;
  const int heads = 2 * p.hk + p.hq;
  const unsigned long long units = static_cast<unsigned long long>(p.M) * p.groups;
  const unsigned long long step = static_cast<unsigned long long>(gridDim.x) * (kAppendThreads / L);
  // the warp's lane groups run the same number of steps: the shuffles take whole warps
  for (unsigned long long base = static_cast<unsigned long long>(blockIdx.x) * (kAppendThreads / L); base < units; base += step) {
    const unsigned long long u = base + threadIdx.x / L;
    const bool live = u < units;
    // neighbouring lane groups take neighbouring tokens and the same heads, so that a warp's
    // rows go the same way (k, v or q)
    const int g = !live ? 0 : units <= 0xffffffffull ? static_cast<int>(static_cast<unsigned>(u) / static_cast<unsigned>(p.M))
                                                     : static_cast<int>(u / static_cast<unsigned long long>(p.M));
    const long long m = live ? static_cast<long long>(u) - g * p.M : 0;
    const int h0 = g * p.per_group, h1 = live ? min(h0 + p.per_group, heads) : h0;
    // slot and position, the first heads' pieces, then the table entries, which wait for the
    // position: the loads' latencies overlap
    const bool turns = p.rotate && live && (h0 < p.hk || h1 > 2 * p.hk);
    const int at = turns ? __ldg(p.rot.pos + m) : 0;
    long long slot = live ? __ldg(p.slots + m) : -1;
    const int lane = threadIdx.x & 31, half8 = p.rot.half / 8, c8 = f0 / 8;
    const int from = c8 < half8 ? lane + half8 : c8 < 2 * half8 ? lane - half8 : lane;
    LaneTurn t;
    long long row0 = 0;        // the slot's row of head 0
    const bf16* k_row = p.k.x + m * p.k.ts;
    const bf16* v_row = p.v.x + m * p.v.ts - p.hk * p.v.hs;
    const bf16* q_row = p.q.x + m * p.q.ts - 2 * p.hk * p.q.hs;
    auto row_of = [&](int h) {
      const bf16* base = h >= 2 * p.hk ? q_row : h >= p.hk ? v_row : k_row;
      return base + h * (h >= 2 * p.hk ? p.q.hs : h >= p.hk ? p.v.hs : p.k.hs);
    };
    for (int jb = 0; jb < p.per_group; jb += kHeadBatch) {
    uint4 w[kHeadBatch];
#pragma unroll
    for (int i = 0; i < kHeadBatch; ++i) {
      const int h = h0 + jb + i;
      w[i] = h < h1 ? *reinterpret_cast<const uint4*>(row_of(h) + f0) : make_uint4(0, 0, 0, 0);
    }
    if (jb == 0) {
      t.turned = 0;
      if (turns) load_turn<VEC>(p, at, f0, t);
      const long long page = slot >> p.cache.page_shift;
      if (slot >= 0 && page >= p.cache.n_pages) {
        atomicOr(p.status, kStatusInput);
        slot = -1;
      }
      row0 = (page * p.cache.heads << p.cache.page_shift) + (slot & ((1 << p.cache.page_shift) - 1));
    }
#pragma unroll
    for (int i = 0; i < kHeadBatch; ++i) {
      const int h = h0 + jb + i;
      if (jb + i >= p.per_group) break;
      const bool row = h < h1;
      const bool is_q = h >= 2 * p.hk, is_v = !is_q && h >= p.hk;
      float y[8];
      turn_piece<VEC>(p, w[i], row ? row_of(h) : p.k.x, f0, from, t, row && p.rotate && !is_v, y);
      // the row's largest magnitude (a NaN if it holds one)
      float top = 0.0f;
      // every lane of the row has read its partners' features before any writes (yq may be q;
      // the vote below orders no memory)
      if (FMT == LORA_KV_BF16 || !VEC) __syncwarp();
      if (FMT != LORA_KV_BF16 && __any_sync(0xffffffffu, row && !is_q)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max_abs_nan(top, y[e]);
#pragma unroll
        for (int d = L / 2; d > 0; d >>= 1) top = max_abs_nan(top, __shfl_xor_sync(0xffffffffu, top, d));
      }
      if (!row) continue;
      if (is_q) {
        *reinterpret_cast<uint4*>(p.yq.y + m * p.yq.ts + (h - 2 * p.hk) * p.yq.hs + f0) = pack8(y);
        continue;
      }
      if (slot < 0) continue;
      const long long r = row0 + (static_cast<long long>(is_v ? h - p.hk : h) << p.cache.page_shift);
      if constexpr (FMT == LORA_KV_BF16) {
        *reinterpret_cast<uint4*>(static_cast<bf16*>(is_v ? p.cache.v : p.cache.k) + r * D + f0) = pack8(y);
      } else {
        const bool fine = top < INFINITY;
        const float scale = fine ? fmaxf(__fmul_rn(top, 1.0f / Quant<FMT>::kTop), 1.17549435e-38f) : __uint_as_float(0x7FC00000u);
        const float inv = __frcp_rn(scale);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __fmul_rn(y[e], inv);
        uint2 c = Quant<FMT>::codes(y);
        if (!fine) c = make_uint2(0, 0);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? p.cache.v : p.cache.k) + r * D + f0) = c;
        if (f0 == 0) (is_v ? p.cache.vs : p.cache.ks)[r] = scale;
      }
    }
    }
  }
}

struct ReadParams {
  CacheArgs cache;
  const int* table;
  long long max_pages;
  const int* cu;
  int n_seqs;
  long long total;
  bf16* k;
  bf16* v;
  int per_group, groups;     // rows (k's heads, then v's) a lane group walks; such groups
  unsigned* status;
};

__device__ __forceinline__ float code_value(uint8_t c, int fmt) {
  if (fmt == LORA_KV_INT8) return static_cast<float>(static_cast<int8_t>(c));
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

// (blocks of 256 an SM and rows in flight a lane: 3 and 8 took 31.0, 6 and 4 28.1, 7 and 4
// 29.4 us for the 24,000 int8 positions of eight sequences)
template <int D, int FMT>
__global__ void __launch_bounds__(256, 6) read_kernel(const __grid_constant__ ReadParams p) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int L = D / 8;
  const int f0 = (threadIdx.x % L) * 8;
  const int hk = p.cache.heads;
  const unsigned long long units = static_cast<unsigned long long>(p.total) * p.groups;
  const unsigned long long step = static_cast<unsigned long long>(gridDim.x) * (256 / L);
  for (unsigned long long u = static_cast<unsigned long long>(blockIdx.x) * (256 / L) + threadIdx.x / L; u < units;
       u += step) {
    const long long r = static_cast<long long>(u / static_cast<unsigned>(p.groups));
    const int g = static_cast<int>(u - static_cast<unsigned long long>(r) * p.groups);
    const int b = owner_of(p.cu, p.n_seqs, r);
    long long page = -1;
    int off = 0;
    if (b >= 0) {
      const long long i = r - __ldg(p.cu + b);
      const long long at = i >> p.cache.page_shift;
      off = static_cast<int>(i & ((1 << p.cache.page_shift) - 1));
      if (at < p.max_pages) page = __ldg(p.table + b * p.max_pages + at);
    }
    if (page < 0 || page >= p.cache.n_pages) {
      atomicOr(p.status, kStatusInput);
      page = -1;
    }
    const int h0 = g * p.per_group, h1 = min(h0 + p.per_group, 2 * hk);
    auto dst = [&](int h) { return (h >= hk ? p.v : p.k) + (r * hk + (h >= hk ? h - hk : h)) * D + f0; };
    if (page < 0) {
      for (int h = h0; h < h1; ++h) *reinterpret_cast<uint4*>(dst(h)) = make_uint4(0, 0, 0, 0);
      continue;
    }
    constexpr int kBatch = 4;
    for (int hb = h0; hb < h1; hb += kBatch) {
      uint4 w[kBatch];                 // the codes of 8-bit formats are its first half
      float scale[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = hb + i;
        if (h >= h1) break;
        const bool is_v = h >= hk;
        const long long src = ((page * hk + (is_v ? h - hk : h)) << p.cache.page_shift) + off;
        const void* base = is_v ? p.cache.v : p.cache.k;
        if constexpr (FMT == LORA_KV_BF16) {
          w[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const bf16*>(base) + src * D + f0));
        } else {
          const uint2 c = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(base) + src * D + f0));
          w[i].x = c.x, w[i].y = c.y;
          scale[i] = __ldg((is_v ? p.cache.vs : p.cache.ks) + src);
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (hb + i >= h1) break;
        if constexpr (FMT != LORA_KV_BF16) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            y[e] = code_value(static_cast<uint8_t>((e < 4 ? w[i].x : w[i].y) >> (8 * (e % 4))), FMT) * scale[i];
          w[i] = pack8(y);
        }
        *reinterpret_cast<uint4*>(dst(hb + i)) = w[i];
      }
    }
  }
}

typedef void (*AppendKernel)(const AppendParams);
typedef void (*ReadKernel)(const ReadParams);

template <int D>
static AppendKernel append_of(int fmt, bool vec) {
  if (fmt == LORA_KV_BF16) return vec ? append_kernel<D, LORA_KV_BF16, true> : append_kernel<D, LORA_KV_BF16, false>;
  if (fmt == LORA_KV_FP8) return vec ? append_kernel<D, LORA_KV_FP8, true> : append_kernel<D, LORA_KV_FP8, false>;
  return vec ? append_kernel<D, LORA_KV_INT8, true> : append_kernel<D, LORA_KV_INT8, false>;
}
template <int D>
static ReadKernel read_of(int fmt) {
  return fmt == LORA_KV_BF16 ? read_kernel<D, LORA_KV_BF16>
                             : fmt == LORA_KV_FP8 ? read_kernel<D, LORA_KV_FP8> : read_kernel<D, LORA_KV_INT8>;
}

}  // namespace lgb

using namespace lgb;

extern "C" lora_status_t lora_kv_append(int64_t M, const lora_kv_cache_t* cache, const lora_heads_t* k,
                                        const lora_heads_t* v, const int64_t* slots, const lora_heads_t* q,
                                        const lora_heads_t* yq, const lora_rotary_t* rot, void* ws, size_t ws_bytes,
                                        cudaStream_t stream) {
  NvtxRange nvtx_range("lora_kv_append");
  const bool with_q = q != nullptr && q->data != nullptr;
  if (M < 0 || !k || !v || (with_q && (!yq || !rot))) return LORA_ERR_INVALID_ARG;
  if (M > 0 && ((rot && !rot->pos) || !k->data || !v->data || !slots || (with_q && !yq->data))) return LORA_ERR_INVALID_ARG;
  LGB_TRY(check_cache(cache));
  if (k->heads != cache->heads || v->heads != cache->heads) return LORA_ERR_INVALID_ARG;
  if (M > kMaxExtent) return LORA_ERR_UNSUPPORTED;
  LGB_TRY(check_heads_in(k));
  LGB_TRY(check_heads_in(v));
  if (rot) LGB_TRY(check_rotary(rot, cache->head_dim));
  if (with_q) {
    LGB_TRY(check_heads_in(q));
    LGB_TRY(check_heads_out(yq, M, cache->head_dim));
    if (yq->heads != q->heads) return LORA_ERR_INVALID_ARG;
  }
  if (!aligned(slots, 8)) return LORA_ERR_ALIGNMENT;
  LGB_TRY(check_ws(ws, ws_bytes, kWsHeader));
  if (M == 0) return LORA_OK;
  AppendParams p;
  std::memset(&p, 0, sizeof(p));
  p.k = HeadsView{static_cast<const bf16*>(k->data), k->token_stride, k->head_stride};
  p.v = HeadsView{static_cast<const bf16*>(v->data), v->token_stride, v->head_stride};
  p.hk = static_cast<int>(cache->heads);
  if (with_q) {
    p.q = HeadsView{static_cast<const bf16*>(q->data), q->token_stride, q->head_stride};
    p.yq = HeadsOut{static_cast<bf16*>(yq->data), yq->token_stride, yq->head_stride};
    p.hq = static_cast<int>(q->heads);
  }
  p.M = M;
  p.slots = reinterpret_cast<const long long*>(slots);
  p.cache = cache_args(cache);
  p.rotate = rot != nullptr;
  if (rot) {
    p.rot = rotary_args(rot);
    p.interleaved = rot->layout == LORA_ROTARY_INTERLEAVED;
  }
  const int D = cache->head_dim, heads = 2 * p.hk + p.hq;
  p.per_group = heads_per_group(M, D / 8, heads);
  p.groups = static_cast<int>(ceil_div(heads, p.per_group));
  p.status = static_cast<unsigned*>(ws);
  const bool vec = rot == nullptr || rot->rot_dim % 16 == 0;
  const AppendKernel f = D == 64 ? append_of<64>(cache->format, vec)
                                 : D == 128 ? append_of<128>(cache->format, vec) : append_of<256>(cache->format, vec);
  const int64_t blocks = ceil_div(M * p.groups, kAppendThreads / (D / 8));
  return launch_counted(f, dim3(static_cast<unsigned>(blocks < (1 << 30) ? blocks : (1 << 30))), dim3(kAppendThreads), 0,
                        LORA_KIND_CACHE, stream, p);
}

extern "C" lora_status_t lora_kv_read(int64_t n_seqs, int64_t total, const lora_kv_cache_t* cache,
                                      const int32_t* page_table, int64_t max_pages, const int32_t* cu_kv, void* k,
                                      void* v, void* ws, size_t ws_bytes, cudaStream_t stream) {
  NvtxRange nvtx_range("lora_kv_read");
  if (n_seqs < 1 || total < 0 || !page_table || max_pages < 1 || !cu_kv || (total > 0 && (!k || !v)))
    return LORA_ERR_INVALID_ARG;
  LGB_TRY(check_cache(cache));
  if (total > kMaxExtent || n_seqs > kMaxExtent || max_pages > kMaxExtent) return LORA_ERR_UNSUPPORTED;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(page_table, 4) || !aligned(cu_kv, 4)) return LORA_ERR_ALIGNMENT;
  LGB_TRY(check_ws(ws, ws_bytes, kWsHeader));
  if (total == 0) return LORA_OK;
  ReadParams p;
  p.cache = cache_args(cache);
  p.table = page_table;
  p.max_pages = max_pages;
  p.cu = cu_kv;
  p.n_seqs = static_cast<int>(n_seqs);
  p.total = total;
  p.k = static_cast<bf16*>(k);
  p.v = static_cast<bf16*>(v);
  const int D = cache->head_dim, rows = 2 * cache->heads;
  p.per_group = heads_per_group(total, D / 8, rows);
  p.groups = static_cast<int>(ceil_div(rows, p.per_group));
  p.status = static_cast<unsigned*>(ws);
  const ReadKernel f = D == 64 ? read_of<64>(cache->format) : D == 128 ? read_of<128>(cache->format)
                                                                      : read_of<256>(cache->format);
  const int64_t blocks = ceil_div(total * p.groups, 256 / (D / 8));
  return launch_counted(f, dim3(static_cast<unsigned>(blocks < (1 << 30) ? blocks : (1 << 30))), dim3(256), 0,
                        LORA_KIND_CACHE, stream, p);
}
