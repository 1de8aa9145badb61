// RMS norm with the residual's addition, in bf16 or in 8-bit codes with a scale for each row
// (lora_rms_norm), and its gradient (lora_rms_norm_backward); include/lora_gb300.h is the
// contract.
//
// Both read and write every byte once, so memory bounds them.  A row belongs to T neighbouring
// threads that hold it in registers, NV pieces of 8 features each, between the sum over the
// row and its use; T grows with the row so that a thread has two to eight loads in flight.
// Measured: 8192 rows of 4096, residual added, e4m3 out, 235 MB in 38.3 us (6.1 TB/s, 91% of a copy's
// rate; 256 threads with 2 pieces, 38.5 with 128 and 4, 46.4 with 512 and 1); 131,168 rows of 128 as
// slices of a packed buffer, 68 MB in 14.3 us (17.8 with one row a group of threads); 16 rows of 896
// 2.1 us in a graph.  The gradient of 4095 rows of 4096 with ds and dweight, 134 MB in 27.2 us (4.9
// TB/s, 74%; 32.8 with the next row's loads in registers), 3 of them the join of the blocks' dweight.
// Narrow rows' gradient with dweight, L2 flushed between replays: 131,168 rows of 128 36.0 us, of 256
// 52.4 (42.1 and 62.6 while the block's join had shared memory of its own and seven blocks an SM fitted).
#include "serve.cuh"

namespace lgb {

struct NormArgs {
  HeadsView x, res;          // res.x NULL: no residual
  HeadsOut sum;              // sum.y NULL: not written
  const bf16* w;
  float offset, eps;
  long long rows;
  int heads, dim;
  void* y;
  float* y_scale;
  float* rstd;
};

struct NormGradArgs {
  HeadsView dy, s, ds;       // ds.x NULL: none
  const bf16* w;
  float offset;
  const float* rstd;
  long long rows;
  int heads, dim;
  bf16* dx;
  float* part;               // [blocks][dim] sums for dweight, or NULL
};

// Element offset of a row of a view.
__device__ __forceinline__ long long row_offset(long long r, int heads, long long ts, long long hs) {
  if (heads == 1) return r * ts;
  const unsigned m = static_cast<unsigned>(r) / static_cast<unsigned>(heads);      // r is below 2^31
  return m * ts + static_cast<int>(static_cast<unsigned>(r) - m * heads) * hs;
}

// Sum (or NaN-keeping maximum) over the T threads of a row: shuffles, and for rows wider than a
// warp one exchange through shared memory, whose slots alternate so that one barrier is enough.
template <int T, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* slots) {
#pragma unroll
  for (int d = (T < 32 ? T : 32) / 2; d > 0; d >>= 1) {
    const float o = __shfl_xor_sync(0xffffffffu, v, d);
    v = MAX ? max_abs_nan(v, o) : v + o;
  }
  if constexpr (T > 32) {
    if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
    __syncthreads();
    v = slots[threadIdx.x & (T / 32 - 1)];
#pragma unroll
    for (int d = T / 64; d > 0; d >>= 1) {
      const float o = __shfl_xor_sync(0xffffffffu, v, d);
      v = MAX ? max_abs_nan(v, o) : v + o;
    }
  }
  return v;
}

constexpr int norm_threads(int t) { return t <= 32 ? 128 : t; }

// R: rows a group of threads takes at once, so that narrow rows too have loads in flight.
template <int T, int NV, int R, int FMT>
__global__ void __launch_bounds__(norm_threads(T)) norm_kernel(const __grid_constant__ NormArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kRows = norm_threads(T) / T;     // groups of a block
  __shared__ float slots[3][32];
  const int t = threadIdx.x % T;
  // a group's rows are kRows apart, so that a block's rows stay together
  const long long r0 = static_cast<long long>(blockIdx.x) * (kRows * R) + threadIdx.x / T;
  uint4 w[R][NV];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const long long r = r0 + j * kRows;
    const bf16* x = p.x.x + (r < p.rows ? row_offset(r, p.heads, p.x.ts, p.x.hs) : 0);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (i * T + t);
      w[j][i] = r < p.rows && c < p.dim ? *reinterpret_cast<const uint4*>(x + c) : make_uint4(0, 0, 0, 0);
    }
  }
  if (p.res.x != nullptr) {
    uint4 v[R][NV];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const long long r = r0 + j * kRows;
      const bf16* res = p.res.x + (r < p.rows ? row_offset(r, p.heads, p.res.ts, p.res.hs) : 0);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = 8 * (i * T + t);
        v[j][i] = r < p.rows && c < p.dim ? *reinterpret_cast<const uint4*>(res + c) : make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const long long r = r0 + j * kRows;
      bf16* sum = p.sum.y + (r < p.rows ? row_offset(r, p.heads, p.sum.ts, p.sum.hs) : 0);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = 8 * (i * T + t);
        float a[8], b[8];
        unpack8(w[j][i], a);
        unpack8(v[j][i], b);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] += b[e];
        w[j][i] = pack8(a);
        if (r < p.rows && c < p.dim) *reinterpret_cast<uint4*>(sum + c) = w[j][i];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const long long r = r0 + j * kRows;
    const bool live = r < p.rows;
    // sum of the squares of k times the row
    auto squares = [&](float k, float* joint) {
      float sq = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float a[8];
        unpack8(w[j][i], a);
#pragma unroll
        for (int e = 0; e < 8; ++e) sq = fmaf(k * a[e], k * a[e], sq);
      }
      return row_reduce<T, false>(sq, joint);
    };
    const float sq = squares(1.0f, slots[0]);
    float rstd = rsqrtf(sq / static_cast<float>(p.dim) + p.eps);
    // A row whose squares leave f32's range (above, or below where eps does not cover it) is
    // summed again 2^80 smaller, where 32768 squares of bf16's largest value are below 2^112, or 2^70 larger.
    const bool again = sq == INFINITY || (sq < 1e-24f && p.eps < 1e-18f);
    if (T > 32 ? again : __any_sync(0xffffffffu, again)) {
      const float k = sq == INFINITY ? 0x1p-80f : 0x1p70f;
      const float q = squares(k, slots[2]);
      if (again) rstd = rsqrtf(q / static_cast<float>(p.dim) + p.eps * k * k) * k;
    }
    if (live && t == 0 && p.rstd != nullptr) p.rstd[r] = rstd;
    // y of one piece, not rounded
    auto piece = [&](int i, float (&y)[8]) {
      const int c = 8 * (i * T + t);
      float g[8];
      unpack8(c < p.dim ? __ldg(reinterpret_cast<const uint4*>(p.w + c)) : make_uint4(0, 0, 0, 0), g);
      unpack8(w[j][i], y);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = y[e] * rstd * (g[e] + p.offset);
    };
    if constexpr (FMT == LORA_NORM_BF16) {
      bf16* out = static_cast<bf16*>(p.y) + r * p.dim;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = 8 * (i * T + t);
        float y[8];
        piece(i, y);
        if (live && c < p.dim) *reinterpret_cast<uint4*>(out + c) = pack8(y);
      }
    } else {
      // (y is computed twice rather than held: registers)
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float y[8];
        piece(i, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max_abs_nan(top, y[e]);
      }
      top = row_reduce<T, true>(top, slots[1]);
      const bool fine = top < INFINITY;
      const float scale = fine ? fmaxf(__fmul_rn(top, 1.0f / Quant<LORA_KV_FP8>::kTop), 1.17549435e-38f) : __uint_as_float(0x7FC00000u);
      const float inv = __frcp_rn(scale);
      uint8_t* out = static_cast<uint8_t*>(p.y) + r * p.dim;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = 8 * (i * T + t);
        float y[8];
        piece(i, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __fmul_rn(y[e], inv);
        uint2 codes = Quant<LORA_KV_FP8>::codes(y);
        if (!fine) codes = make_uint2(0, 0);
        if (live && c < p.dim) *reinterpret_cast<uint2*>(out + c) = codes;
      }
      if (live && t == 0) p.y_scale[r] = scale;
    }
  }
}

// Resident blocks of the gradient's kernel on an SM: 1024 threads, so 64 registers each.
constexpr int norm_grad_blocks_sm(int t) { return 1024 / norm_threads(t); }

// Rows a thread has on their way, in a ring of its own in shared memory (48 bytes a piece and row
// of dy, s and ds): 192 KB of an SM's.
constexpr int norm_grad_stages(int nv) { return 4 / nv; }
constexpr int norm_grad_smem(int t, int nv) { return norm_threads(t) * nv * norm_grad_stages(nv) * 48; }

// The GPU is filled once and blocks walk rows with a stride.  A thread copies its own pieces of the
// next rows to shared memory ahead of their use (nobody else reads them: no barrier).  Its features
// stay the same, so it sums its part of dweight in registers and leaves one partial row a block.
template <int T, int NV, bool DW>
__global__ void __launch_bounds__(norm_threads(T), norm_grad_blocks_sm(T)) norm_grad_kernel(const __grid_constant__ NormGradArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kThreadsOf = norm_threads(T), kRows = kThreadsOf / T, kStages = norm_grad_stages(NV);
  __shared__ float slots[2][32];
  extern __shared__ __align__(16) uint4 ring[];   // [stage][tensor][piece][thread]
  const int t = threadIdx.x % T;
  const float inv_dim = 1.0f / static_cast<float>(p.dim);
  const long long step = static_cast<long long>(gridDim.x) * kRows;
  const bool add = p.ds.x != nullptr;
  float dw[DW ? NV : 1][8];
  uint4 wg[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * (i * T + t);
    wg[i] = c < p.dim ? __ldg(reinterpret_cast<const uint4*>(p.w + c)) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < (DW ? NV : 1); ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.0f;
  auto at = [&](int stage, int tensor, int i) { return ring + ((stage * 3 + tensor) * NV + i) * kThreadsOf + threadIdx.x; };
  auto fetch = [&](long long r, int stage) {
    if (r < p.rows) {
      const bf16* dy = p.dy.x + row_offset(r, p.heads, p.dy.ts, p.dy.hs);
      const bf16* s = p.s.x + row_offset(r, p.heads, p.s.ts, p.s.hs);
      const bf16* ds = add ? p.ds.x + row_offset(r, p.heads, p.ds.ts, p.ds.hs) : nullptr;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = 8 * (i * T + t);
        if (c >= p.dim) continue;
        copy16_async(at(stage, 0, i), dy + c);
        copy16_async(at(stage, 1, i), s + c);
        if (add) copy16_async(at(stage, 2, i), ds + c);
      }
    }
    copy_async_commit();
  };
  const long long first = static_cast<long long>(blockIdx.x) * kRows + threadIdx.x / T;
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) fetch(first + k * step, k);
  float rstd = first < p.rows ? __ldg(p.rstd + first) : 0.0f;
  int turn = 0, stage = 0;
  for (long long base = static_cast<long long>(blockIdx.x) * kRows; base < p.rows; base += step) {
    const long long r = base + threadIdx.x / T;
    const bool live = r < p.rows;
    fetch(r + (kStages - 1) * step, (stage + kStages - 1) % kStages);
    copy_async_wait<kStages - 1>();
    const float rstd_next = r + step < p.rows ? __ldg(p.rstd + r + step) : 0.0f;
    uint4 wy[NV], ws[NV];
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool own = live && 8 * (i * T + t) < p.dim;
      wy[i] = own ? *at(stage, 0, i) : make_uint4(0, 0, 0, 0);
      ws[i] = own ? *at(stage, 1, i) : make_uint4(0, 0, 0, 0);
      float g[8], a[8], n[8];
      unpack8(wg[i], g);
      unpack8(wy[i], a);
      unpack8(ws[i], n);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n[e] *= rstd;
        if (DW) dw[i][e] = fmaf(a[e], n[e], dw[i][e]);
        dot = fmaf(a[e] * (g[e] + p.offset), n[e], dot);
      }
    }
    dot = row_reduce<T, false>(dot, slots[turn]) * inv_dim;
    turn ^= 1;
    if (live) {
      bf16* dx = p.dx + r * p.dim;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = 8 * (i * T + t);
        if (c >= p.dim) continue;
        float g[8], a[8], n[8];
        unpack8(wg[i], g);
        unpack8(wy[i], a);
        unpack8(ws[i], n);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] = rstd * (a[e] * (g[e] + p.offset) - n[e] * rstd * dot);
        if (add) {
          unpack8(*at(stage, 2, i), n);
#pragma unroll
          for (int e = 0; e < 8; ++e) a[e] += n[e];
        }
        *reinterpret_cast<uint4*>(dx + c) = pack8(a);
      }
    }
    rstd = rstd_next;
    stage = (stage + 1) % kStages;
  }
  if constexpr (DW) {
    // the block's row groups, summed in their order
    float* out = p.part + static_cast<long long>(blockIdx.x) * p.dim;
    if constexpr (kRows > 1) {
      // (in the ring, whose copies have all been waited for: 4 KB more would cost the SM's eighth block)
      static_assert(kRows * 8 * T * NV * 4 <= norm_grad_smem(T, NV));
      auto* join = reinterpret_cast<float (*)[8 * T * NV]>(ring);
      copy_async_wait<0>();
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) join[threadIdx.x / T][8 * (i * T + t) + e] = dw[i][e];
      __syncthreads();
      for (int c = threadIdx.x; c < p.dim; c += norm_threads(T)) {
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < kRows; ++k) v += join[k][c];
        out[c] = v;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = 8 * (i * T + t);
        if (c >= p.dim) continue;
        *reinterpret_cast<float4*>(out + c) = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
        *reinterpret_cast<float4*>(out + c + 4) = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
      }
    }
  }
}

struct NormSumArgs {
  const float* part;
  int blocks, dim;
  bf16* dw;
};

// dweight of the blocks' partial rows, in their order: 32 features a block, 16 threads each.
__global__ void __launch_bounds__(512) norm_sum_kernel(const __grid_constant__ NormSumArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float join[16][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
  float v = 0.0f;
  if (c < p.dim) {
#pragma unroll 8
    for (int b = k; b < p.blocks; b += 16) v += __ldcg(p.part + static_cast<long long>(b) * p.dim + c);
  }
  join[k][threadIdx.x & 31] = v;
  __syncthreads();
  if (k != 0 || c >= p.dim) return;
#pragma unroll
  for (int j = 1; j < 16; ++j) v += join[j][threadIdx.x];
  p.dw[c] = __float2bfloat16_rn(v);
}

// Calls f with the row's shape as tags (threads, pieces a thread).
template <int V>
struct IntTag {
  static constexpr int value = V;
};
template <typename F>
lora_status_t norm_shape(int dim, F&& f) {
  const int n = dim / 8;
  if (n <= 8) return f(IntTag<8>{}, IntTag<1>{});
  if (n <= 16) return f(IntTag<16>{}, IntTag<1>{});
  if (n <= 32) return f(IntTag<32>{}, IntTag<1>{});
  if (n <= 64) return f(IntTag<32>{}, IntTag<2>{});
  if (n <= 128) return f(IntTag<32>{}, IntTag<4>{});
  if (n <= 256) return f(IntTag<128>{}, IntTag<2>{});
  if (n <= 512) return f(IntTag<256>{}, IntTag<2>{});
  if (n <= 1024) return f(IntTag<256>{}, IntTag<4>{});
  if (n <= 2048) return f(IntTag<512>{}, IntTag<4>{});
  return f(IntTag<1024>{}, IntTag<4>{});
}
// The gradient's: one piece a thread as far as blocks reach.
template <typename F>
lora_status_t norm_grad_shape(int dim, F&& f) {
  const int n = dim / 8;
  if (n <= 8) return f(IntTag<8>{}, IntTag<1>{});
  if (n <= 16) return f(IntTag<16>{}, IntTag<1>{});
  if (n <= 32) return f(IntTag<32>{}, IntTag<1>{});
  if (n <= 64) return f(IntTag<64>{}, IntTag<1>{});
  if (n <= 128) return f(IntTag<128>{}, IntTag<1>{});
  if (n <= 256) return f(IntTag<256>{}, IntTag<1>{});
  if (n <= 512) return f(IntTag<512>{}, IntTag<1>{});
  if (n <= 1024) return f(IntTag<1024>{}, IntTag<1>{});
  if (n <= 2048) return f(IntTag<1024>{}, IntTag<2>{});
  return f(IntTag<1024>{}, IntTag<4>{});
}

constexpr int kNormMaxDim = 32768;
constexpr int kNormSms = 152;               // blocks of the gradient, and so the partial rows of dweight that
                                            // size the workspace, are those of a GB300

// Blocks of the gradient's kernel: as many as the GPU holds, or the rows fill.
static int64_t norm_grad_blocks(int64_t rows, int dim) {
  int64_t blocks = 0;
  norm_grad_shape(dim, [&](auto t, auto) {
    constexpr int T = decltype(t)::value;
    const int64_t need = ceil_div(rows, norm_threads(T) / T), most = kNormSms * norm_grad_blocks_sm(T);
    blocks = need < most ? need : most;
    return LORA_OK;
  });
  return blocks;
}

template <int T, int NV, bool DW>
static lora_status_t launch_norm_grad(const NormGradArgs& p, int64_t blocks, cudaStream_t st) {
  auto* k = norm_grad_kernel<T, NV, DW>;
  static std::atomic<unsigned long long> configured{0};
  if (ensure_smem_limit(k, norm_grad_smem(T, NV), configured) != cudaSuccess) return LORA_ERR_CUDA;
  return launch_counted(k, dim3(static_cast<unsigned>(blocks)), dim3(norm_threads(T)), norm_grad_smem(T, NV), LORA_KIND_NORM, st, p);
}

static bool present(const lora_heads_t* v) { return v != nullptr && v->data != nullptr; }
static lora_status_t check_norm_sizes(int64_t M, int64_t heads, int dim) {
  if (M < 0 || heads < 1 || dim < 1) return LORA_ERR_INVALID_ARG;
  if (dim > kNormMaxDim || M > kMaxExtent || heads > kMaxExtent || M > kMaxExtent / heads) return LORA_ERR_UNSUPPORTED;
  return dim % 8 ? LORA_ERR_ALIGNMENT : LORA_OK;
}
static HeadsView view_of(const lora_heads_t* v) {
  return present(v) ? HeadsView{static_cast<const bf16*>(v->data), v->token_stride, v->head_stride} : HeadsView{nullptr, 0, 0};
}

}  // namespace lgb

using namespace lgb;

extern "C" lora_status_t lora_rms_norm(int64_t M, int dim, const lora_heads_t* x, const lora_heads_t* residual,
                                       const void* weight, float offset, float eps, int format, const lora_heads_t* sum,
                                       void* y, float* y_scale, float* rstd, void* ws, size_t ws_bytes,
                                       cudaStream_t stream) {
  NvtxRange nvtx_range("lora_rms_norm");
  if (!x || !weight || !std::isfinite(offset) || !std::isfinite(eps) || eps < 0.0f ||
      (format != LORA_NORM_BF16 && format != LORA_NORM_FP8) || (y_scale != nullptr) != (format == LORA_NORM_FP8))
    return LORA_ERR_INVALID_ARG;
  LGB_TRY(check_norm_sizes(M, x->heads, dim));
  if (M > 0 && (!x->data || !y)) return LORA_ERR_INVALID_ARG;
  const bool add = present(residual);
  if (add != present(sum)) return LORA_ERR_INVALID_ARG;
  LGB_TRY(check_heads_in(x));
  if (add) {
    if (residual->heads != x->heads || sum->heads != x->heads) return LORA_ERR_INVALID_ARG;
    LGB_TRY(check_heads_in(residual));
    LGB_TRY(check_heads_out(sum, M, dim));
  }
  if (!aligned(weight, 16) || !aligned(y, format == LORA_NORM_FP8 ? 8 : 16) || !aligned(y_scale, 4) || !aligned(rstd, 4)) return LORA_ERR_ALIGNMENT;
  LGB_TRY(check_ws(ws, ws_bytes, kWsHeader));
  if (M == 0) return LORA_OK;
  NormArgs p;
  p.x = view_of(x);
  p.res = view_of(residual);
  p.sum = add ? HeadsOut{static_cast<bf16*>(sum->data), sum->token_stride, sum->head_stride} : HeadsOut{nullptr, 0, 0};
  p.w = static_cast<const bf16*>(weight);
  p.offset = offset;
  p.eps = eps;
  p.heads = static_cast<int>(x->heads);
  p.rows = M * x->heads;
  p.dim = dim;
  p.y = y;
  p.y_scale = y_scale;
  p.rstd = rstd;
  return norm_shape(dim, [&](auto t, auto nv) {
    constexpr int T = decltype(t)::value, NV = decltype(nv)::value, K = norm_threads(T) / T;
    constexpr int R = NV == 1 ? 2 : 1;               // (four: 14.8 us instead of 14.3, eight 18.7)
    // several rows a group once that leaves the GPU full
    const bool many = R > 1 && p.rows >= static_cast<int64_t>(num_sms()) * 8 * K * R;
    const unsigned grid = static_cast<unsigned>(ceil_div(p.rows, many ? K * R : K));
    const bool wide = format == LORA_NORM_BF16;
    return launch_counted(many ? (wide ? norm_kernel<T, NV, R, LORA_NORM_BF16> : norm_kernel<T, NV, R, LORA_NORM_FP8>)
                               : (wide ? norm_kernel<T, NV, 1, LORA_NORM_BF16> : norm_kernel<T, NV, 1, LORA_NORM_FP8>),
                          dim3(grid), dim3(norm_threads(T)), 0, LORA_KIND_NORM, stream, p);
  });
}

extern "C" size_t lora_rms_norm_workspace_bytes(int64_t M, int64_t heads, int dim) {
  if (check_norm_sizes(M, heads, dim) != LORA_OK) return 0;
  Carve c(nullptr);
  c.take(kWsHeader);
  c.take_n<float>(norm_grad_blocks(M * heads, dim) * dim);
  return c.off;
}

extern "C" lora_status_t lora_rms_norm_backward(int64_t M, int dim, const lora_heads_t* dy, const lora_heads_t* s,
                                                const void* weight, float offset, const float* rstd,
                                                const lora_heads_t* ds, void* dx, void* dweight, void* ws,
                                                size_t ws_bytes, cudaStream_t stream) {
  NvtxRange nvtx_range("lora_rms_norm_backward");
  if (!dy || !s || !weight || !std::isfinite(offset)) return LORA_ERR_INVALID_ARG;
  LGB_TRY(check_norm_sizes(M, s->heads, dim));
  if (M > 0 && (!dy->data || !s->data || !rstd || !dx)) return LORA_ERR_INVALID_ARG;
  if (dy->heads != s->heads || (present(ds) && ds->heads != s->heads)) return LORA_ERR_INVALID_ARG;
  LGB_TRY(check_heads_in(dy));
  LGB_TRY(check_heads_in(s));
  if (present(ds)) LGB_TRY(check_heads_in(ds));
  if (!aligned(weight, 16) || !aligned(dx, 16) || !aligned(dweight, 2) || !aligned(rstd, 4)) return LORA_ERR_ALIGNMENT;
  LGB_TRY(check_ws(ws, ws_bytes, lora_rms_norm_workspace_bytes(M, s->heads, dim)));
  NormGradArgs p;
  p.dy = view_of(dy);
  p.s = view_of(s);
  p.ds = view_of(ds);
  p.w = static_cast<const bf16*>(weight);
  p.offset = offset;
  p.rstd = rstd;
  p.heads = static_cast<int>(s->heads);
  p.rows = M * s->heads;
  p.dim = dim;
  p.dx = static_cast<bf16*>(dx);
  Carve c(ws);
  c.take(kWsHeader);
  p.part = c.take_n<float>(norm_grad_blocks(p.rows, dim) * dim);
  const bool want = dweight != nullptr;
  const int64_t blocks = norm_grad_blocks(p.rows, dim);
  if (M > 0)
    LGB_TRY(norm_grad_shape(dim, [&](auto t, auto nv) {
      constexpr int T = decltype(t)::value, NV = decltype(nv)::value;
      return want ? launch_norm_grad<T, NV, true>(p, blocks, stream) : launch_norm_grad<T, NV, false>(p, blocks, stream);
    }));
  if (!want) return LORA_OK;
  NormSumArgs q;
  q.part = p.part;
  q.blocks = static_cast<int>(blocks);
  q.dim = dim;
  q.dw = static_cast<bf16*>(dweight);
  return launch_counted(norm_sum_kernel, dim3(static_cast<unsigned>(ceil_div(dim, 32))), dim3(512), 0, LORA_KIND_NORM,
                        stream, q);
}
