// Cross entropy of a frozen head with its gradient (lora_linear_ce); include/lora_gb300.h is
// the contract, gemm_ce.cuh has the GEMMs and the mathematics they share with this file.
//
// A call packs the labelled rows, then takes them piece by piece:
//   loss alone     CE_STATS, join of the row's partial results
//   with dx        reference z_y + 40 for each row (a dot product), CE_GRAD, join, [CE_GRAD and
//                  join again where a row's logits stand 60 above its reference or more],
//                  CE_PART over the exponentials, join of the k-ranges with the label's row of W
//   capped and smoothed at once: CE_STATS, join, CE_GRAD with the sum as its reference, CE_PART
//                  (the smoothing's part of the gradient then depends on each logit's slope)
// A row's largest logit is at least its label's.  So the reference, 40 above the label's logit,
// leaves the largest exponential between e^-40 and, where the largest logit stands less than 100
// above the label's, e^60: it, the sums and the product stay inside the range of f32 and bf16
// (a weight below 2^-68 of the label's counts as zero).  A row beyond that is seen by its sum,
// and its piece's second try takes the row's maximum itself for the reference.
#include "gemm_ce.cuh"
#include "serve.cuh"

namespace lgb {

constexpr float kCeAhead = 40.0f * kLog2e;         // the reference above the label's logit
constexpr float kCeMost = 1.5474250491067253e26f;  // 2^87: a row's sum of exponentials past it is taken again
constexpr int64_t kCeGradBytes = int64_t(1) << 30; // exponentials of a piece
constexpr int64_t kCeStatBytes = int64_t(1) << 28; // partial results of a piece (the loss alone)
constexpr int kCeColumnBlocks = 304;               // row ranges of W for its column sums

// The rows of a call as the kernels see them; arrays over packed rows but for pos.
struct CeRows {
  int* count;              // labelled rows
  int* pos;                // [M] place of a token among them, -1: none
  int* idx;                // token of a packed row
  int* label;
  float* ref2;             // the reference, in units of ln 2 as all logits here
  float* zlab;             // the label's logit
  float* rs;               // factors of the row's gradient: of sum e W, and of W_label
  float* coef;
};

struct CePackArgs {
  const long long* labels;
  long long M;
  long long ignore;
  long long vocab;
  CeRows r;
  CePiece* piece;
  int pieces, piece_rows;
  int tiles_n, kb, pairs;  // of CE_PART
  unsigned* status;
};

// One block: the labelled tokens' places, in order, and what each piece holds.
__global__ void __launch_bounds__(1024) ce_pack_kernel(const __grid_constant__ CePackArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ int warps[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int n = 0;
  for (long long base = 0; base < p.M; base += 4096) {
    const long long m = base + 4 * threadIdx.x;
    long long y[4];
    bool seen[4];
    int mine = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[j] = m + j < p.M ? __ldg(p.labels + m + j) : p.ignore;
      seen[j] = y[j] != p.ignore && m + j < p.M;
      if (seen[j] && (y[j] < 0 || y[j] >= p.vocab)) {
        atomicOr(p.status, kStatusInput);
        seen[j] = false;
      }
      mine += seen[j];
    }
    int upto = mine;                                 // inclusive sums over the warp, then the block
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = upto;
    __syncthreads();
    int total = warps[lane];
    int before = 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, total, d);
      if (lane >= d) total += o;
    }
    before = warp == 0 ? 0 : __shfl_sync(0xffffffffu, total, warp - 1);
    total = __shfl_sync(0xffffffffu, total, 31);
    int at = n + before + upto - mine;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (m + j >= p.M) break;
      p.r.pos[m + j] = seen[j] ? at : -1;
      if (!seen[j]) continue;
      p.r.idx[at] = static_cast<int>(m + j);
      p.r.label[at] = static_cast<int>(y[j]);
      ++at;
    }
    n += total;
  }
  if (threadIdx.x == 0) *p.r.count = n;
  for (int k = threadIdx.x; k < p.pieces; k += 1024) {
    const long long left = n - static_cast<long long>(k) * p.piece_rows;
    CePiece q;
    q.live = left <= 0 ? 0 : left < p.piece_rows ? static_cast<int>(left) : p.piece_rows;
    q.splits = ce_splits((q.live + 255) / 256 * p.tiles_n, p.kb, p.pairs);
    q.redo = 0;
    q.pad = 0;
    p.piece[k] = q;
  }
}

struct CeGatherArgs {
  const bf16* x;
  const bf16* W;
  long long M;
  int h;
  CeRows r;
  bf16* packed;            // [count][h]
  CeLogit lg;
  int want_ref;
  float* loss;
  float* lse;              // NULL: not wanted
  bf16* dx;                // NULL: the loss alone
};

// A warp a token: packs its row and takes the reference from its label's logit, or clears what
// an unlabelled token has.
__global__ void __launch_bounds__(256) ce_gather_kernel(const __grid_constant__ CeGatherArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  for (long long m = blockIdx.x * 8ll + (threadIdx.x >> 5); m < p.M; m += 8ll * gridDim.x) {
    const int at = __ldcg(p.r.pos + m);
    if (at < 0) {
      if (lane == 0) {
        p.loss[m] = 0.0f;
        if (p.lse != nullptr) p.lse[m] = 0.0f;
      }
      if (p.dx != nullptr)
        for (int c = 8 * lane; c < p.h; c += 256) *reinterpret_cast<uint4*>(p.dx + m * p.h + c) = make_uint4(0, 0, 0, 0);
      continue;
    }
    const bf16* x = p.x + m * p.h;
    const bf16* w = p.W + static_cast<long long>(__ldcg(p.r.label + at)) * p.h;
    bf16* out = p.packed + static_cast<long long>(at) * p.h;
    float dot = 0.0f;
#pragma unroll 4
    for (int c = 8 * lane; c < p.h; c += 256) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(x + c));
      *reinterpret_cast<uint4*>(out + c) = v;
      if (p.want_ref) {
        float a[8], b[8];
        unpack8(v, a);
        unpack8(__ldg(reinterpret_cast<const uint4*>(w + c)), b);
#pragma unroll
        for (int e = 0; e < 8; ++e) dot = fmaf(a[e], b[e], dot);
      }
    }
    if (!p.want_ref) continue;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
    if (lane == 0) {
      float slope;
      p.r.ref2[at] = (p.lg.cap2 > 0.0f ? ce_logit<true>(dot, p.lg, slope) : ce_logit<false>(dot, p.lg, slope)) + kCeAhead;
    }
  }
}

enum CeJoin : int { CE_JOIN_LOSS = 0, CE_JOIN_EXACT = 1, CE_JOIN_GRAD = 2, CE_JOIN_REDO = 3 };
struct CeJoinArgs {
  CePiece* piece;
  int mode;
  CeRows r;                // at the piece's first row (count: the call's)
  const float2* part;
  const float* zsum;
  long long ldp;
  int slots;
  int vocab;
  float cap2;              // 0: no cap
  float scale, smoothing;
  int mean;
  float* loss;             // by token
  float* lse;
};

constexpr int kJoinWarps = 16;

// The partial results of 32 rows, a lane a row, shared out over the block's warps and joined in
// a fixed order; then the row's loss and its factors.
__global__ void __launch_bounds__(32 * kJoinWarps) ce_join_kernel(const __grid_constant__ CeJoinArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float tops[kJoinWarps][32], sums[kJoinWarps][32], zs[kJoinWarps][32];
  const int live = __ldcg(&p.piece->live);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x * 32 + lane;
  if (static_cast<int>(blockIdx.x) * 32 >= live) return;
  if (p.mode == CE_JOIN_REDO && __ldcg(&p.piece->redo) == 0) return;
  const bool ok = row < live, relative = p.mode <= CE_JOIN_EXACT;
  float top = -INFINITY, sum = 0.0f, z = 0.0f;
  auto add = [&](float t, float s) {
    if (!relative) {
      sum += s;
      top = fmaxf(top, t);
      return;
    }
    // sums relative to their own maxima; an empty one (no column but the label's) adds nothing
    if (t == -INFINITY && s == 0.0f) return;
    const float most = fmaxf(top, t);
    sum = sum * exp2f(top - most) + s * exp2f(t - most);
    top = most;
  };
  if (ok) {
#pragma unroll 8
    for (int k = warp; k < p.slots; k += kJoinWarps) {
      const float2 o = __ldcg(p.part + k * p.ldp + row);
      add(o.x, o.y);
      if (p.zsum != nullptr) z += __ldcg(p.zsum + k * p.ldp + row);
    }
  }
  tops[warp][lane] = top;
  sums[warp][lane] = sum;
  zs[warp][lane] = z;
  __syncthreads();
  if (warp != 0 || !ok) return;
  for (int k = 1; k < kJoinWarps; ++k) {
    add(tops[k][lane], sums[k][lane]);
    z += zs[k][lane];
  }
  const float zl = __ldcg(p.r.zlab + row), ref2 = relative ? top : p.r.ref2[row];
  if (p.mode == CE_JOIN_GRAD && sum > kCeMost) {     // the row's place is off: take it again from its maximum
    p.r.ref2[row] = top;
    p.piece->redo = 1;                               // (every writer writes the same)
  }
  // d: the others' log-sum over the label's logit, in units of ln 2
  const float others = ref2 + log2f(sum), d = others - zl;
  const float tail = log1pf(exp2f(-fabsf(d)));
  const float ce = d > 0.0f ? fmaf(d, kLn2, tail) : tail;
  const int token = __ldg(p.r.idx + row);
  const float eps = p.smoothing;
  p.loss[token] = p.zsum != nullptr ? ce + eps * kLn2 * (zl - z / p.vocab) : ce;
  if (p.lse != nullptr) p.lse[token] = fmaf(zl, kLn2, ce);
  if (p.mode == CE_JOIN_LOSS) return;
  const int n = __ldcg(p.r.count);
  const float g = p.scale / (p.mean ? static_cast<float>(n) : 1.0f);
  float slope = 1.0f;
  if (p.cap2 > 0.0f) {
    const float t = zl / p.cap2;
    slope = 1.0f - t * t;
  }
  const float away = expm1f(-ce);                    // p_label - 1
  if (p.mode == CE_JOIN_EXACT) {
    p.r.ref2[row] = fmaf(zl, 1.0f, ce * kLog2e);
    p.r.rs[row] = g;
    p.r.coef[row] = g * slope * (away + eps - eps / p.vocab);
  } else {
    p.r.rs[row] = g / (sum + exp2f(zl - ref2));
    p.r.coef[row] = g * slope * (away + eps);
  }
}

struct CeColumnArgs {
  const bf16* W;
  long long vocab;
  int h;
  float* part;             // [gridDim.y][h]
  float* sum;              // [h]
};
// Column sums of W (the smoothing's part of the gradient): row ranges, then their join.
__global__ void __launch_bounds__(128) ce_column_kernel(const __grid_constant__ CeColumnArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  const int c = 8 * (blockIdx.x * 128 + threadIdx.x);
  if (c >= p.h) return;
  const long long a = p.vocab * blockIdx.y / gridDim.y, b = p.vocab * (blockIdx.y + 1) / gridDim.y;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
#pragma unroll 8
  for (long long v = a; v < b; ++v) {
    float w[8];
    unpack8(__ldg(reinterpret_cast<const uint4*>(p.W + v * p.h + c)), w);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += w[e];
  }
  float* out = p.part + static_cast<long long>(blockIdx.y) * p.h + c;
  *reinterpret_cast<float4*>(out) = make_float4(acc[0], acc[1], acc[2], acc[3]);
  *reinterpret_cast<float4*>(out + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
}
__global__ void __launch_bounds__(256) ce_column_join_kernel(const __grid_constant__ CeColumnArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float join[8][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
  float v = 0.0f;
  if (c < p.h)
    for (int b = k; b < kCeColumnBlocks; b += 8) v += __ldcg(p.part + static_cast<long long>(b) * p.h + c);
  join[k][threadIdx.x & 31] = v;
  __syncthreads();
  if (k != 0 || c >= p.h) return;
#pragma unroll
  for (int j = 1; j < 8; ++j) v += join[j][threadIdx.x];
  p.sum[c] = v;
}

struct CeDxArgs {
  const CePiece* piece;
  CeRows r;                // at the piece's first row
  const float* slab;
  int tiles_n, h;
  const bf16* W;
  const float* column;     // column sums of W, or NULL
  float scale, share;      // logit scale, smoothing / vocab
  int mean;
  bf16* dx;
};
// dx rows of a piece: the k-ranges' sums times the row's factor, the label's row of W, and the
// smoothing's part.  A thread takes eight features.
__global__ void __launch_bounds__(256) ce_dx_kernel(const __grid_constant__ CeDxArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  const int live = __ldcg(&p.piece->live), splits = __ldcg(&p.piece->splits);
  const int per = p.h / 8;
  const long long tiles = static_cast<long long>((live + 255) / 256) * p.tiles_n, total = static_cast<long long>(live) * per;
  const int n = __ldcg(p.r.count);
  const float flat = p.column == nullptr ? 0.0f : p.scale * p.share / (p.mean ? static_cast<float>(n) : 1.0f);
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += 256ll * gridDim.x) {
    const int row = static_cast<int>(i / per), c = 8 * static_cast<int>(i - static_cast<long long>(row) * per);
    const float* src = p.slab + ((static_cast<long long>(row >> 8) * p.tiles_n + (c >> 8)) * 256 + (row & 255)) * 256 + (c & 255);
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      const uint4 a = ld_global_cg_v4(src + s * tiles * 65536), b = ld_global_cg_v4(src + s * tiles * 65536 + 4);
      const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += __uint_as_float(v[e]);
    }
    const float rs = __ldcg(p.r.rs + row), coef = __ldcg(p.r.coef + row);
    float w[8];
    unpack8(__ldg(reinterpret_cast<const uint4*>(p.W + static_cast<long long>(__ldcg(p.r.label + row)) * p.h + c)), w);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = fmaf(rs, acc[e], coef * w[e]);
    if (p.column != nullptr) {
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(-flat, __ldcg(p.column + c + e), acc[e]);
    }
    *reinterpret_cast<uint4*>(p.dx + static_cast<long long>(__ldcg(p.r.idx + row)) * p.h + c) = pack8(acc);
  }
}

struct CeTotalArgs {
  const float* loss;
  long long M;
  const int* count;        // NULL: no tokens
  int mean;
  float* total;
};
__global__ void __launch_bounds__(1024) ce_total_kernel(const __grid_constant__ CeTotalArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float slots[32];
  float v = 0.0f;
  for (long long m = threadIdx.x; m < p.M;) {        // 32 losses at a time: short chains
    float part = 0.0f;
#pragma unroll 8
    for (int k = 0; k < 32 && m < p.M; ++k, m += 1024) part += __ldcg(p.loss + m);
    v += part;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  v = slots[threadIdx.x];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  const int n = p.count != nullptr ? __ldcg(p.count) : 0;
  if (threadIdx.x == 0) *p.total = v / static_cast<float>(p.mean && n > 0 ? n : 1);
}

// ---------------------------------------------------------------- host

struct CePlan {
  int64_t rows = 0, pieces = 0, slots = 0, lde = 0, slab_tiles = 0;
  bool exact = false, columns = false;
};
static CePlan ce_plan(int64_t M, int64_t h, int64_t vocab, const lora_ce_t& o, bool want_dx) {
  CePlan P;
  P.slots = ceil_div(vocab, 256) * kCeSlots;
  P.lde = round_up(vocab, 16);
  const int64_t per = want_dx ? 2 * P.lde : P.slots * 8;
  int64_t most = (want_dx ? kCeGradBytes : kCeStatBytes) / per / 256 * 256;
  if (most < 256) most = 256;
  P.pieces = ceil_div(M, most);
  P.rows = P.pieces > 0 ? round_up(ceil_div(M, P.pieces), 256) : 0;
  const int64_t tiles = P.rows / 256 * ceil_div(h, 256);
  const int64_t cut = tiles * kCeMaxSplits < kCeSlabTiles ? tiles * kCeMaxSplits : kCeSlabTiles;
  P.slab_tiles = tiles > cut ? tiles : cut;
  P.exact = want_dx && o.smoothing > 0.0f && o.softcap > 0.0f;
  P.columns = want_dx && o.smoothing > 0.0f && o.softcap == 0.0f;
  return P;
}

struct CeSpace {
  CeRows r;
  CePiece* piece;
  float* loss;
  bf16* packed;
  float2* part;
  float* zsum;
  float* column_part;
  float* column;
  bf16* e;
  float* slab;
};
static size_t ce_carve(void* ws, int64_t M, int64_t h, const lora_ce_t& o, bool want_dx, const CePlan& P, CeSpace& s) {
  Carve c(ws);
  c.take(kWsHeader);
  s.r.count = c.take_n<int>(1);
  s.piece = c.take_n<CePiece>(P.pieces);
  s.r.pos = c.take_n<int>(M);
  s.r.idx = c.take_n<int>(M);
  s.r.label = c.take_n<int>(M);
  s.r.ref2 = c.take_n<float>(M);
  s.r.zlab = c.take_n<float>(M);
  s.r.rs = c.take_n<float>(M);
  s.r.coef = c.take_n<float>(M);
  s.loss = c.take_n<float>(M);
  s.packed = c.take_n<bf16>(M * h);
  s.part = c.take_n<float2>(P.slots * P.rows);
  s.zsum = o.smoothing > 0.0f ? c.take_n<float>(P.slots * P.rows) : nullptr;
  s.column_part = P.columns ? c.take_n<float>(kCeColumnBlocks * h) : nullptr;
  s.column = P.columns ? c.take_n<float>(h) : nullptr;
  s.e = want_dx ? c.take_n<bf16>(P.rows * P.lde) : nullptr;
  s.slab = want_dx ? c.take_n<float>(P.slab_tiles * 65536) : nullptr;
  return c.off;
}

static CeLogit ce_logit_of(const lora_ce_t& o) {
  CeLogit lg;
  lg.k2 = o.logit_scale * kLog2e;
  lg.cap2 = o.softcap * kLog2e;
  lg.kc = o.softcap > 0.0f ? 2.0f * kLog2e * (o.logit_scale / o.softcap) : 0.0f;
  return lg;
}

static lora_status_t check_ce(int64_t M, int64_t h, int64_t vocab, const lora_ce_t* o) {
  if (M < 0 || !o) return LORA_ERR_INVALID_ARG;
  lora_status_t st = LORA_OK;
  check_size(h, st);
  check_size(vocab, st);
  if (st == LORA_ERR_INVALID_ARG) return st;
  if (!std::isfinite(o->logit_scale) || o->logit_scale == 0.0f || !std::isfinite(o->softcap) || o->softcap < 0.0f ||
      !(o->smoothing >= 0.0f && o->smoothing < 1.0f) ||
      (o->reduction != LORA_LOSS_SUM && o->reduction != LORA_LOSS_MEAN))
    return LORA_ERR_INVALID_ARG;
  const CeLogit lg = ce_logit_of(*o);
  if (!std::isfinite(lg.k2) || !std::isfinite(lg.cap2) || !std::isfinite(lg.kc)) return LORA_ERR_INVALID_ARG;
  if (st != LORA_OK || M > kMaxExtent) return LORA_ERR_UNSUPPORTED;
  return h % 8 ? LORA_ERR_ALIGNMENT : LORA_OK;
}

static lora_status_t ce_gemm(int kind, CeGemmParams& p, cudaStream_t st) {
  p.timeout_ns = wait_timeout_ns();
  p.inject_stall = take_expiry();
  const int slot = trace_begin(LORA_KIND_LOSS, st);
  const cudaError_t e = launch_ce_gemm(kind, p, num_sms() / 2 * 2, st);
  trace_end(slot, st);
  if (e != cudaSuccess) return LORA_ERR_CUDA;
  count_launch();
  return LORA_OK;
}

}  // namespace lgb

using namespace lgb;

extern "C" size_t lora_linear_ce_workspace_bytes(int64_t M, int64_t h, int64_t vocab, const lora_ce_t* opts, int want_dx) {
  if (check_ce(M, h, vocab, opts) != LORA_OK) return 0;
  CeSpace s;
  return ce_carve(nullptr, M, h, *opts, want_dx != 0, ce_plan(M, h, vocab, *opts, want_dx != 0), s);
}

extern "C" lora_status_t lora_linear_ce(int64_t M, int64_t h, int64_t vocab, const void* x, const void* W,
                                        const int64_t* labels, const lora_ce_t* opts, float* loss, float* lse, float* total,
                                        void* dx, void* ws, size_t ws_bytes, cudaStream_t stream) {
  NvtxRange nvtx_range("lora_linear_ce");
  if (!W || !total || (M > 0 && (!x || !labels))) return LORA_ERR_INVALID_ARG;
  LGB_TRY(check_ce(M, h, vocab, opts));
  if (dx != nullptr && dx == x) return LORA_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(W, 16) || !aligned(dx, 16) || !aligned(labels, 8) || !aligned(loss, 4) || !aligned(lse, 4) ||
      !aligned(total, 4))
    return LORA_ERR_ALIGNMENT;
  const lora_ce_t& o = *opts;
  const bool want = dx != nullptr, mean = o.reduction == LORA_LOSS_MEAN;
  const CePlan P = ce_plan(M, h, vocab, o, want);
  CeSpace s;
  LGB_TRY(check_ws(ws, ws_bytes, ce_carve(ws, M, h, o, want, P, s)));
  CeTotalArgs t;
  t.loss = loss != nullptr ? loss : s.loss;
  t.M = M;
  t.count = M > 0 ? s.r.count : nullptr;
  t.mean = mean;
  t.total = total;
  if (M > 0) {
    unsigned* status = static_cast<unsigned*>(ws);
    const int tiles_n = static_cast<int>(ceil_div(vocab, 256)), tiles_h = static_cast<int>(ceil_div(h, 256));
    const int kb_h = static_cast<int>(ceil_div(h, kBK)), kb_v = static_cast<int>(ceil_div(vocab, kBK));
    const CeLogit lg = ce_logit_of(o);

    CePackArgs pack;
    pack.labels = reinterpret_cast<const long long*>(labels);
    pack.M = M;
    pack.ignore = o.ignore_index;
    pack.vocab = vocab;
    pack.r = s.r;
    pack.piece = s.piece;
    pack.pieces = static_cast<int>(P.pieces);
    pack.piece_rows = static_cast<int>(P.rows);
    pack.tiles_n = tiles_h;
    pack.kb = kb_v;
    pack.pairs = num_sms() / 2;
    pack.status = status;
    LGB_TRY(launch_counted(ce_pack_kernel, dim3(1), dim3(1024), 0, LORA_KIND_LOSS, stream, pack));

    CeGatherArgs gather;
    gather.x = static_cast<const bf16*>(x);
    gather.W = static_cast<const bf16*>(W);
    gather.M = M;
    gather.h = static_cast<int>(h);
    gather.r = s.r;
    gather.packed = s.packed;
    gather.lg = lg;
    gather.want_ref = want && !P.exact;
    gather.loss = const_cast<float*>(t.loss);
    gather.lse = lse;
    gather.dx = static_cast<bf16*>(dx);
    const int64_t rows8 = ceil_div(M, 8);
    LGB_TRY(launch_counted(ce_gather_kernel, dim3(static_cast<unsigned>(rows8 < (1 << 20) ? rows8 : (1 << 20))), dim3(256), 0,
                           LORA_KIND_LOSS, stream, gather));
    if (P.columns) {
      CeColumnArgs ca;
      ca.W = gather.W;
      ca.vocab = vocab;
      ca.h = gather.h;
      ca.part = s.column_part;
      ca.sum = s.column;
      LGB_TRY(launch_counted(ce_column_kernel, dim3(static_cast<unsigned>(ceil_div(h, 1024)), kCeColumnBlocks), dim3(128), 0,
                             LORA_KIND_LOSS, stream, ca));
      LGB_TRY(launch_counted(ce_column_join_kernel, dim3(static_cast<unsigned>(ceil_div(h, 32))), dim3(256), 0, LORA_KIND_LOSS,
                             stream, ca));
    }
    for (int64_t k = 0; k < P.pieces; ++k) {
      const int64_t row0 = k * P.rows;
      const int64_t rows = M - row0 < P.rows ? M - row0 : P.rows;
      if (rows <= 0) break;
      CeRows r = s.r;
      r.idx += row0;
      r.label += row0;
      r.ref2 += row0;
      r.zlab += row0;
      r.rs += row0;
      r.coef += row0;
      CeGemmParams g;
      std::memset(static_cast<void*>(&g), 0, sizeof(g));
      if (!encode_map(&g.a, s.packed + row0 * h, h, rows, h, kBK, kBM) || !encode_map(&g.b, W, h, vocab, h, kBK, 128))
        return LORA_ERR_CUDA;
      g.piece = s.piece + k;
      g.kb_total = kb_h;
      g.kvalid = static_cast<int>(h);
      g.tiles_n = tiles_n;
      g.band = raster_band();
      g.status = status;
      g.vocab = static_cast<int>(vocab);
      g.lg = lg;
      g.label = r.label;
      g.ref2 = r.ref2;
      g.part = s.part;
      g.zsum = s.zsum;
      g.zlab = r.zlab;
      g.ldp = P.rows;
      g.e = s.e;
      g.lde = P.lde;
      g.minus = P.exact ? o.smoothing / static_cast<float>(vocab) : 0.0f;
      CeJoinArgs j;
      j.piece = s.piece + k;
      j.r = r;
      j.part = s.part;
      j.zsum = s.zsum;
      j.ldp = P.rows;
      j.slots = static_cast<int>(P.slots);
      j.vocab = static_cast<int>(vocab);
      j.cap2 = lg.cap2;
      j.scale = o.logit_scale;
      j.smoothing = o.smoothing;
      j.mean = mean;
      j.loss = const_cast<float*>(t.loss);
      j.lse = lse;
      auto join = [&](int mode) {
        j.mode = mode;
        return launch_counted(ce_join_kernel, dim3(static_cast<unsigned>(ceil_div(rows, 32))), dim3(32 * kJoinWarps), 0,
                              LORA_KIND_LOSS, stream, j);
      };
      if (!want || P.exact) {
        LGB_TRY(ce_gemm(CE_STATS, g, stream));
        LGB_TRY(join(want ? CE_JOIN_EXACT : CE_JOIN_LOSS));
      }
      if (!want) continue;
      if (P.exact) g.zsum = nullptr;
      LGB_TRY(ce_gemm(CE_GRAD, g, stream));
      if (!P.exact) {
        LGB_TRY(join(CE_JOIN_GRAD));
        g.when_redo = 1;
        LGB_TRY(ce_gemm(CE_GRAD, g, stream));
        LGB_TRY(join(CE_JOIN_REDO));
      }
      CeGemmParams d;
      std::memset(static_cast<void*>(&d), 0, sizeof(d));
      if (!encode_map(&d.a, s.e, vocab, rows, P.lde, kBK, kBM) || !encode_map(&d.b, W, h, vocab, h, 64, 64))
        return LORA_ERR_CUDA;
      d.piece = s.piece + k;
      d.kb_total = kb_v;
      d.kvalid = static_cast<int>(vocab);
      d.tiles_n = tiles_h;
      d.band = raster_band();
      d.status = status;
      d.slab = s.slab;
      LGB_TRY(ce_gemm(CE_PART, d, stream));
      CeDxArgs a;
      a.piece = s.piece + k;
      a.r = r;
      a.slab = s.slab;
      a.tiles_n = tiles_h;
      a.h = static_cast<int>(h);
      a.W = gather.W;
      a.column = s.column;
      a.scale = o.logit_scale;
      a.share = o.smoothing / static_cast<float>(vocab);
      a.mean = mean;
      a.dx = gather.dx;
      const int64_t blocks = ceil_div(rows * (h / 8), 256);
      LGB_TRY(launch_counted(ce_dx_kernel, dim3(static_cast<unsigned>(blocks < (1 << 20) ? blocks : (1 << 20))), dim3(256), 0,
                             LORA_KIND_LOSS, stream, a));
    }
  }
  return launch_counted(ce_total_kernel, dim3(1), dim3(1024), 0, LORA_KIND_LOSS, stream, t);
}
