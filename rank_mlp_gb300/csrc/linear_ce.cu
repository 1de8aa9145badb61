// Cross entropy of a frozen head with its gradient (lora_linear_ce), and the scaling of that gradient
// (lora_scale_rows); include/lora_gb300.h is the contract, gemm_ce.cuh has the GEMMs and the mathematics they share with this file.
//
// A call packs the labelled rows, then takes them piece by piece:
//   loss alone     CE_STATS, join of the row's partial results
//   with dx        reference z_y + 40 for each row (a dot product), CE_GRAD, join, CE_PART over the
//                  exponentials, join of the k-ranges with the label's row of W
//   capped and smoothed at once: CE_STATS, join, CE_GRAD with lse as its reference, CE_PART
//                  (the smoothing's part of the gradient then depends on each logit's slope); the
//                  weights' sums, which come after the join, are joined by CE_PART's epilogue warps
// A row's largest logit is at least its label's.  So the reference, 40 above the label's logit,
// leaves the largest exponential between e^-40 and, where the largest logit stands less than 100
// above the label's, e^60: it, the sums and the product stay inside the range of f32 and bf16
// (a weight below 2^-68 of the label's counts as zero).  A row beyond that is seen by its sum,
// and its piece is taken again the last way: one such token among 4095 x 896 x 131,072, a single piece, makes
// 1.3 ms 2.6, among 4096 x 4096 x 131,072 5.6 ms 11.
#include "gemm_ce.cuh"
#include "serve.cuh"

namespace lgb {

constexpr float kCeAhead = 40.0f * kLog2e;         // the reference above the label's logit
constexpr float kCeMost = 1.5474250491067253e26f;  // 2^87: a row's sum of exponentials past it is taken again
constexpr int64_t kCeGradBytes = int64_t(1) << 30; // exponentials of a piece, and its product's sums
constexpr int64_t kCeStatBytes = int64_t(1) << 28; // partial results of a piece (the loss alone)
constexpr int64_t kCeMaxVocab = int64_t(1) << 24;   // (256 rows' exponentials stay in a TMA map's reach)
constexpr int kCeColumnBlocks = 304;               // row ranges of W for its column sums

// The rows of a call as the kernels see them; arrays over packed rows but for pos.
struct CeRows {
  int* count;              // labelled rows
  unsigned* joined;        // [2] blocks of the last piece's joins that are done
  int* pos;                // [M] place of a token among them, -1: none
  int* idx;                // token of a packed row
  int* label;
  float* ref2;             // the reference, in units of ln 2 as all logits here
  float* zlab;             // the label's logit
  float* slope;            // with a cap: its tanh's slope there
  float* rs;               // factors of the row's gradient: of sum e W, and of W_label
  float* coef;
};

// What the pieces' descriptions are made of.
struct CePieces {
  CePiece* piece;
  int pieces, piece_rows;
  int tiles_n, kb, pairs;  // of CE_PART
};
__device__ __forceinline__ void write_pieces(const CePieces& p, const CeRows& r, int n) {
  if (threadIdx.x == 0) {
    *r.count = n;
    r.joined[0] = r.joined[1] = 0;
  }
  for (int k = threadIdx.x; k < p.pieces; k += blockDim.x) {
    const long long left = n - static_cast<long long>(k) * p.piece_rows;
    p.piece[k] = ce_piece(left <= 0 ? 0 : left < p.piece_rows ? static_cast<int>(left) : p.piece_rows, p.tiles_n, p.kb, p.pairs);
  }
}

struct CeLabels {
  const long long* y;
  long long M, ignore, vocab;
};

struct CePackArgs {
  CeLabels labels;
  CeRows r;
  CePieces plan;
  unsigned* status;
};

// One block: the labelled tokens' places, in order, and what each piece holds.
__global__ void __launch_bounds__(1024) ce_pack_kernel(const __grid_constant__ CePackArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ int warps[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int n = 0;
  for (long long base = 0; base < p.labels.M; base += 4096) {
    const long long m = base + 4 * threadIdx.x;
    long long y[4];
    bool seen[4];
    int mine = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[j] = m + j < p.labels.M ? __ldg(p.labels.y + m + j) : p.labels.ignore;
      seen[j] = y[j] != p.labels.ignore;
      if (seen[j] && (y[j] < 0 || y[j] >= p.labels.vocab)) {
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
      if (m + j >= p.labels.M) break;
      p.r.pos[m + j] = seen[j] ? at : -1;
      if (!seen[j]) continue;
      p.r.idx[at] = static_cast<int>(m + j);
      p.r.label[at] = static_cast<int>(y[j]);
      ++at;
    }
    n += total;
  }
  write_pieces(p.plan, p.r, n);
}

struct CeGatherArgs {
  const bf16* x;
  const bf16* W;
  int h;
  CeLabels labels;
  CeRows r;
  CePieces plan;
  bf16* packed;            // [count][h]
  CeLogit lg;
  int want_ref;
  float* loss;
  float* lse;              // NULL: not wanted
  bf16* dx;                // NULL: the loss alone
  unsigned* status;
};

// A warp a token: packs its row and takes the reference from its label's logit, or clears what
// an unlabelled token has.  ALONE (fewer tokens than kCeAloneRows): no ce_pack_kernel has run; a block
// counts the labelled tokens before its own eight by itself.  (A head of 4096 x 896: 64 tokens 36.0 us
// instead of 38.3, 8192 140 instead of 147, 16384 248 instead of 257, 32768 the same.)
constexpr int kCeAloneRows = 16384;
template <bool ALONE>
__global__ void __launch_bounds__(256) ce_gather_kernel(const __grid_constant__ CeGatherArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int at_alone = -1, label_alone = 0;
  if constexpr (ALONE) {
    __shared__ int upto[8], all[8];
    const int M = static_cast<int>(p.labels.M), first = blockIdx.x * 8;
    int n = 0, total = 0;                            // labelled tokens before the block's, and in all
    for (int m = threadIdx.x; m < (blockIdx.x == 0 ? M : first); m += 256) {
      const long long y = __ldg(p.labels.y + m);
      const bool seen = y != p.labels.ignore && y >= 0 && y < p.labels.vocab;
      n += seen && m < first;
      total += seen;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      n += __shfl_xor_sync(0xffffffffu, n, d);
      total += __shfl_xor_sync(0xffffffffu, total, d);
    }
    if (lane == 0) upto[warp] = n, all[warp] = total;
    __syncthreads();
    n = total = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) n += upto[k], total += all[k];
    if (blockIdx.x == 0) write_pieces(p.plan, p.r, total);
    // the block's own eight: lane k of each warp looks at token k
    const int m = first + (lane & 7);
    const long long y = m < M ? __ldg(p.labels.y + m) : p.labels.ignore;
    bool seen = y != p.labels.ignore;
    if (seen && (y < 0 || y >= p.labels.vocab)) {
      if (threadIdx.x < 8) atomicOr(p.status, kStatusInput);
      seen = false;
    }
    const unsigned mask = __ballot_sync(0xffffffffu, seen) & 0xFFu;
    label_alone = static_cast<int>(__shfl_sync(0xffffffffu, y, warp));
    at_alone = (mask >> warp) & 1u ? n + __popc(mask & ((1u << warp) - 1u)) : -1;
    if (at_alone >= 0 && lane == 0) {
      p.r.idx[at_alone] = first + warp;
      p.r.label[at_alone] = label_alone;
    }
  }
  for (long long m = blockIdx.x * 8ll + warp; m < p.labels.M; m += 8ll * gridDim.x) {
    const int at = ALONE ? at_alone : __ldcg(p.r.pos + m);
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
    const bf16* w = p.W + static_cast<long long>(ALONE ? label_alone : __ldcg(p.r.label + at)) * p.h;
    bf16* out = p.packed + static_cast<long long>(at) * p.h;
    float dot = 0.0f;
    for (int c0 = 8 * lane; c0 < p.h; c0 += 1024) {  // four pieces of both rows on their way at a time
      uint4 v[4], u[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = c0 + 256 * k < p.h ? c0 + 256 * k : c0;
        v[k] = __ldg(reinterpret_cast<const uint4*>(x + c));
        if (p.want_ref) u[k] = __ldg(reinterpret_cast<const uint4*>(w + c));
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = c0 + 256 * k;
        if (c >= p.h) break;
        *reinterpret_cast<uint4*>(out + c) = v[k];
        if (p.want_ref) {
          float a[8], b[8];
          unpack8(v[k], a);
          unpack8(u[k], b);
#pragma unroll
          for (int e = 0; e < 8; ++e) dot = fmaf(a[e], b[e], dot);
        }
      }
    }
    if (!p.want_ref) continue;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
    if (lane == 0) {
      float slope;
      p.r.ref2[at] = (p.lg.cap2 > 0.0f ? ce_logit<CE_CAP>(dot, p.lg, slope) : ce_logit<CE_NO_CAP>(dot, p.lg, slope)) + kCeAhead;
    }
  }
}

enum CeJoin : int { CE_JOIN_LOSS = 0, CE_JOIN_EXACT = 1, CE_JOIN_GRAD = 2 };
struct CeJoinArgs {
  CePiece* piece;
  int mode;
  int when_redo;           // 1: only if the piece's `redo` is set
  CeRows r;                // at the piece's first row (count, joined: the call's)
  const float2* part;      // CE_JOIN_LOSS, CE_JOIN_EXACT
  const float* psum;       // CE_JOIN_GRAD
  const float* wsum;
  const float* tsum;       // (psum itself without a cap)
  const float* zsum;
  long long ldp;
  int slots;
  int vocab;
  float cap2;              // 0: no cap
  float scale, smoothing, minus;
  int mean;
  float* loss;             // by token
  float* lse;
  float* total;            // of the last piece: the call's total; else NULL
  long long M;
};

constexpr int kJoinWarps = 32;

// Rows [32 blockIdx.x, + 32) of a piece: a lane a row, their partial results are shared out over the
// block's warps; then a warp a row, the warps' shares are joined, in a fixed order, and the row's
// loss and factors follow.
template <int MODE>
__device__ __forceinline__ void ce_join_rows(const CeJoinArgs& p, int live) {
  __shared__ float tops[kJoinWarps][33], sums[kJoinWarps][33], zs[kJoinWarps][33];
  __shared__ float weights[MODE == CE_JOIN_GRAD ? 2 : 1][MODE == CE_JOIN_GRAD ? kJoinWarps : 1][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr bool kRelative = MODE != CE_JOIN_GRAD;   // sums relative to their own maxima
  float top = -INFINITY, sum = 0.0f, z = 0.0f, t = 0.0f, w = 0.0f;
  const bool own = MODE == CE_JOIN_GRAD && p.tsum != p.psum;       // sums of the weights that are not those of the loss
  auto add = [&](float t, float s) {
    if (t == -INFINITY && s == 0.0f) return;         // no column but the label's
    const float most = fmaxf(top, t);
    sum = sum * exp2f(top - most) + s * exp2f(t - most);
    top = most;
  };
  if (static_cast<int>(blockIdx.x) * 32 + lane < live) {
    const int row = blockIdx.x * 32 + lane;
#pragma unroll 8
    for (int k = warp; k < p.slots; k += kJoinWarps) {
      if constexpr (kRelative) {
        const float2 o = __ldcg(p.part + k * p.ldp + row);
        add(o.x, o.y);
      } else {
        sum += __ldcg(p.psum + k * p.ldp + row);
        w += __ldcg(p.wsum + k * p.ldp + row);
      }
      if (p.zsum != nullptr) z += __ldcg(p.zsum + k * p.ldp + row);
    }
    if (own) {
#pragma unroll 8
      for (int k = warp; k < p.slots; k += kJoinWarps) t += __ldcg(p.tsum + k * p.ldp + row);
    }
  }
  tops[warp][lane] = top;
  sums[warp][lane] = sum;
  zs[warp][lane] = z;
  if constexpr (MODE == CE_JOIN_GRAD) weights[0][warp][lane] = w, weights[1][warp][lane] = t;
  const int row = blockIdx.x * 32 + warp;
  float zl = 0.0f, ref2 = 0.0f;                      // (on their way across the barrier)
  int token = 0, count = 1;
  if (row < live) {
    zl = __ldcg(p.r.zlab + row);
    if (!kRelative) ref2 = __ldcg(p.r.ref2 + row);
    token = __ldg(p.r.idx + row);
    count = __ldcg(p.r.count);
  }
  __syncthreads();
  if (row >= live) return;
  top = tops[lane][warp];
  sum = sums[lane][warp];
  z = zs[lane][warp];
  if constexpr (MODE == CE_JOIN_GRAD) w = weights[0][lane][warp], t = weights[1][lane][warp];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    if constexpr (kRelative) {
      // (both lanes of a pair take the same order: the same bits)
      const float at = __shfl_xor_sync(0xffffffffu, top, d), o = __shfl_xor_sync(0xffffffffu, sum, d), most = fmaxf(top, at);
      const float mine = sum == 0.0f && top == -INFINITY ? 0.0f : sum * exp2f(top - most);
      const float theirs = o == 0.0f && at == -INFINITY ? 0.0f : o * exp2f(at - most);
      sum = mine + theirs;
      top = most;
    } else {
      sum += __shfl_xor_sync(0xffffffffu, sum, d);
      w += __shfl_xor_sync(0xffffffffu, w, d);
      t += __shfl_xor_sync(0xffffffffu, t, d);
    }
    z += __shfl_xor_sync(0xffffffffu, z, d);
  }
  if (lane != 0) return;
  if (kRelative) ref2 = top;
  if (MODE == CE_JOIN_GRAD && sum > kCeMost) p.piece->redo = 1;     // (every writer writes the same)
  // d: the others' log-sum over the label's logit, in units of ln 2
  const float others = ref2 + log2f(sum), d = others - zl;
  const float tail = log1pf(exp2f(-fabsf(d)));
  const float ce = d > 0.0f ? fmaf(d, kLn2, tail) : tail;
  const float eps = p.smoothing;
  p.loss[token] = p.zsum != nullptr ? ce + eps * kLn2 * (zl - z / p.vocab) : ce;
  if (p.lse != nullptr) p.lse[token] = fmaf(zl, kLn2, ce);
  if (MODE == CE_JOIN_LOSS) return;
  const float g = p.scale / (p.mean ? static_cast<float>(count) : 1.0f);
  const float slope = p.cap2 > 0.0f ? __ldcg(p.r.slope + row) : 1.0f;
  const float away = expm1f(-ce);                    // p_label - 1
  if (MODE == CE_JOIN_EXACT) {
    p.r.ref2[row] = fmaf(ce, kLog2e, zl);
    p.r.rs[row] = g;
    p.r.coef[row] = g * slope * (away + eps - p.minus);
  } else {
    float rs = g / (sum + exp2f(zl - ref2)), coef = g * slope * (away + eps);
    ce_balance(own ? t : sum, w, rs, coef);
    p.r.rs[row] = rs;
    p.r.coef[row] = coef;
  }
}

// The block that is the last of its launch to get here sums the losses of all tokens, in a fixed order.
__device__ __forceinline__ void ce_total(const CeJoinArgs& p) {
  __shared__ float slots[kJoinWarps];
  __shared__ int last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(p.r.joined + p.when_redo, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  if (p.mode == CE_JOIN_GRAD && __ldcg(&p.piece->redo) != 0) return;      // left to the second try
  float v = 0.0f;
  for (long long m = threadIdx.x; m < p.M;) {        // 32 losses at a time: short chains
    float part = 0.0f;
#pragma unroll 8
    for (int k = 0; k < 32 && m < p.M; ++k, m += 32 * kJoinWarps) part += __ldcg(p.loss + m);
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
  const int n = __ldcg(p.r.count);
  if (threadIdx.x == 0) *p.total = v / static_cast<float>(p.mean && n > 0 ? n : 1);
}

__global__ void __launch_bounds__(32 * kJoinWarps) ce_join_kernel(const __grid_constant__ CeJoinArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  if (p.when_redo && __ldcg(&p.piece->redo) == 0) return;
  const int live = __ldcg(&p.piece->live);
  if (static_cast<int>(blockIdx.x) * 32 < live) {
    if (p.mode == CE_JOIN_GRAD) {
      ce_join_rows<CE_JOIN_GRAD>(p, live);
    } else if (p.mode == CE_JOIN_EXACT) {
      ce_join_rows<CE_JOIN_EXACT>(p, live);
    } else {
      ce_join_rows<CE_JOIN_LOSS>(p, live);
    }
  }
  if (p.total != nullptr) ce_total(p);
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
  int tiles_n, band, h;
  const bf16* W;
  const float* column;     // column sums of W, or NULL
  float scale, share;      // logit scale, smoothing / vocab
  int mean;
  bf16* dx;
};
// dx rows of a piece: the k-ranges' sums times the row's factor, the label's row of W, and the
// smoothing's part.  An item is eight features of a row; a thread has kDxItems on their way.
constexpr int kDxItems = 2;
constexpr int kDxAhead = 6;              // and a cut tile's further k-ranges of an item likewise
constexpr int kDxBlocks = 3;             // resident blocks an SM
__global__ void __launch_bounds__(256, kDxBlocks) ce_dx_kernel(const __grid_constant__ CeDxArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  const int live = __ldcg(&p.piece->live), whole = __ldcg(&p.piece->whole), splits = __ldcg(&p.piece->splits);
  const unsigned per = p.h / 8;
  const int tiles_m = (live + 255) / 256;
  const long long cut = static_cast<long long>(tiles_m * p.tiles_n - whole) * 65536;
  const unsigned long long total = static_cast<unsigned long long>(live) * per, step = 256ull * gridDim.x;
  const float flat = p.column == nullptr ? 0.0f : p.scale * p.share / (p.mean ? static_cast<float>(__ldcg(p.r.count)) : 1.0f);
  for (unsigned long long i0 = blockIdx.x * 256ull + threadIdx.x; i0 < total; i0 += kDxItems * step) {
    int row[kDxItems], c[kDxItems], label[kDxItems], token[kDxItems], parts[kDxItems];
    float rs[kDxItems], coef[kDxItems];
    const float* src[kDxItems];
    uint4 v[kDxItems][2], w[kDxItems];
#pragma unroll
    for (int k = 0; k < kDxItems; ++k) {
      const unsigned long long i = i0 + k * step < total ? i0 + k * step : i0;
      const unsigned r = total <= 0xffffffffull ? static_cast<unsigned>(i) / per : static_cast<unsigned>(i / per);
      row[k] = static_cast<int>(r);
      c[k] = 8 * static_cast<int>(i - static_cast<unsigned long long>(r) * per);
      label[k] = __ldcg(p.r.label + row[k]);
      rs[k] = __ldcg(p.r.rs + row[k]);
      coef[k] = __ldcg(p.r.coef + row[k]);
      token[k] = __ldcg(p.r.idx + row[k]);
      const int place = ce_tile_place(row[k] >> 8, c[k] >> 8, tiles_m, p.tiles_n, p.band);
      parts[k] = place < whole ? 1 : splits;
      src[k] = p.slab + static_cast<long long>(place) * 65536 + (row[k] & 255) * 256 + (c[k] & 255);
      v[k][0] = __ldcg(reinterpret_cast<const uint4*>(src[k]));
      v[k][1] = __ldcg(reinterpret_cast<const uint4*>(src[k]) + 1);
    }
#pragma unroll
    for (int k = 0; k < kDxItems; ++k)
      w[k] = __ldg(reinterpret_cast<const uint4*>(p.W + static_cast<long long>(label[k]) * p.h + c[k]));
#pragma unroll
    for (int k = 0; k < kDxItems; ++k) {
      if (i0 + k * step >= total) break;
      float acc[8] = {__uint_as_float(v[k][0].x), __uint_as_float(v[k][0].y), __uint_as_float(v[k][0].z), __uint_as_float(v[k][0].w),
                      __uint_as_float(v[k][1].x), __uint_as_float(v[k][1].y), __uint_as_float(v[k][1].z), __uint_as_float(v[k][1].w)};
      for (int s = 1; s < parts[k]; s += kDxAhead) {
        float4 u[kDxAhead][2];                       // past the last: it again, left out
#pragma unroll
        for (int j = 0; j < kDxAhead; ++j) {
          const float4* from = reinterpret_cast<const float4*>(src[k] + min(s + j, parts[k] - 1) * cut);
          u[j][0] = __ldcg(from);
          u[j][1] = __ldcg(from + 1);
        }
#pragma unroll
        for (int j = 0; j < kDxAhead; ++j) {
          if (s + j >= parts[k]) break;
          acc[0] += u[j][0].x, acc[1] += u[j][0].y, acc[2] += u[j][0].z, acc[3] += u[j][0].w;
          acc[4] += u[j][1].x, acc[5] += u[j][1].y, acc[6] += u[j][1].z, acc[7] += u[j][1].w;
        }
      }
      float x[8];
      unpack8(w[k], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(rs[k], acc[e], coef[k] * x[e]);
      if (p.column != nullptr) {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = fmaf(-flat, __ldcg(p.column + c[k] + e), acc[e]);
      }
      *reinterpret_cast<uint4*>(p.dx + static_cast<long long>(token[k]) * p.h + c[k]) = pack8(acc);
    }
  }
}

struct ScaleArgs {
  const bf16* x;
  const float* g;
  int g_stride;
  bf16* y;
  long long M;
  int h;
};
// Rows times their factors, a 16-byte piece a thread and step: bound by memory.
__global__ void __launch_bounds__(256) scale_rows_kernel(const __grid_constant__ ScaleArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  const unsigned per = p.h / 8;
  const unsigned long long total = static_cast<unsigned long long>(p.M) * per;
  for (unsigned long long i = blockIdx.x * 256ull + threadIdx.x; i < total; i += 256ull * gridDim.x) {
    const long long m = p.g_stride == 0 ? 0 : total <= 0xffffffffull ? static_cast<unsigned>(i) / per : static_cast<long long>(i / per);
    const float g = __ldg(p.g + m);
    float v[8];
    unpack8(reinterpret_cast<const uint4*>(p.x)[i], v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= g;
    reinterpret_cast<uint4*>(p.y)[i] = pack8(v);
  }
}

// ---------------------------------------------------------------- host

struct CePlan {
  int64_t rows = 0, pieces = 0, slots = 0, blocks = 0, slab_tiles = 0;
  bool exact = false, columns = false;
};
static CePlan ce_plan(int64_t M, int64_t h, int64_t vocab, const lora_ce_t& o, bool want_dx) {
  CePlan P;
  P.slots = ceil_div(vocab, 256) * kCeSlots;
  P.blocks = ceil_div(vocab, kBK);
  const int64_t per = want_dx ? 2 * kBK * P.blocks : P.slots * 8;
  int64_t most = (want_dx ? kCeGradBytes : kCeStatBytes) / per / 256 * 256;
  const int64_t sums = kCeGradBytes / (4 * round_up(h, 256)) / 256 * 256;
  if (want_dx && most > sums) most = sums;
  if (most < 256) most = 256;
  P.pieces = ceil_div(M, most);
  P.rows = P.pieces > 0 ? round_up(ceil_div(M, P.pieces), 256) : 0;
  const int64_t tiles = P.rows / 256 * ceil_div(h, 256);
  P.slab_tiles = tiles + (tiles * kCeMaxSplits < kCeTailUnits ? tiles * kCeMaxSplits : kCeTailUnits);
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
  float* psum;
  float* wsum;
  float* tsum;
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
  s.r.joined = c.take_n<unsigned>(2);
  s.piece = c.take_n<CePiece>(P.pieces);
  s.r.pos = c.take_n<int>(M);
  s.r.idx = c.take_n<int>(M);
  s.r.label = c.take_n<int>(M);
  s.r.ref2 = c.take_n<float>(M);
  s.r.zlab = c.take_n<float>(M);
  s.r.slope = o.softcap > 0.0f ? c.take_n<float>(M) : nullptr;
  s.r.rs = c.take_n<float>(M);
  s.r.coef = c.take_n<float>(M);
  s.loss = c.take_n<float>(M);
  s.packed = c.take_n<bf16>(M * h);
  s.part = c.take_n<float2>(P.slots * P.rows);
  s.psum = reinterpret_cast<float*>(s.part);       // (never both at a time)
  s.wsum = s.psum + P.slots * P.rows;
  s.tsum = want_dx && o.softcap > 0.0f ? c.take_n<float>(P.slots * P.rows) : s.psum;
  s.zsum = o.smoothing > 0.0f ? c.take_n<float>(P.slots * P.rows) : nullptr;
  s.column_part = P.columns ? c.take_n<float>(kCeColumnBlocks * h) : nullptr;
  s.column = P.columns ? c.take_n<float>(h) : nullptr;
  s.e = want_dx ? c.take_n<bf16>(P.rows * kBK * P.blocks) : nullptr;
  s.slab = want_dx ? c.take_n<float>(P.slab_tiles * 65536) : nullptr;
  return c.off;
}

static CeLogit ce_logit_of(const lora_ce_t& o) {
  CeLogit lg;
  lg.k2 = o.logit_scale * kLog2e;
  lg.cap2 = o.softcap * kLog2e;
  lg.kc = o.softcap > 0.0f ? o.logit_scale / o.softcap : 0.0f;
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
  if (st != LORA_OK || M > kMaxExtent || vocab > kCeMaxVocab) return LORA_ERR_UNSUPPORTED;
  return h % 8 ? LORA_ERR_ALIGNMENT : LORA_OK;
}

static bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
  return p < q + static_cast<uintptr_t>(b_bytes) && q < p + static_cast<uintptr_t>(a_bytes);
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
  if (!aligned(x, 16) || !aligned(W, 16) || !aligned(dx, 16) || !aligned(labels, 8) || !aligned(loss, 4) || !aligned(lse, 4) ||
      !aligned(total, 4))
    return LORA_ERR_ALIGNMENT;
  // (other rows of x are packed, and W is read, while rows of dx are written)
  if (dx != nullptr && M > 0 && (overlap(dx, M * h * 2, x, M * h * 2) || overlap(dx, M * h * 2, W, vocab * h * 2))) return LORA_ERR_INVALID_ARG;
  const lora_ce_t& o = *opts;
  const bool want = dx != nullptr, mean = o.reduction == LORA_LOSS_MEAN;
  const CePlan P = ce_plan(M, h, vocab, o, want);
  CeSpace s;
  LGB_TRY(check_ws(ws, ws_bytes, ce_carve(ws, M, h, o, want, P, s)));
  if (M == 0) return cudaMemsetAsync(total, 0, sizeof(float), stream) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
  if (loss == nullptr) loss = s.loss;
  unsigned* status = static_cast<unsigned*>(ws);
  const int tiles_n = static_cast<int>(ceil_div(vocab, 256)), tiles_h = static_cast<int>(ceil_div(h, 256));
  const int kb_h = static_cast<int>(ceil_div(h, kBK)), kb_v = static_cast<int>(ceil_div(vocab, kBK));
  const CeLogit lg = ce_logit_of(o);
  const float share = o.smoothing / static_cast<float>(vocab);

  CeGatherArgs gather;
  gather.x = static_cast<const bf16*>(x);
  gather.W = static_cast<const bf16*>(W);
  gather.h = static_cast<int>(h);
  gather.labels = CeLabels{reinterpret_cast<const long long*>(labels), M, o.ignore_index, vocab};
  gather.r = s.r;
  gather.plan = CePieces{s.piece, static_cast<int>(P.pieces), static_cast<int>(P.rows), tiles_h, kb_v, num_sms() / 2};
  gather.packed = s.packed;
  gather.lg = lg;
  gather.want_ref = want && !P.exact;
  gather.loss = loss;
  gather.lse = lse;
  gather.dx = static_cast<bf16*>(dx);
  gather.status = status;
  const bool alone = M <= kCeAloneRows;
  if (!alone) {
    CePackArgs pack;
    pack.labels = gather.labels;
    pack.r = s.r;
    pack.plan = gather.plan;
    pack.status = status;
    LGB_TRY(launch_counted(ce_pack_kernel, dim3(1), dim3(1024), 0, LORA_KIND_LOSS, stream, pack));
  }
  const int64_t rows8 = ceil_div(M, 8);
  LGB_TRY(launch_counted(alone ? ce_gather_kernel<true> : ce_gather_kernel<false>,
                         dim3(static_cast<unsigned>(rows8 < (1 << 20) ? rows8 : (1 << 20))), dim3(256), 0, LORA_KIND_LOSS,
                         stream, gather));
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
    if (r.slope != nullptr) r.slope += row0;
    r.rs += row0;
    r.coef += row0;
    CeGemmParams g;
    std::memset(static_cast<void*>(&g), 0, sizeof(g));
    if (!encode_map(&g.a, s.packed + row0 * h, h, rows, h, kBK, kBM) || !encode_map(&g.b, W, h, vocab, h, kBK, 128))
      return LORA_ERR_CUDA;
    g.piece = s.piece + k;
    g.kb_total = kb_h;
    g.kb_range = static_cast<int>(ceil_div(kb_h, ceil_div(kb_h, kCeRangeKb)));
    g.kvalid = static_cast<int>(h);
    g.tiles_n = tiles_n;
    g.band = raster_band();
    g.status = status;
    g.vocab = static_cast<int>(vocab);
    g.lg = lg;
    g.label = r.label;
    g.ref2 = r.ref2;
    g.part = s.part;
    g.psum = s.psum;
    g.wsum = s.wsum;
    g.tsum = s.tsum;
    g.zlab = r.zlab;
    g.slope = r.slope;
    g.ldp = P.rows;
    g.e = s.e;
    g.blocks = static_cast<int>(P.blocks);
    g.minus = P.exact ? share : 0.0f;
    CeJoinArgs j;
    j.piece = s.piece + k;
    j.r = r;
    j.part = s.part;
    j.psum = s.psum;
    j.wsum = s.wsum;
    j.tsum = s.tsum;
    j.zsum = s.zsum;
    j.ldp = P.rows;
    j.slots = static_cast<int>(P.slots);
    j.vocab = static_cast<int>(vocab);
    j.cap2 = lg.cap2;
    j.scale = o.logit_scale;
    j.smoothing = o.smoothing;
    j.minus = g.minus;
    j.mean = mean;
    j.loss = loss;
    j.lse = lse;
    j.total = row0 + rows == M ? total : nullptr;
    j.M = M;
    auto join = [&](int mode, int when_redo) {
      j.mode = mode;
      j.when_redo = when_redo;
      return launch_counted(ce_join_kernel, dim3(static_cast<unsigned>(ceil_div(rows, 32))), dim3(32 * kJoinWarps), 0,
                            LORA_KIND_LOSS, stream, j);
    };
    // the row's sum on its own, then (for dx) exponentials relative to it
    auto exact = [&](int when_redo) {
      g.when_redo = when_redo;
      g.zsum = s.zsum;
      LGB_TRY(ce_gemm(CE_STATS, g, stream));
      LGB_TRY(join(want ? CE_JOIN_EXACT : CE_JOIN_LOSS, when_redo));
      g.zsum = nullptr;
      return want ? ce_gemm(CE_GRAD, g, stream) : LORA_OK;
    };
    if (!want || P.exact) {
      LGB_TRY(exact(0));
    } else {
      g.zsum = s.zsum;
      LGB_TRY(ce_gemm(CE_GRAD, g, stream));
      LGB_TRY(join(CE_JOIN_GRAD, 0));
      LGB_TRY(exact(1));
    }
    if (!want) continue;
    CeGemmParams d;
    std::memset(static_cast<void*>(&d), 0, sizeof(d));
    if (!encode_map(&d.a, s.e, kBK, P.rows * P.blocks, kBK, kBK, kBM) || !encode_map(&d.b, W, h, vocab, h, 64, 64))
      return LORA_ERR_CUDA;
    d.piece = s.piece + k;
    d.blocks = static_cast<int>(P.blocks);
    d.kb_total = kb_v;
    d.kb_range = ce_part_long(rows, tiles_h, kb_v, num_sms() / 2) ? kCePartKb : kb_v;
    d.kvalid = static_cast<int>(vocab);
    d.tiles_n = tiles_h;
    d.narrow = h - (tiles_h - 1) * int64_t(256) <= 128;
    d.band = raster_band();
    d.status = status;
    d.slab = s.slab;
    d.balance = P.exact ? 1 : 2;
    d.tsum = s.tsum;
    d.wsum = s.wsum;
    d.ldp = P.rows;
    d.slots = static_cast<int>(P.slots);
    d.rs = r.rs;
    d.coef = r.coef;
    LGB_TRY(ce_gemm(CE_PART, d, stream));
    CeDxArgs a;
    a.piece = s.piece + k;
    a.r = r;
    a.slab = s.slab;
    a.tiles_n = tiles_h;
    a.band = d.band;
    a.h = static_cast<int>(h);
    a.W = gather.W;
    a.column = s.column;
    a.scale = o.logit_scale;
    a.share = share;
    a.mean = mean;
    a.dx = gather.dx;
    const int64_t blocks = ceil_div(rows * (h / 8), 256), most = kDxBlocks * num_sms();
    LGB_TRY(launch_counted(ce_dx_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(256), 0,
                           LORA_KIND_LOSS, stream, a));
  }
  return LORA_OK;
}

extern "C" lora_status_t lora_scale_rows(int64_t M, int64_t h, const void* x, const float* g, int g_stride, void* y, void* ws,
                                         size_t ws_bytes, cudaStream_t stream) {
  NvtxRange nvtx_range("lora_scale_rows");
  if (M < 0 || h < 1 || (g_stride != 0 && g_stride != 1) || (M > 0 && (!x || !g || !y))) return LORA_ERR_INVALID_ARG;
  if (M > kMaxExtent || h > kMaxExtent) return LORA_ERR_UNSUPPORTED;
  if (h % 8 || !aligned(x, 16) || !aligned(y, 16) || !aligned(g, 4)) return LORA_ERR_ALIGNMENT;
  LGB_TRY(check_ws(ws, ws_bytes, kWsHeader));
  if (M == 0) return LORA_OK;
  ScaleArgs p;
  p.x = static_cast<const bf16*>(x);
  p.g = g;
  p.g_stride = g_stride;
  p.y = static_cast<bf16*>(y);
  p.M = M;
  p.h = static_cast<int>(h);
  const int64_t blocks = ceil_div(M * (h / 8), 256);          // below 2^59
  return launch_counted(scale_rows_kernel, dim3(static_cast<unsigned>(blocks < (1 << 30) ? blocks : (1 << 30))), dim3(256), 0,
                        LORA_KIND_LOSS, stream, p);
}
