// What the attention kernels over the paged cache share: arguments, the shared-out work,
// the split sums and their joining.
//
// Work.  Query rows of one sequence that read the same cache head are packed, row = token *
// hs + head of the slice (a slice is the hs query heads of a cache head that one tile
// takes, all of them unless they outnumber its rows), as many whole tokens as a tile's
// rows hold.  An item is (sequence, slice, tile of tt tokens); it has one unit for every KT
// positions that its rows see (one where they see none) and IT units before them, for what
// an item costs beside its tiles (Q, merging, the output).  The lengths are known on the
// device only, so every CTA counts all units itself and takes an equal, contiguous share of
// them: long and short sequences, causal tiles and few-row batches fill the GPU alike.  An
// item that a share boundary cuts leaves its parts' maxima, sums and unnormalised outputs in
// the workspace, at most two of them per CTA, and a second launch joins them in a fixed
// order.
#pragma once

#include "serve.cuh"

namespace lgb {

struct AttnParams {
  CUtensorMap kmap, vmap;    // pages as rows [n_pages * heads * page_size] x head_dim
  CUtensorMap qmap;          // many-row kernel: q as [tokens x heads x head_dim]
  HeadsView q;
  int hq, group;             // query heads; of them per cache head
  int hs, spg, slices;       // heads per slice, slices per cache head, slices in all
  int th, tt;                // tokens of a row half (rows / hs), and of a tile
  int M;
  CacheArgs cache;
  const int* table;
  long long max_pages;
  const int* kv_len;
  const int* cu_q;
  int n_seqs;
  float scale_log2;          // score scale times log2(e)
  int causal;
  int window;                // 0: none
  bf16* out;
  float* lse;
  unsigned* status;
  unsigned long long timeout_ns;
  int inject_stall;          // failure-path tests: the first stage is never filled
  float* part_o;             // [CTAs][2][R][D]
  float2* part_ml;           // [CTAs][2][R]: maximum (log2 scale) and sum
  struct JoinDesc* join;     // [CTAs]
};

struct JoinDesc {
  int parts;                 // parts of the item that starts, but does not end, in this CTA (0: none)
  int q0, n, kv;             // its sequence
  int slice, rt;
};

struct Seq {
  int q0, n, kv;
};

// Sequence b with its device values cut to what exists; `report` flags what was cut.
__device__ __forceinline__ Seq load_seq(const AttnParams& p, int b, bool report) {
  const int c0 = __ldg(p.cu_q + b), c1 = __ldg(p.cu_q + b + 1), kv = __ldg(p.kv_len + b);
  const long long most = min(p.max_pages << p.cache.page_shift, 0x7fff0000ll);   // tile ends stay 32-bit
  Seq s;
  s.q0 = min(max(c0, 0), p.M);
  s.n = min(max(c1, s.q0), p.M) - s.q0;
  s.kv = static_cast<int>(min(static_cast<long long>(max(kv, 0)), most));
  if (report && (s.q0 != c0 || s.q0 + s.n != c1 || s.kv != kv)) atomicOr(p.status, kStatusInput);
  return s;
}

__device__ __forceinline__ int row_tiles(const AttnParams& p, const Seq& s) { return (s.n + p.tt - 1) / p.tt; }

// The lowest position that token t's window leaves it (0 without a window).
__device__ __forceinline__ int first_seen(const AttnParams& p, const Seq& s, int t) {
  return p.window > 0 ? static_cast<int>(max(0ll, static_cast<long long>(s.kv) - s.n + t - p.window + 1)) : 0;
}

// Tiles [j0, j1) of KT positions that row tile rt sees any of; one empty tile if none.
template <int KT>
__device__ __forceinline__ void item_tiles(const AttnParams& p, const Seq& s, int rt, int& j0, int& j1) {
  const int t0 = rt * p.tt, t1 = min(s.n, t0 + p.tt) - 1;
  const int off = s.kv - s.n;
  const int hi = p.causal ? max(0, min(s.kv, off + t1 + 1)) : s.kv;
  j0 = first_seen(p, s, t0) / KT;
  j1 = max(j0 + 1, (hi + KT - 1) / KT);
}

// The positions [lo, hi) that the row of token t sees.
__device__ __forceinline__ void row_range(const AttnParams& p, const Seq& s, int t, int& lo, int& hi) {
  const int pos = s.kv - s.n + t;
  hi = p.causal ? min(s.kv, pos + 1) : s.kv;
  lo = first_seen(p, s, t);
}

// Token and query head of row r of tile rt's half q; false past the half's tokens, the
// sequence or the slice.
__device__ __forceinline__ bool row_owner(const AttnParams& p, const Seq& s, int slice, int rt, int q, int r, int& tok,
                                          int& head) {
  const int t = r / p.hs, g = r - t * p.hs;
  const int kvh = slice / p.spg, first = (slice - kvh * p.spg) * p.hs;
  tok = rt * p.tt + q * p.th + t;
  head = kvh * p.group + first + g;
  return t < p.th && tok < s.n && first + g < p.group;
}

// A CTA's share, found by all NT threads together.
struct Plan {
  long long units, quota;    // of this CTA; of a full share
  int b, slice, rt, skip;    // where it starts: the item, and the units of it that precede
  Seq s;                     // that item's sequence
};
template <int NT>
struct PlanScratch {
  long long warp_sum[NT / 32];
  long long base, cost;
  Plan plan;
};

template <int KT, int IT>
__device__ __forceinline__ long long seq_cost(const AttnParams& p, const Seq& s, bool live) {
  // units of one slice; sequences of more than four row tiles are counted by the whole warp
  const int nrt = live ? row_tiles(p, s) : 0;
  long long c = 0;
  if (nrt <= 4)
    for (int rt = 0; rt < nrt; ++rt) {
      int j0, j1;
      item_tiles<KT>(p, s, rt, j0, j1);
      c += j1 - j0 + IT;
    }
  unsigned many = __ballot_sync(0xffffffffu, nrt > 4);
  const int lane = threadIdx.x & 31;
  while (many) {
    const int src = __ffs(many) - 1;
    many &= many - 1;
    Seq o;
    o.q0 = 0;
    o.n = __shfl_sync(0xffffffffu, s.n, src);
    o.kv = __shfl_sync(0xffffffffu, s.kv, src);
    const int tiles = __shfl_sync(0xffffffffu, nrt, src);
    long long sum = 0;
    for (int rt = lane; rt < tiles; rt += 32) {
      int j0, j1;
      item_tiles<KT>(p, o, rt, j0, j1);
      sum += j1 - j0 + IT;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == src) c = sum;
  }
  return c;
}

template <int NT>
__device__ __forceinline__ long long block_scan(long long v, PlanScratch<NT>& sh, long long& total) {
  // exclusive prefix sum over the block's threads
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  __syncthreads();
  if (lane == 31) sh.warp_sum[warp] = inc;
  __syncthreads();
  long long before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += sh.warp_sum[w];
    total += sh.warp_sum[w];
  }
  return before + inc - v;
}

template <int KT, int IT, int NT>
__device__ __forceinline__ void make_plan(const AttnParams& p, PlanScratch<NT>& sh) {
  const int tid = threadIdx.x;
  const bool one = p.n_seqs <= NT;
  long long all = 0, c = 0, cost1 = 0, first = 0;
  Seq s = {0, 0, 0};
  for (int b0 = 0; b0 < p.n_seqs; b0 += NT) {
    const bool live = b0 + tid < p.n_seqs;
    if (live) s = load_seq(p, b0 + tid, blockIdx.x == 0);
    cost1 = seq_cost<KT, IT>(p, s, live);
    c = cost1 * p.slices;
    long long total;
    first = block_scan<NT>(c, sh, total);
    all += total;
  }
  const long long up = all + gridDim.x - 1;
  const long long quota = max(up <= 0x7fffffff ? static_cast<long long>(static_cast<unsigned>(up) / gridDim.x) : up / gridDim.x, 1ll);
  const long long u0 = quota * blockIdx.x;
  if (tid == 0) {
    sh.plan.quota = quota;
    sh.plan.units = max(0ll, min(quota, all - u0));
  }
  __syncthreads();
  if (u0 >= all) return;
  long long before = 0;
  for (int b0 = 0; b0 < p.n_seqs; b0 += NT) {
    long long total = 0;
    if (!one) {
      const bool live = b0 + tid < p.n_seqs;
      if (live) s = load_seq(p, b0 + tid, false);
      cost1 = seq_cost<KT, IT>(p, s, live);
      c = cost1 * p.slices;
      first = block_scan<NT>(c, sh, total);
    }
    if (u0 >= before + first && u0 < before + first + c) {     // (c is the slices' units together)
      sh.plan.b = b0 + tid;
      sh.plan.s = s;
      sh.base = u0 - before - first;
      sh.cost = cost1;
    }
    before += total;
  }
  __syncthreads();
  if (tid < 32) {
    // 32-bit division where it fits (a 64-bit one takes several times as long)
    s = sh.plan.s;
    const long long base = sh.base, cost = sh.cost;
    const int slice = base <= 0x7fffffff && cost <= 0x7fffffff
                          ? static_cast<int>(static_cast<unsigned>(base) / static_cast<unsigned>(cost))
                          : static_cast<int>(base / cost);
    long long rem = base - slice * cost;
    const int tiles = row_tiles(p, s);
    for (int rt0 = 0; rt0 < tiles; rt0 += 32) {
      int j0 = 0, j1 = -IT;
      if (rt0 + tid < tiles) item_tiles<KT>(p, s, rt0 + tid, j0, j1);
      const int units = j1 - j0 + IT;
      long long inc = units;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, inc, d);
        if (tid >= d) inc += o;
      }
      if (rem < inc && rem >= inc - units) {
        sh.plan.slice = slice;
        sh.plan.rt = rt0 + tid;
        sh.plan.skip = static_cast<int>(rem - (inc - units));
      }
      const long long window = __shfl_sync(0xffffffffu, inc, 31);
      if (rem < window) break;
      rem -= window;
    }
  }
  __syncthreads();
}

// One CTA's part of an item: tiles [ja, jb).
struct Span {
  Seq s;
  int b, slice, rt;
  int ja, jb;
  bool starts, ends;         // holds the item's first / last tile
  int after;                 // units of the item after this part
};

// No row of the item sees a position before this one.  Pages that lie wholly before it may have
// been released: their table entries are not looked at, and their boxes are loaded from
// before the first row of the cache, which TMA fills with zeros (their scales are not loaded).
__device__ __forceinline__ int lowest_seen(const AttnParams& p, const Span& w) { return first_seen(p, w.s, w.rt * p.tt); }

// Walks a CTA's share; every role walks it by itself.
template <int KT, int IT>
struct Walker {
  long long left;
  int b, slice, rt, skip;
  Seq s;
  int tiles;
  __device__ __forceinline__ Walker(const AttnParams& p, const Plan& plan)
      : left(plan.units), b(plan.b), slice(plan.slice), rt(plan.rt), skip(plan.skip), s(plan.s) {
    tiles = left > 0 ? row_tiles(p, s) : 0;
  }
  __device__ __forceinline__ bool next(const AttnParams& p, Span& w) {
    while (left > 0) {
      if (rt == tiles) {
        rt = 0;
        if (++slice == p.slices) {
          slice = 0;
          do {
            if (++b >= p.n_seqs) return false;
            s = load_seq(p, b, false);
          } while (s.n == 0);
          tiles = row_tiles(p, s);
        }
      }
      int j0, j1;
      item_tiles<KT>(p, s, rt, j0, j1);
      // units [skip, till) of the item's IT + (j1 - j0)
      const int units = IT + j1 - j0, till = static_cast<int>(min(static_cast<long long>(units), skip + left));
      left -= till - skip;
      w.ja = j0 + max(0, skip - IT);
      w.jb = j0 + max(0, till - IT);
      w.s = s;
      w.b = b;
      w.slice = slice;
      w.rt = rt;
      w.starts = w.ja == j0;
      w.ends = w.jb == j1;
      w.after = units - till;
      skip = 0;
      ++rt;
      if (w.ja < w.jb) return true;       // else the share ended in the item's first units
    }
    return false;
  }
};

// Bounded wait (the GEMM kernels' rule: wall-clock limit, abort flag shared by the CTA).
__device__ __forceinline__ bool attn_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, const AttnParams& p) {
  if (mbar_try_wait_short(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (;;) {
    if (mbar_try_wait_short(bar, parity)) return true;
    if (*abort_flag) return false;
    if (global_timer_ns() - t0 > p.timeout_ns) {
      *abort_flag = 1;
      atomicOr(p.status, kStatusTimeout);
      return false;
    }
  }
}
__device__ __forceinline__ void attn_wait_drain(uint32_t bar, uint32_t parity, const AttnParams& p) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > 20000000ull) {
      atomicOr(p.status, kStatusTimeout);
      return;
    }
  }
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float log2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A running maximum is raised only when a tile exceeds it by more than this (log2): until
// then the weights are at most 2^8, which f32 sums and bf16 weights hold as exactly as
// smaller ones, and the output accumulators need no rescaling.
constexpr float kMaxSlack = 8.0f;

// ---------------------------------------------------------------- joining the parts

// Blocks (CTA c, rows): the item that starts in c's share and continues in the following
// CTAs' (part 0 in slot [c][1], the others in slots [c + i][0]).  Each thread joins four
// features of a row: sum_i 2^(m_i - max m) o_i over sum_i 2^(m_i - max m) l_i.
template <int D, int R>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ AttnParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int c = blockIdx.x;
  const JoinDesc d = p.join[c];
  if (d.parts == 0) return;
  constexpr int kCols = D / 4;
  const Seq s = {d.q0, d.n, d.kv};
  const int col = threadIdx.x % kCols;
  for (int r = blockIdx.y * (128 / kCols) + threadIdx.x / kCols; r < R; r += gridDim.y * (128 / kCols)) {
    int tok, head;
    if (!row_owner(p, s, d.slice, d.rt, R > 128 ? r >> 7 : 0, R > 128 ? r & 127 : r, tok, head)) continue;
    const float2* ml = p.part_ml + r;
    float top = -INFINITY;
#pragma unroll 4
    for (int i = 0; i < d.parts; ++i) top = fmaxf(top, ml[(2ll * (c + i) + (i == 0)) * R].x);
    const float ref = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int i = 0; i < d.parts; ++i) {
      const long long slot = 2ll * (c + i) + (i == 0);
      const float2 v = ml[slot * R];
      const float4 x = *reinterpret_cast<const float4*>(p.part_o + (slot * R + r) * D + 4 * col);
      const float w = exp2_approx(v.x - ref);
      sum += w * v.y;
      o.x += w * x.x;
      o.y += w * x.y;
      o.z += w * x.z;
      o.w += w * x.w;
    }
    const float inv = top == -INFINITY && sum == 0.0f ? 0.0f : 1.0f / sum;
    const long long row = static_cast<long long>(d.q0 + tok) * p.hq + head;
    uint2 w;
    w.x = pack_bf16x2(o.x * inv, o.y * inv);
    w.y = pack_bf16x2(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(p.out + row * D + 4 * col) = w;
    if (p.lse != nullptr && col == 0)
      p.lse[row] = inv == 0.0f && sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
  }
}

// ---------------------------------------------------------------- launches

// Most CTAs of a launch, whatever the device: the parts' slots are sized for it.
constexpr int kMaxFewCtas = 480;
constexpr int kMaxManyCtas = 160;

constexpr int kFewRows = 16;          // rows of the few-row kernel's tiles
// The many-row kernel's tiles: one or two row halves of 128 (one at head_dim 256).
lora_status_t launch_attn_many(AttnParams& p, int halves, int head_dim, int format, cudaStream_t st);
lora_status_t launch_attn_few(AttnParams& p, int head_dim, int format, cudaStream_t st);

// Slices and tiles of a call whose row halves hold `rows` rows.
inline void set_tiles(AttnParams& p, int rows, int halves) {
  p.spg = static_cast<int>(ceil_div(p.group, rows));
  p.hs = static_cast<int>(ceil_div(p.group, p.spg));
  p.slices = p.cache.heads * p.spg;
  p.th = rows / p.hs;
  p.tt = halves * p.th;
}

// The cache's pages as rows, in boxes of at most `tile` rows of one page.
inline bool encode_pages(AttnParams& p, int row_elems, int elem_bytes, int box_bytes, int tile) {
  const uint64_t rows = static_cast<uint64_t>(p.cache.n_pages) * p.cache.heads << p.cache.page_shift;
  const uint32_t box_rows = (1 << p.cache.page_shift) < tile ? 1 << p.cache.page_shift : tile;
  return encode_map_rows(&p.kmap, p.cache.k, elem_bytes, rows, row_elems, box_rows, box_bytes) &&
         encode_map_rows(&p.vmap, p.cache.v, elem_bytes, rows, row_elems, box_rows, box_bytes);
}

}  // namespace lgb
