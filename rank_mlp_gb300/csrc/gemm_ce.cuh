// The linear cross entropy's GEMMs on CTA pairs (256 x 256 tiles, tcgen05 cta_group::2), and
// what they share with the kernels between them (linear_ce.cu).
//
// Logits never leave the chip as such.  One GEMM multiplies the hidden rows by the head's
// K-major rows and its epilogue, a row a thread, turns a tile's 256 logits into
//   CE_STATS   the row's maximum and sum of exponentials relative to it
//   CE_GRAD    the row's exponentials relative to a reference known beforehand, stored in bf16
//              (and their sum)
// the other, CE_PART, multiplies those exponentials by the head read MN-major.
//
// With e_v = 2^(z_v - ref) the gradient of a row is, up to the row's factor, sum_v e_v W_v / S
// minus W_y: bf16's range lets e_v keep its relative precision whatever the reference, so the
// product needs no second pass over the logits once S is known.  The label's own term is left
// out of e and S: it joins in f32 from the label's logit, where 1 - p_y keeps its precision
// however near p_y is to 1.
//
// Rounding the weights to bf16 moves their sum, and what a head's rows have in common is multiplied by
// that sum: it would no longer be what the label's term takes off.  So the weights' sums before and
// after the rounding are kept beside S, and ce_balance makes the second one the first.
//
// Rows are the labelled tokens, packed; their number is on the device, so a launch covers the
// most rows there can be and its units follow from the number it finds.
//
// Bound by the matrix units and, at 14 k-blocks a tile, by what the epilogue adds: 3686 rows x 896
// against 131072 words take 615 us (1.41 PFLOP/s).  Before the weights' sums were kept it was 600 us, 538 without
// the stores of the exponentials, 558 with them all in one place (so their way to memory costs most), 505 with no
// epilogue.  At 64 k-blocks capped logits run at 1.4 to 1.5 PFLOP/s, the loss alone at 1.65; CE_PART at 1.55 to 1.7.
#pragma once

#include "gemm_pair.cuh"

namespace lgb {

enum CeKind : int { CE_STATS = 0, CE_GRAD = 1, CE_PART = 2 };

constexpr int kCeStages = 6;
// Eight epilogue warps, two for each TMEM lane quarter, and so two partial results of a row in a tile.
// (Four took as long at 14 and at 64 k-blocks a tile: 1275 and 5282 us for 1271 and 5306 with eight.)
constexpr int kCeWarps = 8;
constexpr int kCeSlots = kCeWarps / 4;
// k-blocks that a logit is summed over in tensor memory at most.  The matrix units cut what falls below the
// last place of their running sum, always toward zero, so that a logit comes out short by a share of
// itself that grows with the products it sums.  Longer rows are taken in parts that are joined in f32
// in the epilogue's registers.  The loss's error at h = 4096 over 5003 words, in 1e-6 of itself, without parts, with
// parts of 16 (h = 896; f32 products at 4096):
//   normal         1.85   0.40   (0.36, 0.15)
//   heavy-tailed   4.74   1.38   (1.18, 1.07)
//   label-pulled   2.12   0.48   (0.46, 0.54)
//   lse, one sign  6.7    0.87   (0.73)
// 2048 tokens x 4096 against 50,257 words, the loss alone: 490 us without parts, 496 with parts of 32
// k-blocks, 508 with 16, 535 with 8; 4096 capped rows with dx the same within 1% but for parts of 8 (2% more).
constexpr int kCeRangeKb = 16;
// The same for the product with the head, whose weights are all positive: where the head's rows have a part in
// common its sums grow steadily over the whole vocabulary.  (4096 rows, 131,072 words, a common part five times the
// rows' own: dx off by 4e-3 along it without parts, 4.2e-4 with parts of 256 k-blocks, 9e-5 with 64, 5e-5 with 16;
// 1255, 1265, 1270 and 1280 us at h = 896.)
constexpr int kCePartKb = 64;
constexpr int kCeMaxSplits = 32;
constexpr int kCeTailUnits = 304;        // units of a launch at most that are parts of tiles
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// What a launch finds on the device about its piece of the rows.
struct CePiece {
  int live;                // labelled rows of the piece
  int whole;               // CE_PART: tiles done in one unit, a multiple of the CTA pairs,
  int splits;              // and the k-ranges that each tile after them is cut into
  unsigned redo;           // CE_GRAD's sums left their range: the launches of the second try run
};

// Logits in units of ln 2 from accumulator values: z2 = v * k2, or cap2 * tanh(v * kc).
struct CeLogit {
  float k2, cap2, kc;
};

struct CeGemmParams {
  CUtensorMap a, b;
  const CePiece* piece;
  int when_redo;           // 1: only if the piece's `redo` is set
  int kb_total, kvalid;    // 64-wide k-blocks, valid K
  int kb_range;            // k-blocks of a part of the sums
  int tiles_n, band;
  int narrow;              // CE_PART: 1 if the last n-tile is 128 columns wide
  unsigned* status;
  unsigned long long timeout_ns;
  int inject_stall;
  // CE_STATS, CE_GRAD (arrays start at the piece's first row)
  int vocab;
  CeLogit lg;
  const int* label;
  const float* ref2;
  float2* part;            // CE_STATS: [tiles_n * kCeSlots][ldp] (maximum, sum), both without the label
  float* psum;             // CE_GRAD: the sums alone,
  float* wsum;             // those of the weights as they are stored in e,
  float* tsum;             // and before their rounding (with a cap; without, they are psum)
  float* zsum;             // [tiles_n * kCeSlots][ldp] sums of z2, label included, or NULL
  float* zlab;             // the label's z2
  float* slope;            // with a cap: its tanh's slope (z2 near the cap says little of it)
  long long ldp;
  __nv_bfloat16* e;        // [rows / 128][blocks][128][64]: what one CTA takes of a k-block together
  int blocks;              // 64-wide blocks of the vocabulary
  float minus;             // CE_GRAD: taken off each exponential before the tanh's slope
  // CE_PART
  float* slab;             // [units][256][256]
  int balance;             // rows' factors follow the weights' sums here: 0 no, 1 yes, 2 if the piece's `redo` is set
  int slots;
  float* rs;
  float* coef;
};

// The product with the head has few tiles and a long K.  Whole waves of tiles on the CTA pairs are
// done a tile a unit; the `tail` tiles that are left, fewer than pairs, are cut into k-ranges: the
// busiest pair then works through ceil(tail s / pairs) units of kb / s k-blocks, each of which also
// has its 256 KB of partial sums written and read back, at a pair's share of the memory rate
// about the time of kCeSlabKb k-blocks.
constexpr int kCeSlabKb = 21;
__host__ __device__ inline int ce_splits(int tail, int kb, int pairs) {
  int best = 1;
  float least = 3.0e38f;
  for (int s = 1; s <= kCeMaxSplits; ++s) {
    if (s > 1 && (tail * s > kCeTailUnits || kb < 4 * s)) break;
    const float cost = static_cast<float>((tail * s + pairs - 1) / pairs) * (static_cast<float>(kb) / s + kCeSlabKb);
    if (cost < least * 0.999f) {
      least = cost;
      best = s;
    }
  }
  return best;
}
__host__ __device__ inline CePiece ce_piece(int live, int tiles_n, int kb, int pairs) {
  const int tiles = (live + 255) / 256 * tiles_n;
  CePiece q;
  q.live = live;
  q.whole = tiles / pairs * pairs;
  q.splits = tiles > q.whole ? ce_splits(tiles - q.whole, kb, pairs) : 1;
  q.redo = 0;
  return q;
}

// Whether a piece of up to `rows` rows can have units of more than kCePartKb k-blocks, however many of them are
// labelled.  The kernel without parts takes 63 registers a thread instead of 168, so that the next kernel's blocks
// fit beside it: 64 tokens x 896 x 32,000 64.0 us instead of 65.8.
inline bool ce_part_long(int64_t rows, int tiles_n, int kb, int pairs) {
  for (int64_t m = 1; m <= (rows + 255) / 256; ++m) {
    if (m * tiles_n >= pairs) return kb > kCePartKb;
    const int s = ce_splits(static_cast<int>(m) * tiles_n, kb, pairs);
    if ((kb + s - 1) / s > kCePartKb) return true;
  }
  return false;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// z2 of an accumulator value, and with a cap the tanh's slope 1 - tanh^2.  From 0.55 on both come from
// q = 2 / (1 + e^(2|x|)): tanh |x| = 1 - q, 1 - tanh^2 x = q (2 - q).  Below it 1 - q would keep the last places of 1,
// so a logit those of its cap; there tanh x = x + x^3 R(x^2), R fitted to within 4e-8 of tanh itself.
enum CeCap : int { CE_NO_CAP = 0, CE_CAP = 1, CE_CAP_LOW = 2 };      // LOW: |x| is below 0.55
constexpr float kCeLow = 0.55f;
template <int CAP>
__device__ __forceinline__ float ce_logit(float v, const CeLogit& lg, float& slope) {
  if constexpr (CAP == CE_NO_CAP) {
    slope = 1.0f;
    return v * lg.k2;
  } else {
    const float x = v * lg.kc, u = x * x;
    const float r = fmaf(fmaf(fmaf(0.016437581f, u, -0.052671812f), u, 0.13320725f), u, -0.33332947f);
    const float low = fmaf(x * u, r, x);
    if constexpr (CAP == CE_CAP_LOW) {
      slope = fmaf(-low, low, 1.0f);
      return lg.cap2 * low;
    } else {
      const float q = __fdividef(2.0f, 1.0f + exp2_approx(fabsf(x) * (2.0f * kLog2e)));
      const bool small = fabsf(x) < kCeLow;
      slope = small ? fmaf(-low, low, 1.0f) : q * (2.0f - q);
      return lg.cap2 * (small ? low : copysignf(1.0f - q, x));
    }
  }
}

// Factors of a row (rs: of its weights' product with W, coef: of the label's row of W) for weights that
// summed to t and, rounded, to w.  All weights are multiplied by t / w, which weights of one sign move by 2^-8
// at most.  Where it is more, their signs differ and they cancel (the smoothing's part, with a cap), and the
// difference goes to the label instead.
__device__ __forceinline__ void ce_balance(float t, float w, float& rs, float& coef) {
  if (fabsf(t - w) <= 0x1p-8f * fabsf(t) && w != 0.0f) {
    rs *= t / w;
  } else {
    coef = fmaf(rs, t - w, coef);
  }
}

// mbar_arrive_cluster that orders no memory: what it announces is that tensor memory has been read
// (tcgen05.wait::ld, then the fence before it).  A releasing arrive would first wait for the
// thread's stores of exponentials.
__device__ __forceinline__ void arrive_read(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

__device__ __forceinline__ bool ce_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, const CeGemmParams& p) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (global_timer_ns() - t0 > p.timeout_ns) {
      *abort_flag = 1;
      atomicOr(p.status, kStatusTimeout);
      return false;
    }
  }
}
__device__ __forceinline__ void ce_wait_drain(uint32_t bar, uint32_t parity, const CeGemmParams& p) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > 20000000ull) {
      atomicOr(p.status, kStatusTimeout);
      return;
    }
  }
}

// The units of a CTA pair: tiles in bands of n-tiles (the n-tile fastest inside a band); of the
// tiles cut into k-ranges all first ranges, then all second ones, so that pairs working at the same
// time read the same slices.
struct CeUnit {
  int u, tm, tn, kb0, kb1;
};
struct CeIter {
  int q, turn, step, end, whole, tail, tiles_m, splits;
  __device__ __forceinline__ CeIter(const CeGemmParams& p, int live, int whole_, int splits_, int pair, int npairs) {
    tiles_m = (live + 2 * kBM - 1) / (2 * kBM);
    const int tiles = tiles_m * p.tiles_n;
    whole = whole_ < 0 ? tiles : min(whole_, tiles);
    tail = tiles - whole;
    splits = splits_;
    q = pair;
    turn = 0;
    step = npairs;
    end = whole + tail * splits;
  }
  // Dealt round-robin, each round starting one pair further: a pair's units then fall on different
  // n-tiles, and the narrow one is every pair's in turn.
  __device__ __forceinline__ bool next(const CeGemmParams& p, CeUnit& U) {
    const int u = turn * step + q;
    if (u >= end) return false;
    ++turn;
    if (++q == step) q = 0;
    int t = u;
    U.u = u;
    U.kb0 = 0;
    U.kb1 = p.kb_total;
    if (u >= whole) {
      const int v = u - whole, s = v / tail;
      t = whole + v - s * tail;
      U.kb0 = static_cast<int>(static_cast<long long>(p.kb_total) * s / splits);
      U.kb1 = static_cast<int>(static_cast<long long>(p.kb_total) * (s + 1) / splits);
    }
    const int b = t / (tiles_m * p.band);
    const int rem = t - b * tiles_m * p.band;
    const int nb = min(p.band, p.tiles_n - b * p.band);
    U.tm = rem / nb;
    U.tn = b * p.band + rem % nb;
    return true;
  }
};
// The place of tile (tm, tn) in that order.
__device__ __forceinline__ int ce_tile_place(int tm, int tn, int tiles_m, int tiles_n, int band) {
  const int b = tn / band, nb = min(band, tiles_n - b * band);
  return b * tiles_m * band + tm * nb + tn - b * band;
}

// 32 logits of a row, columns [col0, col0 + 32): into the row's running (top, sum, zs), the label's
// own into zlab, and for CE_GRAD their weights into e and the weights' sums, rounded and not, into ws and
// (with a cap) ts.  Whole warps call it.
template <int KIND, bool CAP>
__device__ __forceinline__ void ce_chunk(const CeGemmParams& p, const uint32_t (&v)[32], int col0, int row, bool ok, int label,
                                         float ref2, float& top, float& sum, float& zs, float& ws, float& ts) {
  if (col0 >= p.vocab) return;                   // wholly past the vocabulary
  const int at = label - col0;                   // the label's place in the chunk
  const int width = p.vocab - col0;              // columns below the vocabulary's size
  const bool plain = !__any_sync(0xffffffffu, static_cast<unsigned>(at) < 32u) && width >= 32;
  // the label's column and those past the vocabulary leave the sums
  auto chunk = [&](auto plain_tag, auto cap_tag) {
    constexpr bool PLAIN = decltype(plain_tag)::value != 0;
    constexpr int LOGIT = decltype(cap_tag)::value;
    if constexpr (KIND == CE_STATS) {
      float z[32], most = -INFINITY;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        float slope;
        z[j] = ce_logit<LOGIT>(__uint_as_float(v[j]), p.lg, slope);
        if (!PLAIN) {
          if (p.zsum != nullptr && j < width) zs += z[j];
          if (j == at) {
            p.zlab[row] = z[j];
            if (CAP) p.slope[row] = slope;
          }
          if (j == at || j >= width) z[j] = -INFINITY;
        }
        most = fmaxf(most, z[j]);
      }
      if (PLAIN && p.zsum != nullptr) {
#pragma unroll
        for (int j = 0; j < 32; ++j) zs += z[j];
      }
      if (most > top) {
        sum *= exp2_approx(top - most);
        top = most;
      }
      const float base = top == -INFINITY ? 0.0f : top;
      float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        s0 += exp2_approx(z[j] - base);
        s1 += exp2_approx(z[j + 1] - base);
      }
      sum += s0 + s1;
    } else {
      uint32_t w[16];
      // of the exponentials, of the weights as stored and as they were, two terms an instruction (one each: 64 x 896 x
      // 32,000 64.9 us instead of 62.0)
      TwoSums all, stored, before;
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        float x[2], e[2], d[2];
        if (!CAP) fma_two(__uint_as_float(v[j]), __uint_as_float(v[j + 1]), p.lg.k2, -ref2, d[0], d[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float slope = 1.0f, z = 0.0f;
          if (CAP || !PLAIN || p.zsum != nullptr) z = ce_logit<LOGIT>(__uint_as_float(v[j + h]), p.lg, slope);
          x[h] = exp2_approx(CAP ? z - ref2 : d[h]);
          if (p.zsum != nullptr && (PLAIN || j + h < width)) zs += z;
          if (!PLAIN) {
            if (j + h == at) {
              p.zlab[row] = z;
              if (CAP) p.slope[row] = slope;
            }
            if (j + h == at || j + h >= width) x[h] = 0.0f;
          }
          e[h] = CAP ? (x[h] - p.minus) * slope : x[h];
          if (CAP && !PLAIN && (j + h == at || j + h >= width)) e[h] = 0.0f;
        }
        w[j / 2] = pack_bf16x2(e[0], e[1]);
        all.add(x[0], x[1]);
        stored.add(__uint_as_float(w[j / 2] << 16), __uint_as_float(w[j / 2] & 0xFFFF0000u));
        if (CAP) before.add(e[0], e[1]);
      }
      sum += all.total();
      ws += stored.total();
      if (CAP) ts += before.total();
      if (ok) {
        // (the same stores into rows of the whole vocabulary: 635 us for 608)
        __nv_bfloat16* dst = p.e + (static_cast<long long>(row >> 7) * p.blocks + (col0 >> 6)) * 8192 + (row & 127) * 64 + (col0 & 63);
        st_global_v8(dst, w);
        st_global_v8(dst + 16, w + 8);
      }
    }
  };
  if constexpr (CAP) {
    // Where all of a chunk's logits are far enough below the cap, as most are, neither the exponential nor the
    // quotient is needed.  (4096 tokens x 4096 x 131,072 words, cap 30: 5.25 ms; 5.65 with the general form
    // throughout, 5.11 with the exponential's form alone.)
    float most = 0.0f;
#pragma unroll
    for (int j = 0; j < 32; ++j) most = fmaxf(most, fabsf(__uint_as_float(v[j])));
    if (!plain) {
      chunk(ActTag<0>{}, ActTag<CE_CAP>{});
    } else if (__all_sync(0xffffffffu, most * fabsf(p.lg.kc) < kCeLow)) {
      chunk(ActTag<1>{}, ActTag<CE_CAP_LOW>{});
    } else {
      chunk(ActTag<1>{}, ActTag<CE_CAP>{});
    }
  } else if (plain) {
    chunk(ActTag<1>{}, ActTag<CE_NO_CAP>{});
  } else {
    chunk(ActTag<0>{}, ActTag<CE_NO_CAP>{});
  }
}

// What the epilogue of one tile row has on its way: the row's running results over the warp's share `part`
// of the tile's columns.
template <int KIND, bool CAP>
struct CeRow {
  static constexpr int kSpan = 256 / kCeSlots;
  int row, label, first;
  bool ok;                 // the row is one of the piece's
  float ref2;
  float top = -INFINITY, sum = 0.0f, zs = 0.0f, ws = 0.0f, ts = 0.0f;
  __device__ __forceinline__ CeRow(const CeGemmParams& p, const CeUnit& U, int row_, bool ok_, int part) : row(row_), ok(ok_) {
    first = U.tn * 256 + part * kSpan;
    label = ok ? __ldg(p.label + row) : -1;
    ref2 = KIND == CE_GRAD && ok ? __ldcg(p.ref2 + row) : 0.0f;
  }
  __device__ __forceinline__ void chunk(const CeGemmParams& p, const uint32_t (&v)[32], int c) {
    ce_chunk<KIND, CAP>(p, v, first + c, row, ok, label, ref2, top, sum, zs, ws, ts);
  }
  __device__ __forceinline__ void store(const CeGemmParams& p, const CeUnit& U, int part) const {
    if (!ok) return;
    const long long at = (static_cast<long long>(U.tn) * kCeSlots + part) * p.ldp + row;
    if (KIND == CE_STATS) {
      p.part[at] = make_float2(top, sum);
    } else {
      p.psum[at] = sum;
      p.wsum[at] = ws;
      if (CAP) p.tsum[at] = ts;
    }
    if (p.zsum != nullptr) p.zsum[at] = zs;
  }
};

// The epilogue of one tile row, 32 columns at a time, each read from tensor memory while those before are
// worked on; release() once all have been read.  Warp-collective.
template <int KIND, bool CAP, typename F>
__device__ __forceinline__ void ce_rows(const CeGemmParams& p, const CeUnit& U, uint32_t tacc, int row, bool ok, int part,
                                        F&& release) {
  constexpr int kSpan = CeRow<KIND, CAP>::kSpan;
  const uint32_t from = tacc + part * kSpan;
  uint32_t va[32], vb[32];
  __syncwarp();
  tmem_ld32(from, va);
  CeRow<KIND, CAP> r(p, U, row, ok, part);
#pragma unroll 1
  for (int c = 0; c < kSpan; c += 64) {
    tmem_ld_wait_for(va);
    __syncwarp();
    tmem_ld32(from + c + 32, vb);
    r.chunk(p, va, c);
    tmem_ld_wait_for(vb);
    __syncwarp();
    if (c + 64 < kSpan) {
      tmem_ld32(from + c + 64, va);
    } else {
      release();
    }
    r.chunk(p, vb, c + 32);
  }
  r.store(p, U, part);
}

// The same for logits summed in parts, which have been joined in registers.
template <int KIND, bool CAP>
__device__ __forceinline__ void ce_rows_joined(const CeGemmParams& p, const CeUnit& U,
                                               const uint32_t (&z)[CeRow<KIND, CAP>::kSpan / 32][32], int row, bool ok, int part) {
  CeRow<KIND, CAP> r(p, U, row, ok, part);
#pragma unroll
  for (int c = 0; c < CeRow<KIND, CAP>::kSpan / 32; ++c) r.chunk(p, z[c], 32 * c);
  r.store(p, U, part);
}

// LONG: units of more than kb_range k-blocks.  A unit's parts take the two accumulators in turn, as units do otherwise.
template <int KIND, bool LONG>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(pair_threads(kCeWarps), 1)
    ce_gemm_kernel(const __grid_constant__ CeGemmParams p) {
  constexpr int STAGES = kCeStages;
  constexpr bool B_MN = KIND == CE_PART;
  using C = PairCfg<STAGES, kCeWarps>;
  constexpr int BN = C::BN;
  if (p.when_redo) {                      // the second try, seldom needed: leave before taking anything
    pdl_wait();
    if (__ldcg(&p.piece->redo) == 0) return;
  }
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * C::kStageBytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = static_cast<int>(blockIdx.x >> 1);
  const int npairs = static_cast<int>(gridDim.x >> 1);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 4);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 2 * kCeWarps);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&p.a);
    tma_prefetch_map(&p.b);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  cluster_sync_all();                     // both CTAs' barriers exist before any remote arrive
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();                             // the previous kernels' writes are visible from here
  pdl_launch_dependents();
  // every thread of the launch reads the same words: all roles walk the same units
  const int live = __ldcg(&p.piece->live);
  const int whole = KIND == CE_PART ? __ldcg(&p.piece->whole) : -1, splits = KIND == CE_PART ? __ldcg(&p.piece->splits) : 1;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int armed[STAGES];
      for (int s = 0; s < STAGES; ++s) armed[s] = -1;
      bool ok = true, first_stage = true;
      CeIter it(p, live, whole, splits, pair, npairs);
      CeUnit U;
      while (ok && it.next(p, U)) {
        const int a_row = U.tm * (2 * kBM) + static_cast<int>(rank) * kBM;
        const bool narrow = KIND == CE_PART && p.narrow && U.tn == p.tiles_n - 1;
        const int b_row = U.tn * BN + static_cast<int>(rank) * (narrow ? C::kBLocal / 2 : C::kBLocal);
        for (int j = U.kb0; j < U.kb1; ++j) {
          const int kc = j * kBK;
          if (!ce_wait(empty_bar(stage), phase ^ 1u, abort_flag, p)) { ok = false; break; }
          const uint32_t fb = full_bar(stage);
          if (p.inject_stall && first_stage && leader) {   // failure-path tests: never arm it
            first_stage = false;
            if (++stage == STAGES) { stage = 0; phase ^= 1u; }
            continue;
          }
          first_stage = false;
          if (leader) {
            mbar_arrive_expect_tx(fb, narrow ? C::kTxBytes - C::kBBytes : C::kTxBytes);
            armed[stage] = static_cast<int>(phase);
          }
          const uint32_t fb_even = mapa_shared(fb, 0);
          const uint32_t sa = sbase + stage * C::kStageBytes;
          const uint32_t sb = sa + C::kABytes;
          if (KIND == CE_PART) {
            tma_load_2d_pair(sa, &p.a, fb_even, 0, ((U.tm * 2 + static_cast<int>(rank)) * p.blocks + j) * kBM);
          } else {
            tma_load_2d_pair(sa, &p.a, fb_even, kc, a_row);
          }
          if (!B_MN) {
            tma_load_2d_pair(sb, &p.b, fb_even, kc, b_row);
          } else {
#pragma unroll
            for (int c = 0; c < C::kBLocal / 64; ++c)
              if (c == 0 || !narrow) tma_load_2d_pair(sb + c * 8192u, &p.b, fb_even, b_row + c * 64, kc);
          }
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok && leader) {
        for (int s = 0; s < STAGES; ++s)
          if (armed[s] >= 0) ce_wait_drain(full_bar(s), static_cast<uint32_t>(armed[s]), p);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (leader && lane == 0) {
      // kept lean as in the projections' kernel: descriptors are stage 0's plus constants, the
      // next stage is tested before this stage's last MMA
      constexpr uint32_t idesc_full = idesc_bf16_f32(2 * kBM, BN, 0, B_MN ? 1 : 0);
      constexpr uint32_t idesc_narrow = idesc_bf16_f32(2 * kBM, BN / 2, 0, B_MN ? 1 : 0);
      const uint64_t adesc0 = smem_desc_sw128(sbase, 16u, 1024u);
      const uint64_t bdesc0 = B_MN ? smem_desc_sw128(sbase + C::kABytes, 8192u, 1024u)
                                   : smem_desc_sw128(sbase + C::kABytes, 16u, 1024u);
      constexpr uint64_t kStageStep = C::kStageBytes >> 4;
      constexpr uint64_t kAStep = 32 >> 4;
      constexpr uint64_t kBStep = B_MN ? (2048 >> 4) : (32 >> 4);
      int stage = 0;
      uint32_t phase = 0;
      bool landed = false;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      CeIter it(p, live, whole, splits, pair, npairs);
      CeUnit U;
      int upto = 0;                                          // k-blocks of the tile that are done
      bool more = false;
      while (ok && (more || it.next(p, U))) {
        if (!ce_wait(tempty_bar(acc), acc_phase ^ 1u, abort_flag, p)) { ok = false; break; }
        tc_fence_after_sync();
        const int from = more ? upto : U.kb0;
        upto = LONG ? min(from + p.kb_range, U.kb1) : U.kb1;
        more = upto < U.kb1;
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
        const uint32_t idesc = KIND == CE_PART && p.narrow && U.tn == p.tiles_n - 1 ? idesc_narrow : idesc_full;
        uint32_t accumulate = 0;
        for (int j = from; j < upto; ++j) {
          const int kc = j * kBK;
          if (!landed && !ce_wait(full_bar(stage), phase, abort_flag, p)) { ok = false; break; }
          tc_fence_after_sync();
          const int nstage = stage + 1 == STAGES ? 0 : stage + 1;
          const uint32_t nphase = stage + 1 == STAGES ? phase ^ 1u : phase;
          const uint64_t ad = adesc0 + static_cast<uint64_t>(stage) * kStageStep;
          const uint64_t bd = bdesc0 + static_cast<uint64_t>(stage) * kStageStep;
          if (kc + kBK <= p.kvalid && accumulate) {
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k) {
              if (k == kBK / 16 - 1) landed = mbar_test_wait(full_bar(nstage), nphase);
              tc_mma_bf16_pair(d_tmem, ad + k * kAStep, bd + k * kBStep, idesc, 1u);
            }
          } else {
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k) {
              if (k == kBK / 16 - 1) landed = mbar_test_wait(full_bar(nstage), nphase);
              if (kc + 16 * k < p.kvalid) {
                tc_mma_bf16_pair(d_tmem, ad + k * kAStep, bd + k * kBStep, idesc, accumulate);
                accumulate = 1;
              }
            }
          }
          tc_commit_pair_multicast(empty_bar(stage), 0x3);   // frees this stage in both CTAs
          stage = nstage;
          phase = nphase;
        }
        if (!ok) break;
        tc_commit_pair_multicast(tfull_bar(acc), 0x3);       // both halves of the tile, or of its part, ready
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      }
      if (!ok) {
        tc_commit_pair_multicast(drain_bar, 0x1);
        ce_wait_drain(drain_bar, 0, p);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3;
    const int part = (warp - 2) >> 2;
    const int row_in_tile = static_cast<int>(rank) * kBM + q * 32 + lane;
    const uint32_t tempty_even[2] = {mapa_shared(tempty_bar(0), 0), mapa_shared(tempty_bar(1), 0)};
    if constexpr (KIND == CE_PART) {
      // the first tile is some time off: a warp a row, where the rows' factors were made before their weights
      if (p.balance == 1 || (p.balance == 2 && __ldcg(&p.piece->redo) != 0)) {
        const int step = static_cast<int>(gridDim.x) * kCeWarps;
        for (int row = static_cast<int>(blockIdx.x) * kCeWarps + warp - 2; row < live; row += step) {
          float t = 0.0f, w = 0.0f;
          for (int k = lane; k < p.slots; k += 32) {
            t += __ldcg(p.tsum + k * p.ldp + row);
            w += __ldcg(p.wsum + k * p.ldp + row);
          }
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) {
            t += __shfl_xor_sync(0xffffffffu, t, d);
            w += __shfl_xor_sync(0xffffffffu, w, d);
          }
          if (lane == 0) {
            float rs = __ldcg(p.rs + row), coef = __ldcg(p.coef + row);
            ce_balance(t, w, rs, coef);
            p.rs[row] = rs;
            p.coef[row] = coef;
          }
        }
        __syncwarp();
      }
    }
    int acc = 0;
    uint32_t acc_phase = 0;
    CeIter it(p, live, whole, splits, pair, npairs);
    CeUnit U;
    auto landed = [&]() {
      const bool ready = ce_wait(tfull_bar(acc), acc_phase, abort_flag, p);
      if (!__all_sync(0xffffffffu, ready)) return false;
      tc_fence_after_sync();
      return true;
    };
    while (it.next(p, U)) {
      if (!landed()) break;
      const int row = U.tm * (2 * kBM) + row_in_tile;
      uint32_t tacc = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * BN);
      // the accumulator has been read: the MMAs of the tile or part after next may overwrite it
      auto release = [&]() {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive_read(tempty_even[acc]);
      };
      if constexpr (KIND == CE_PART && !LONG) {
        constexpr int kSpan = BN / kCeSlots;
        float* dst = p.slab + (static_cast<long long>(U.u) * (2 * kBM) + row_in_tile) * BN;
#pragma unroll 1
        for (int c = part * kSpan; c < (part + 1) * kSpan && (c < BN / 2 || !p.narrow || U.tn < p.tiles_n - 1); c += 32) {
          uint32_t v[32];
          __syncwarp();
          tmem_ld32(tacc + c, v);
          tmem_ld_wait();
          if (row < live) {
#pragma unroll
            for (int j = 0; j < 32; j += 8) st_global_v8(dst + c + j, v + j);
          }
        }
        release();
      } else if constexpr (LONG) {
        constexpr int kSpan = BN / kCeSlots;
        uint32_t z[kSpan / 32][32];
        const bool wide = KIND != CE_PART || part == 0 || !p.narrow || U.tn < p.tiles_n - 1;   // the tile has the warp's columns
        // (zeros first: the first part as a case of its own spilled 1 KB of registers)
#pragma unroll
        for (int c = 0; c < kSpan; ++c) z[c / 32][c % 32] = 0u;
        bool ok = true;
        for (int kb = U.kb0; kb < U.kb1; kb += p.kb_range) {
          if (kb > U.kb0) {
            if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
            ok = landed();
            if (!ok) break;
            tacc = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * BN);
          }
#pragma unroll
          for (int c = 0; c < kSpan; c += 16) {
            if (!wide) break;
            uint32_t v[16];
            __syncwarp();
            tmem_ld16(tacc + part * kSpan + c, v);
            tmem_ld_wait_for(v);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              uint32_t& sum = z[c / 32][c % 32 + j];
              sum = __float_as_uint(__uint_as_float(sum) + __uint_as_float(v[j]));
            }
          }
          release();
        }
        if (!ok) break;
        if constexpr (KIND == CE_PART) {
          float* dst = p.slab + (static_cast<long long>(U.u) * (2 * kBM) + row_in_tile) * BN + part * kSpan;
          if (wide && row < live) {
#pragma unroll
            for (int c = 0; c < kSpan; c += 8) st_global_v8(dst + c, &z[c / 32][c % 32]);
          }
        } else if (p.lg.cap2 > 0.0f) {
          ce_rows_joined<KIND, true>(p, U, z, row, row < live, part);
        } else {
          ce_rows_joined<KIND, false>(p, U, z, row, row < live, part);
        }
      } else {
        if (p.lg.cap2 > 0.0f) {
          ce_rows<KIND, true>(p, U, tacc, row, row < live, part, release);
        } else {
          ce_rows<KIND, false>(p, U, tacc, row, row < live, part, release);
        }
      }
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
  }

  if (*abort_flag) settle_after_abort();
  __syncwarp();
  tc_fence_before_sync();
  cluster_sync_all();                     // no remote arrive or MMA read of either CTA is pending
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem_base, C::kTmemCols);
  }
}

// Defined in gemm_ce.cu.
cudaError_t launch_ce_gemm(int kind, const CeGemmParams& p, int grid, cudaStream_t st);

}  // namespace lgb
