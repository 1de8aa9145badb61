// Attention over the paged cache for many query rows per cache head (prefill chunks): the
// products run on the tcgen05 tensor cores.
//
// A CTA takes tiles of NQ x 128 packed query rows against KT positions.  Two row halves
// (NQ = 2) read each K and V tile once for 256 rows; one half serves batches of fewer rows,
// and head_dim 256, where the output alone fills half of the tensor memory.
//   S = Q K^T        operands in shared memory, S in tensor memory (two buffers)
//   P = 2^(c S - m)  one thread per row: maximum, exponential and sum without a shuffle;
//                    P replaces S in place, packed as bf16: each weight is rounded by at
//                    most 2^-8 of itself, as an output is, and the sum that divides them is
//                    the sum of the f32 weights.  (Two bf16 parts of a weight, as few rows
//                    carry them, bring the error against 64 bits from 0.0021 to the output
//                    rounding's own 0.0016; a first prefill of 4 x 2048 tokens then takes
//                    203 us instead of 145, 512 tokens over 16,000 263 instead of 207, heads
//                    of 256 5% more: not taken.)
//   O += P V         P from tensor memory, V from shared memory as it lies (MN-major)
// Roles: warp 0 fills a ring of K and V tiles by TMA (one box per page); warp 1 (and, with
// two halves, warp 2) issues the MMAs; warp 3 brings the next item's Q as soon as the last
// scores of this one are done; four warps per row half do the softmax.  The tensor cores
// work on one half's products while the other half's softmax runs (one issuing lane per
// half, so that one lane's barrier work hides behind the other's MMAs); with one half, on
// the next tile's scores.  An accumulator is rescaled, in tensor memory, only when a row's
// maximum rises by more than 2^8 (kMaxSlack).
//
// Bound by the tensor cores and, as much, by the softmax's instructions (an exponential, a
// maximum, two multiply-adds and half a conversion a score), which is why a row's scores stay
// in registers and rows need no shuffles.  Measured: a first prefill of 4 x 2048 tokens, 32
// query heads over 8 cache heads of 128 features, bf16: 145 us, 950 TFLOP/s of products
// needed (half of cuBLAS's rate); 512 new tokens of two sequences after 16,000: 198 us with a
// bf16 cache (1340 TFLOP/s, 70%), 305 us with fp8, where the ring has room for three
// converted tiles and converting sets the pace.
//
// 8-bit caches run in f16: four more warps turn the ring's raw tiles into f16 tiles once for
// all the tile's rows.  K tiles hold the codes, which f16 holds exactly, and a position's K
// scale multiplies its score in f32.  V tiles come in two kinds, told apart by the tile's
// largest and smallest V scale:
//   alike (within 2^6, nearly every tile)  a code times its row's scale over a power of two
//          2^eV that brings the largest scale to (1/2, 1], rounded to f16's 11 bits, eight
//          times finer than the bf16 rows that went into the cache; the weights are
//          2^(s + eV - r)
//   apart  the codes alone, exactly; a position's scale joins its weight as an exponent,
//          2^(s + log2 vs - r) (512 new tokens of two sequences over 16,000 fp8 positions:
//          305 us with every tile alike, 651 us with every tile apart)
// r is a row's own reference: the running maximum of s + eV (s + log2 vs) over what the row
// sees, so that neither a position of little weight nor a hidden one moves the other
// positions' weights out of f16's range, whatever the scales are.  It stands kBoost powers
// of two below the top of f16: a weight is rounded by 2^-11 of itself or, with the 2^6
// above, 2^-25 of the row's largest weight times scale.  The sums are relative to the scores'
// own maximum.  The softmax warps turn their rows of Q, scaled by a power of two to f16's
// upper range (exact for features down to 2^-29 of the row's largest).
#include <type_traits>

#include "paged_attn.cuh"
#include "codes.cuh"

namespace lgb {

template <int D_, int FMT_, int NQ_>
struct ManyCfg {
  static constexpr int D = D_, FMT = FMT_, NQ = NQ_;
  static constexpr bool kRaw = FMT != LORA_KV_BF16;
  static constexpr int R = 128 * NQ;
  static constexpr int KT = D == 256 ? 64 : 128;
  // An item's own cost, in tiles: measured 1, 2, 3, 4, 6 at 176, 167, 161, 163, 167 us for the
  // first prefill of 4 x 2048 tokens.
  static constexpr int kItem = 3;
  static constexpr int kHalves = D / 64;                     // 128-byte columns of a bf16 row
  static constexpr int kTile = KT * D * 2;                   // one bf16 K or V tile
  static constexpr int kQBytes = 128 * D * 2;                // one row half of Q
  static constexpr int kRawBox = D < 128 ? D : 128, kRawBoxes = D / kRawBox;
  static constexpr int kRawTile = kRaw ? KT * D : 0;
  static constexpr int kRawStages = kRaw ? 3 : 0;
  static constexpr int kStages = kRaw ? (D == 64 ? 6 : NQ == 1 && D == 128 ? 4 : 3) : (D == 64 ? 8 : D == 128 && NQ == 1 ? 6 : 5);
  static constexpr int kScaleSlots = (kStages + 2) / 2;      // see the converting warps
  static constexpr int kConvWarps = kRaw ? 4 : 0;
  static constexpr int kSoftWarps = 4 * NQ;
  static constexpr int kThreads = 32 * (4 + kSoftWarps + kConvWarps);
  // Registers a thread of each warpgroup: what the block starts with (kRegs each; the file
  // holds 65536), then shared out so that a softmax row's scores stay in registers.
  static constexpr int kRegs = kThreads == 256 ? 248 : kThreads == 384 ? 168 : 128;
  static constexpr bool kSplitRegs = kThreads > 256;
  static constexpr int kSupportRegs = kRaw && NQ == 2 ? 56 : 80;
  static constexpr int kSoftRegs = !kRaw ? 208 : NQ == 2 ? 192 : 240;
  static constexpr int kConvRegs = NQ == 2 ? 72 : 128;
  static_assert(!kSplitRegs || kSupportRegs + NQ * kSoftRegs + (kRaw ? kConvRegs : 0) <= kRegs * (kThreads / 128), "");
  static constexpr int kSCol0 = 0, kSCols = KT, kOCol0 = 256;
  static constexpr int kOffRing = NQ * kQBytes;
  static constexpr int kOffRaw = kOffRing + kStages * kTile;
  static constexpr int kOffRawScales = kOffRaw + kRawStages * kRawTile;
  static constexpr int kOffScales = kOffRawScales + (kRaw ? kRawStages * 2 * KT * 4 : 0);
  // (a slot: the tile's KT K scales, eV or kApart, the V scales or, apart, their log2)
  static constexpr int kSlotBytes = 2 * KT * 4 + 16;
  static constexpr int kOffBars = (kOffScales + (kRaw ? kScaleSlots * kSlotBytes : 0) + 127) & ~127;
  static constexpr int kNumBars = 2 * kStages + 2 * kRawStages + 6 + 5 * NQ + (kRaw ? kScaleSlots + NQ : 0);
  static constexpr int kOffPlan = kOffBars + kNumBars * 8 + 8;
  static constexpr int kSmem = kOffPlan + static_cast<int>(sizeof(PlanScratch<kThreads>)) + 1024;
  static_assert(kSmem <= 232448, "shared memory of one CTA");
  static_assert(kOffPlan % 8 == 0, "alignment");
};

// D[tmem] (+)= A[tmem, packed bf16] * B[smem]^T, f32 sums.
__device__ __forceinline__ void tc_mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 2^e of a normal exponent.
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float(static_cast<unsigned>(127 + e) << 23); }
// A tile's V scales, from the bits of the smallest and the largest: alike if the largest is at
// most 2^6 times the smallest, finite and below 2^126 (a NaN's bits are above every number's;
// no position at all: 0 and ~0), and at most 2^80 times below `most`, the largest eV of the
// part's tiles before: a row's weights, of which its sum takes part, then stay inside f32.
// eV of a largest scale: 2^(eV - 1) <= x < 2^eV (subnormal ones less).
__device__ __forceinline__ int scale_exponent(unsigned bits) { return max(-125, static_cast<int>(bits >> 23) - 126); }
__device__ __forceinline__ bool scales_alike(unsigned small, unsigned big, int most) {
  return big < 0x7E800000u && (big == 0 || small + (6u << 23) >= big) && scale_exponent(big) >= most - 80;
}
constexpr int kApart = 1000;         // stands for eV where the scales are apart
constexpr float kBoost = 7.0f;       // f16 weights are at most 2^(kBoost + kMaxSlack) = 2^15

// Row halves of an item that hold rows of the sequence.
template <class C>
__device__ __forceinline__ int halves_of(const AttnParams& p, const Span& w) {
  return C::NQ == 2 && w.s.n - w.rt * p.tt > p.th ? 2 : 1;
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1) attn_many_kernel(const __grid_constant__ AttnParams p) {
  constexpr int D = C::D, KT = C::KT, R = C::R, ST = C::kStages, RS = C::kRawStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem), ring = sbase + C::kOffRing;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto& scratch = *reinterpret_cast<PlanScratch<C::kThreads>*>(smem + C::kOffPlan);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };                          // a 16-bit tile is in the ring
  auto empty_bar = [&](int s) { return bar0 + 8u * (ST + s); };
  auto rfull_bar = [&](int s) { return bar0 + 8u * (2 * ST + s); };              // a raw tile
  auto rempty_bar = [&](int s) { return bar0 + 8u * (2 * ST + RS + s); };
  constexpr int kB = 2 * ST + 2 * RS;
  // score buffer b: half b's with two halves, tile b modulo 2 with one
  auto sfull_bar = [&](int b) { return bar0 + 8u * (kB + b); };                  // scores ready
  // weights of the tile's first (h = 0) and second KT / 2 positions ready
  auto pready_bar = [&](int b, int h) { return bar0 + 8u * (kB + 2 + 2 * h + b); };
  auto odone_bar = [&](int q) { return bar0 + 8u * (kB + 6 + q); };              // a half's O += P V is done
  auto qready_bar = [&](int q) { return bar0 + 8u * (kB + 6 + C::NQ + q); };     // a half's Q is in place
  auto qfree_bar = [&](int q) { return bar0 + 8u * (kB + 6 + 2 * C::NQ + q); };  // its last scores are done
  auto drain_bar = [&](int q) { return bar0 + 8u * (kB + 6 + 3 * C::NQ + q); };
  auto scale_bar = [&](int s) { return bar0 + 8u * (kB + 6 + 5 * C::NQ + s); };  // a tile's scales are in slot s
  auto qraw_bar = [&](int q) { return bar0 + 8u * (kB + 6 + 5 * C::NQ + C::kScaleSlots + q); };   // 8-bit: Q as bf16
  auto turn_bar = [&](int q) { return bar0 + 8u * (kB + 6 + 4 * C::NQ + q); };   // half q's lane may issue
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(full_bar(s), C::kRaw ? C::kConvWarps : 1);
      mbar_init(empty_bar(s), C::NQ);
    }
    for (int s = 0; s < RS; ++s) {
      mbar_init(rfull_bar(s), 1);
      mbar_init(rempty_bar(s), C::kConvWarps);
    }
    if (C::kRaw)
      for (int s = 0; s < C::kScaleSlots; ++s) mbar_init(scale_bar(s), C::kConvWarps);
    for (int b = 0; b < 2; ++b) {
      mbar_init(sfull_bar(b), 1);
      mbar_init(pready_bar(b, 0), 4);
      mbar_init(pready_bar(b, 1), 4);
    }
    for (int q = 0; q < C::NQ; ++q) {
      mbar_init(odone_bar(q), 1);
      mbar_init(qready_bar(q), C::kRaw ? 4 : 1);
      if (C::kRaw) mbar_init(qraw_bar(q), 1);
      mbar_init(qfree_bar(q), 1);
      mbar_init(drain_bar(q), 1);
      mbar_init(turn_bar(q), 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_map(&p.kmap);
    tma_prefetch_map(&p.vmap);
    tma_prefetch_map(&p.qmap);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_launch_dependents();
  make_plan<KT, C::kItem, C::kThreads>(p, scratch);
  const Plan plan = scratch.plan;
  Walker<KT, C::kItem> walk(p, plan);
  Span w;
  // (each warpgroup sets its registers at the head of its own branch: the compiler then
  // allocates that branch by the new count)
  if (warp < 4) {
  if constexpr (C::kSplitRegs) regs_lower<C::kSupportRegs>();
  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    const int ps = 1 << p.cache.page_shift;
    const int box_rows = ps < KT ? ps : KT, boxes = KT / box_rows;
    constexpr int NS = C::kRaw ? RS : ST;
    constexpr int kEl = C::kRaw ? 1 : 2, kBox = C::kRaw ? C::kRawBox : 128, kBoxes = C::kRaw ? C::kRawBoxes : C::kHalves;
    constexpr int kDstTile = C::kRaw ? C::kRawTile : C::kTile;
    const uint32_t dst0 = C::kRaw ? sbase + C::kOffRaw : ring;
    auto fbar = [&](int s) { return C::kRaw ? rfull_bar(s) : full_bar(s); };
    auto ebar = [&](int s) { return C::kRaw ? rempty_bar(s) : empty_bar(s); };
    int stage = 0, armed = 0;
    uint32_t phase = 0;
    bool ok = true, first = true;
    while (ok && walk.next(p, w)) {
      const int kvh = w.slice / p.spg;
      const int* row = p.table + static_cast<long long>(w.b) * p.max_pages;
      const int pages = (w.s.kv + ps - 1) >> p.cache.page_shift;
      const int low = lowest_seen(p, w);
      int held = -64, page = 0;           // lane l holds the table's entry held + l
      for (int j = w.ja; ok && j < w.jb; ++j) {
        const int at = (j * KT) >> p.cache.page_shift;
        if (at + boxes > held + 32) {
          held = at;
          page = 0;
          if (at + lane < pages && at + lane >= low >> p.cache.page_shift) {
            page = __ldg(row + at + lane);
            if (page < 0 || page >= p.cache.n_pages) {
              atomicOr(p.status, kStatusInput);
              page = 0;
            }
          }
        }
        const int mine = __shfl_sync(0xffffffffu, page, at - held + (lane < boxes ? lane : 0));
        const int left = w.s.kv - j * KT;
        const int live = left <= 0 ? 0 : min(boxes, (left + box_rows - 1) / box_rows);
        const int skip = max(0, low - j * KT) / box_rows;      // boxes that no row sees, below `live`
        const int r0 = lane * box_rows;
        const long long src = lane < skip ? -box_rows
                                          : ((static_cast<long long>(mine) * p.cache.heads + kvh) << p.cache.page_shift) +
                                                ((j * KT + r0) & (ps - 1));
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {  // the K tile, then the V tile
          ok = attn_wait(ebar(stage), phase ^ 1u, abort_flag, p);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint32_t fb = fbar(stage);
          if (p.inject_stall && first) {  // failure-path tests: leave this stage empty
            first = false;
          } else {
            first = false;
            if (lane == 0) {
              if (live > 0)
                mbar_arrive_expect_tx(fb, box_rows * (live * static_cast<uint32_t>(D * kEl) + (C::kRaw && kv == 0 ? (live - skip) * 8u : 0u)));
              else
                mbar_arrive(fb);
            }
            __syncwarp();
            if (lane < live) {
              const uint32_t dst = dst0 + stage * kDstTile + r0 * kBox;
#pragma unroll
              for (int x = 0; x < kBoxes; ++x)
                tma_load_2d(dst + x * (KT * kBox), kv ? &p.vmap : &p.kmap, fb, x * (kBox / kEl), static_cast<int>(src));
              if (C::kRaw && kv == 0 && lane >= skip) {   // the K tile brings both tiles' scales
                const uint32_t sc = sbase + C::kOffRawScales + stage * (2 * KT * 4) + r0 * 4;
                bulk_load(sc, p.cache.ks + src, box_rows * 4, fb);
                bulk_load(sc + KT * 4, p.cache.vs + src, box_rows * 4, fb);
              }
            }
          }
          ++armed;
          if (++stage == NS) { stage = 0; phase ^= 1u; }
        }
      }
    }
    if (!ok) {
      for (int f = armed > NS ? armed - NS : (p.inject_stall ? 1 : 0); f < armed; ++f)
        attn_wait_drain(fbar(f % NS), (f / NS) & 1, p);
    }
  } else if (warp <= C::NQ) {
    // ------------------------------------------------------------ MMA issuers, one warp per half
    // The whole warp walks the loop, converged, and one elected lane issues: the operands
    // then stay in uniform registers (an MMA of 128 x 128 x 16 lasts 64 cycles, and issuing
    // it from a diverged lane took longer).
    {
      const int q = __shfl_sync(0xffffffffu, warp - 1, 0);
      // (f16 operands: the format fields of A and B, bits 7 and 10, are 0)
      constexpr uint32_t kTypes = C::kRaw ? ~((1u << 7) | (1u << 10)) : ~0u;
      constexpr uint32_t idesc_o = idesc_bf16_f32(128, D, 0, 1) & kTypes;
      // a negative scale negates Q as it is read (bit 13)
      const uint32_t idesc_s = (idesc_bf16_f32(128, KT, 0, 0) & kTypes) | (p.scale_log2 < 0.0f ? 1u << 13 : 0u);
      const uint64_t qdesc = smem_desc_sw128(sbase + q * C::kQBytes, 16u, 1024u);
      const uint64_t kdesc0 = smem_desc_sw128(ring, 16u, 1024u);
      const uint64_t vdesc0 = smem_desc_sw128(ring, KT * 128u, 1024u);
      constexpr uint64_t kTileStep = C::kTile >> 4;
      const uint32_t o_tmem = tmem + C::kOCol0 + q * D;
      auto commit = [&](uint32_t bar) { if (elect_one()) tc_commit(bar); };
      auto arrive = [&](uint32_t bar) { if (elect_one()) mbar_arrive(bar); };
      auto wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, attn_wait(bar, parity, abort_flag, p)) != 0;
      };
      auto next_item = [&]() {          // the walk's values, as uniform ones
        if (!__shfl_sync(0xffffffffu, static_cast<int>(walk.next(p, w)), 0)) return false;
        w.ja = __shfl_sync(0xffffffffu, w.ja, 0);
        w.jb = __shfl_sync(0xffffffffu, w.jb, 0);
        return true;
      };
      auto scores = [&](int st, int buf) {
        const uint32_t d = tmem + C::kSCol0 + buf * C::kSCols;
        const uint64_t b = kdesc0 + st * kTileStep;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tc_mma_bf16(d, qdesc + (k >> 2) * (128 * 128 >> 4) + (k & 3) * 2, b + (k >> 2) * (KT * 128 >> 4) + (k & 3) * 2,
                        idesc_s, k > 0 ? 1u : 0u);
        }
      };
      // O += P V: all at once if the weights are there, else each half of the positions as
      // soon as its weights are
      auto values = [&](int st, int buf, uint32_t phase, bool first) {
        const uint32_t a = tmem + C::kSCol0 + buf * C::kSCols;
        const uint64_t b = vdesc0 + st * kTileStep;
        bool all = __all_sync(0xffffffffu, mbar_test_wait(pready_bar(buf, 1), phase));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!all && !wait(pready_bar(buf, h), phase)) return false;
          if (h == 0 || !all) tc_fence_after_sync();
          if (elect_one()) {
#pragma unroll
            for (int k = h * (KT / 32); k < (h + 1) * (KT / 32); ++k)
              tc_mma_bf16_ts(o_tmem, a + 8 * k, b + k * (2048 >> 4), idesc_o, (k > 0 || !first) ? 1u : 0u);
          }
        }
        return true;
      };
      int st = 0;                         // ring stage and its phase
      uint32_t ph = 0, qphase = 0, pphase = 0;
      auto step = [&](int& s, uint32_t& f) { if (++s == ST) { s = 0; f ^= 1u; } };
      bool ok = true;
      if constexpr (C::NQ == 2) {
        // Turns: O += P V of a tile and the scores of the next go out together, half 0's and
        // half 1's in alternation, so that one half's softmax always has the other half's
        // MMAs to run beside (left to themselves the halves fall into step: both wait for
        // the tensor cores, then both for the exponentials; 10% slower).
        uint32_t tphase = q == 0 ? 1u : 0u;        // half 0 has the first turn
        while (ok && next_item()) {
          const int nq = __shfl_sync(0xffffffffu, halves_of<C>(p, w), 0);
          const bool mine = q < nq, both = nq == 2;
          auto take_turn = [&]() {
            if (!both) return true;
            const bool got = wait(turn_bar(q), tphase);
            tphase ^= 1u;
            return got;
          };
          if (mine) {
            ok = wait(qready_bar(q), qphase);
            qphase ^= 1u;
          }
          // step j: O += P V of tile j - 1, then the scores of tile j
          for (int j = w.ja; ok && j <= w.jb; ++j) {
            const bool pv = j > w.ja, s = j < w.jb;
            const int vst = st;
            if (pv) {
              ok = wait(full_bar(vst), ph);
              step(st, ph);
            }
            if (ok && s) ok = wait(full_bar(st), ph);
            if (ok) ok = take_turn();
            if (!ok) break;
            if (!mine) {                           // every warp follows the ring's phases
              if (pv) arrive(empty_bar(vst));
              if (s) {
                arrive(empty_bar(st));
                step(st, ph);
              }
              continue;
            }
            if (pv) {
              ok = values(vst, q, pphase, j == w.ja + 1);
              if (!ok) break;
              pphase ^= 1u;
            } else {
              tc_fence_after_sync();
            }
            // the other half's warp wakes while these scores are issued
            if (both) arrive(turn_bar(q ^ 1));
            if (s) {
              scores(st, q);
              commit(sfull_bar(q));
            }
            if (pv) {
              commit(odone_bar(q));
              commit(empty_bar(vst));
            }
            if (s) {
              commit(empty_bar(st));
              if (j + 1 == w.jb) commit(qfree_bar(q));
              step(st, ph);
            }
          }
        }
      } else {
        // The scores of tile t + 1 are issued before tile t's O += P V.  So are the next item's
        // first ones with a bf16 cache; with an 8-bit one its Q is turned to f16 by the softmax
        // warps, which come to it only after this item's last O += P V.
        uint32_t T = 0;                   // tiles so far: score buffer T & 1
        auto next_scores = [&](bool new_item, bool last) {
          if (new_item) {
            if (!wait(qready_bar(0), qphase)) return false;
            qphase ^= 1u;
          }
          if (!wait(full_bar(st), ph)) return false;
          tc_fence_after_sync();
          scores(st, T & 1u);
          commit(sfull_bar(T & 1u));
          commit(empty_bar(st));
          if (last) commit(qfree_bar(0));
          ++T;
          step(st, ph);
          return true;
        };
        // ring order: K of tile t + 1 stands after V of tile t, so V's stage is remembered
        bool more = next_item();
        int j = more ? w.ja : 0;
        if (more) ok = next_scores(true, w.ja + 1 == w.jb);
        while (ok && more) {
          const bool first = j == w.ja;
          const int vst = st;
          const uint32_t vph = ph, buf = (T - 1u) & 1u;
          step(st, ph);
          bool fresh = false;
          if (++j == w.jb) {
            more = next_item();
            if (more) {
              j = w.ja;
              fresh = true;
              if (!C::kRaw) ok = next_scores(true, w.ja + 1 == w.jb);
            }
          } else {
            ok = next_scores(false, j + 1 == w.jb);
          }
          if (ok) ok = wait(full_bar(vst), vph);
          if (ok) ok = values(vst, buf, (pphase >> buf) & 1u, first);
          if (!ok) break;
          pphase ^= 1u << buf;
          commit(odone_bar(0));
          commit(empty_bar(vst));
          if (C::kRaw && fresh) ok = next_scores(true, w.ja + 1 == w.jb);
        }
      }
      if (!ok) {
        commit(drain_bar(q));
        attn_wait_drain(drain_bar(q), 0, p);
      }
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ Q loader
    // One box of th tokens x hs heads for 64 features: the packed rows in order, K-major with
    // the 128-byte swizzle.  Rows past the box, the sequence or the slice hold other data
    // and are nobody's.
    if (lane == 0) {
      uint32_t used[2] = {0, 0};          // items of each half so far
      bool ok = true;
      auto qbar = [&](int q) { return C::kRaw ? qraw_bar(q) : qready_bar(q); };
      while (ok && walk.next(p, w)) {
        const int nq = halves_of<C>(p, w), kvh = w.slice / p.spg;
        const int head = kvh * p.group + (w.slice - kvh * p.spg) * p.hs;
#pragma unroll 1
        for (int q = 0; q < nq; ++q) {
          if (used[q] > 0) ok = attn_wait(qfree_bar(q), (used[q] - 1u) & 1u, abort_flag, p);
          if (!ok) break;
          ++used[q];
          mbar_arrive_expect_tx(qbar(q), static_cast<uint32_t>(p.th * p.hs * D * 2));
#pragma unroll
          for (int x = 0; x < C::kHalves; ++x)
            tma_load_3d(sbase + q * C::kQBytes + x * (128 * 128), &p.qmap, qbar(q), 64 * x, head,
                        w.s.q0 + w.rt * p.tt + q * p.th);
        }
      }
      if (!ok)                            // copies in flight land before the block ends
        for (int q = 0; q < C::NQ; ++q)
          if (used[q] > 0) attn_wait_drain(qbar(q), (used[q] - 1u) & 1u, p);
    }
  }
  } else if (warp < 4 + C::kSoftWarps) {
    if constexpr (C::kSplitRegs) regs_raise<C::kSoftRegs>();
    // ------------------------------------------------------------ softmax
    const int q = (warp - 4) >> 2;                // row half
    const int quarter = warp & 3;                 // TMEM lanes of this warp
    const int r = quarter * 32 + lane;            // row of the half
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t o_tmem = tmem + lanes + C::kOCol0 + q * D;
    // (a scale of 0 becomes the smallest normal one: finite scores weigh the same, and a
    // hidden score stays -inf)
    const float scale = fmaxf(fabsf(p.scale_log2), 1.17549435e-38f);
    float c = scale;
    uint32_t qphase = 0;
    const bool out_v8 = rows_v8_aligned(p.out, 16);
    uint32_t T = 0, tile = 0;                     // position tiles, ring tiles before this item
    uint32_t done = 0;                            // O += P V steps of this half so far
    uint32_t sphase = 0;                          // bit b: phase of score buffer b
    bool ok = true;
    while (ok && walk.next(p, w)) {
      const int nq = halves_of<C>(p, w), n = w.jb - w.ja;
      if (q >= nq) {
        T += n;
        tile += 2u * n;
        continue;
      }
      int tok, head, lo, hi;
      const bool own = row_owner(p, w.s, w.slice, w.rt, q, r, tok, head);
      if (own) row_range(p, w.s, tok, lo, hi); else lo = 0, hi = 0x7fffffff;
      const int lo_max = __reduce_max_sync(0xffffffffu, lo), hi_min = __reduce_min_sync(0xffffffffu, hi);
      if constexpr (C::kRaw) {
        ok = attn_wait(qraw_bar(q), qphase, abort_flag, p);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        qphase ^= 1u;
        const uint32_t line = sbase + q * C::kQBytes + r * 128;
        auto piece = [&](int e) { return line + (e >> 3) * (128 * 128) + (((e & 7) ^ (r & 7)) << 4); };
        unsigned big = 0;
#pragma unroll 8
        for (int e = 0; e < D / 8; ++e) {
          const uint4 v = ld_shared_v4(piece(e));
          big = max(max(big, max(v.x & 0x7FFFu, (v.x >> 16) & 0x7FFFu)), max(v.y & 0x7FFFu, (v.y >> 16) & 0x7FFFu));
          big = max(max(big, max(v.z & 0x7FFFu, (v.z >> 16) & 0x7FFFu)), max(v.w & 0x7FFFu, (v.w >> 16) & 0x7FFFu));
        }
        // the row times 2^(14 - exponent of its largest), and the score scale without it
        const float f = __uint_as_float(static_cast<unsigned>(min(254, 268 - static_cast<int>(big >> 7))) << 23);
        c = fmaxf(scale / f, 1.17549435e-38f);
        auto turn2 = [&](uint32_t u) { return pack_f16x2(__uint_as_float(u << 16) * f, __uint_as_float(u & 0xFFFF0000u) * f); };
#pragma unroll 4
        for (int e = 0; e < D / 8; ++e) {
          const uint4 v = ld_shared_v4(piece(e));
          st_shared_v4(piece(e), make_uint4(turn2(v.x), turn2(v.y), turn2(v.z), turn2(v.w)));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(qready_bar(q));
      }
      // top: the row's running maximum (scaled, log2), which the sums are relative to; ref: what
      // the weights are relative to (8-bit: the maximum with the V scales; bf16: top itself)
      float top = -INFINITY, vtop = -INFINITY;
      float& ref = C::kRaw ? vtop : top;
      float2 sum = make_float2(0.0f, 0.0f);          // two partial sums
      for (int i = 0; i < n; ++i) {
        const uint32_t buf = C::NQ == 2 ? q : (T + i) & 1u;
        const int k0 = (w.ja + i) * KT;
        const uint32_t s_tmem = tmem + lanes + C::kSCol0 + buf * C::kSCols;
        const uint32_t vidx = tile + 2u * i + 1u;
        int ev = 0;                               // 8-bit: exponent of the tile's V scales, or kApart
        const float* ks = nullptr;                // and its K scales
        ok = attn_wait(sfull_bar(buf), (sphase >> buf) & 1u, abort_flag, p);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        sphase ^= 1u << buf;
        if (C::kRaw) {
          const uint32_t sc = (vidx >> 1) % C::kScaleSlots;
          ok = attn_wait(scale_bar(sc), ((vidx >> 1) / C::kScaleSlots) & 1u, abort_flag, p);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          ks = reinterpret_cast<const float*>(smem + C::kOffScales + sc * C::kSlotBytes);
          ev = __float_as_int(ks[KT]);
        }
        tc_fence_after_sync();
        const bool edge = k0 < lo_max || k0 + KT > hi_min;
        // Raises the row's maxima to a tile's where one exceeds them by more than the slack.
        auto raise = [&](float cand, float vcand) {
          // (rows that are nobody's hold any numbers: they have no say)
          if (!__any_sync(0xffffffffu, own && (cand > top + kMaxSlack || (C::kRaw && vcand > ref + kMaxSlack)))) return true;
          const float next = fmaxf(top, cand), vnext = C::kRaw ? fmaxf(ref, vcand) : next;
          const float f = vnext == -INFINITY ? 1.0f : exp2_approx(ref - vnext);
          const float fs = !C::kRaw ? f : next == -INFINITY ? 1.0f : exp2_approx(top - next);
          ref = vnext;
          top = next;
          sum.x *= fs;
          sum.y *= fs;
          if (i == 0) return true;
          ok = attn_wait(odone_bar(q), (done - 1u) & 1u, abort_flag, p);
          if (!__all_sync(0xffffffffu, ok)) return false;
          tc_fence_after_sync();
#pragma unroll 1
          for (int x = 0; x < D; x += 16) {
            uint32_t v[16];
            tmem_ld16(o_tmem + x, v);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
            tmem_st16(o_tmem + x, v);
          }
          tmem_st_wait();
          return true;
        };
        // Half of a tile's weights are handed over while the other half is made.
        auto hand_over = [&](int half) {
          tmem_st_wait();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(pready_bar(buf, half));
        };
        // With one half the last scores do not wait for the O += P V before theirs; it has to be
        // seen done before these weights go out, or the wait for the last one below could take
        // its phase for the one before.
        auto last_but_one_done = [&]() {
          if (C::NQ != 1 || i == 0 || i + 1 != n) return true;
          ok = attn_wait(odone_bar(q), (done - 1u) & 1u, abort_flag, p);
          return __all_sync(0xffffffffu, ok) != 0;
        };
        // compiled for tiles that all of the warp's rows see whole (nearly all), and for the others
        auto softmax = [&](auto at_edge) {
        constexpr bool kEdge = decltype(at_edge)::value;
        // the row's scores, read once and held in registers, 32 columns on their way while the
        // 32 before are worked on
        uint32_t v[KT / 32][32];
        // scores of columns [x, x + 32): K scales, mask
        auto finish = [&](uint32_t (&v)[32], int x) {
          if (C::kRaw) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 f = *reinterpret_cast<const float4*>(ks + x + e);
              const float2 a = mul_f32x2(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), make_float2(f.x, f.y));
              const float2 b = mul_f32x2(make_float2(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])), make_float2(f.z, f.w));
              v[e] = __float_as_uint(a.x), v[e + 1] = __float_as_uint(a.y);
              v[e + 2] = __float_as_uint(b.x), v[e + 3] = __float_as_uint(b.y);
            }
          }
          if (kEdge) {
            const int key = k0 + x;
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = key + e >= lo && key + e < hi ? v[e] : 0xFF800000u;   // -inf
          }
        };
        float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        auto maxima = [&](const uint32_t (&v)[32]) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              m[k] = fmaxf(fmaxf(m[k], __uint_as_float(v[e + 2 * k])), __uint_as_float(v[e + 2 * k + 1]));
          }
        };
        tmem_ld32(s_tmem, v[0]);
#pragma unroll
        for (int x = 0; x < KT / 32; ++x) {
          tmem_ld_wait_for(v[x]);
          if (x + 1 < KT / 32) tmem_ld32(s_tmem + 32 * (x + 1), v[x + 1]);
          finish(v[x], 32 * x);
          maxima(v[x]);
        }
        const float cand = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * c;
        if (!raise(cand, cand + ev)) return false;
        const float base = ref == -INFINITY ? 0.0f : C::kRaw ? kBoost + ev - ref : -ref;
        const float2 c2 = make_float2(c, c), ref2 = make_float2(base, base);
        float2 l[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        auto weights = [&](const uint32_t (&v)[32], int x) {
          uint32_t u[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float2 y[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              y[k] = fma_f32x2(make_float2(__uint_as_float(v[e + 2 * k]), __uint_as_float(v[e + 2 * k + 1])), c2, ref2);
              y[k].x = exp2_approx(y[k].x);
              y[k].y = exp2_approx(y[k].y);
              l[k] = add_f32x2(l[k], y[k]);
            }
            u[e / 2] = C::kRaw ? pack_f16x2(y[0].x, y[0].y) : pack_bf16x2(y[0].x, y[0].y);
            u[e / 2 + 1] = C::kRaw ? pack_f16x2(y[1].x, y[1].y) : pack_bf16x2(y[1].x, y[1].y);
          }
          tmem_st16(s_tmem + x / 2, u);
        };
        if (!C::kRaw && k0 + KT > w.s.kv) {
          // rows of V past the sequence hold anything, and zero weights do not silence a
          // NaN: they are cleared before the first weights are handed over (both halves'
          // warps may, with the same zeros)
          ok = attn_wait(full_bar(vidx % ST), (vidx / ST) & 1u, abort_flag, p);
          if (!__all_sync(0xffffffffu, ok)) return false;
          const uint32_t vt = ring + (vidx % ST) * C::kTile;
          for (int row = max(w.s.kv - k0, 0) + quarter; row < KT; row += 4)
            for (int e = lane; e < D / 8; e += 32)
              st_shared_v4(vt + (e >> 3) * (KT * 128) + row * 128 + ((e & 7) << 4), make_uint4(0, 0, 0, 0));
          fence_proxy_async_smem();
        }
#pragma unroll
        for (int x = 0; x < KT / 32; ++x) {
          weights(v[x], 32 * x);
          if (x == KT / 32 - 1 && !last_but_one_done()) return false;
          if (x == KT / 64 - 1) hand_over(0);
          if (x == KT / 32 - 1) hand_over(1);
        }
        l[0] = add_f32x2(l[0], l[1]);
        if (C::kRaw && top != -INFINITY) {     // from the weights' reference to the sums'
          const float f = exp2_approx(-base - top);
          l[0] = mul_f32x2(l[0], make_float2(f, f));
        }
        sum = add_f32x2(sum, l[0]);
        return true;
        };
        // The same with an exponent per position (8-bit), in two passes over the scores: such
        // tiles are few, and the code stays small and out of the others' registers.
        auto softmax_apart = [&]() {
          // the scores of columns [x, x + 32), and the exponents of columns e to e + 3
          auto scores_at = [&](int x, uint32_t (&v)[32]) {
            __syncwarp();
            tmem_ld32(s_tmem + x, v);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              v[e] = k0 + x + e >= lo && k0 + x + e < hi ? __float_as_uint(__uint_as_float(v[e]) * ks[x + e]) : 0xFF800000u;
          };
          auto exponents_at = [&](int e, float (&g)[4]) {
            const float4 f = *reinterpret_cast<const float4*>(ks + KT + 4 + e);
            g[0] = f.x, g[1] = f.y, g[2] = f.z, g[3] = f.w;
          };
          float most = -INFINITY, vmost = -INFINITY;
#pragma unroll 1
          for (int x = 0; x < KT; x += 32) {
            uint32_t v[32];
            scores_at(x, v);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              float g[4];
              exponents_at(x + e, g);
#pragma unroll
              for (int d = 0; d < 4; ++d) {
                most = fmaxf(most, __uint_as_float(v[e + d]));
                vmost = fmaxf(vmost, fmaf(__uint_as_float(v[e + d]), c, g[d]));
              }
            }
          }
          if (!raise(most * c, vmost)) return false;
          const float base = ref == -INFINITY ? 0.0f : kBoost - ref, seen = top == -INFINITY ? 0.0f : -top;
          // (a pass's weights stand where scores of the passes before stood)
#pragma unroll 1
          for (int x = 0; x < KT; x += 32) {
            uint32_t v[32], u[16];
            scores_at(x, v);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              float g[4], y[4];
              exponents_at(x + e, g);
#pragma unroll
              for (int d = 0; d < 4; ++d) {
                const float s = __uint_as_float(v[e + d]);
                // (a hidden position's scale, which may be a NaN, is not looked at)
                y[d] = s == -INFINITY ? 0.0f : exp2_approx(fmaf(s, c, g[d] + base));
                (d % 2 ? sum.y : sum.x) += exp2_approx(fmaf(s, c, seen));
              }
              u[e / 2] = pack_f16x2(y[0], y[1]);
              u[e / 2 + 1] = pack_f16x2(y[2], y[3]);
            }
            tmem_st16(s_tmem + x / 2, u);
            if (x == KT - 32 && !last_but_one_done()) return false;
            if (x == KT / 2 - 32) hand_over(0);
            if (x == KT - 32) hand_over(1);
          }
          return true;
        };
        if (C::kRaw && ev == kApart)
          ok = softmax_apart();
        else
          ok = edge ? softmax(std::true_type{}) : softmax(std::false_type{});
        if (!ok) break;
        ++done;
      }
      T += n;
      tile += 2u * n;
      if (!ok) break;
      ok = attn_wait(odone_bar(q), (done - 1u) & 1u, abort_flag, p);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      tc_fence_after_sync();
      const bool whole = w.starts && w.ends;
      const long long slot = 2ll * blockIdx.x + (w.starts ? 1 : 0);
      const float all = sum.x + sum.y;
      const bool none = top == -INFINITY && all == 0.0f;
      const float inv = none ? 0.0f : 1.0f / all;
      // 8-bit: the output from the weights' reference to the sums', 2^(ref - top - kBoost), in two
      // factors, which stay in f32's range together with what they multiply
      const float back = !C::kRaw ? 1.0f : ref == -INFINITY ? 0.0f : exp2_approx(0.5f * (ref - top - kBoost));
      const int orow = own ? (w.s.q0 + tok) * p.hq + head : -1;       // below 2^31
      const long long prow = slot * R + q * 128 + r;
      // A thread writes its row's whole sectors straight away.  (Rows through shared memory, so
      // that a store touches whole lines of few rows, write faster; but the room is worth more
      // as a ring stage: first prefill of 4 x 2048 tokens 150 us against 167 us.)
#pragma unroll 1
      for (int x = 0; x < D; x += 32) {
        uint32_t v[32];
        __syncwarp();
        tmem_ld32(o_tmem + x, v);
        tmem_ld_wait();
        if (!own) continue;
        if (C::kRaw) {
          const float first = whole ? inv * back : back;
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * first * back);
        }
        if (whole) {
          uint32_t u[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            u[e] = none ? 0u : C::kRaw ? pack_bf16x2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]))
                                       : pack_bf16x2(__uint_as_float(v[2 * e]) * inv, __uint_as_float(v[2 * e + 1]) * inv);
          store_row32_bf16(p.out + static_cast<long long>(orow) * D + x, u, 0, 32, out_v8);
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 8) st_global_v8(p.part_o + prow * D + x + e, v + e);
        }
      }
      if (own) {
        if (!whole)
          p.part_ml[prow] = make_float2(top, all);
        else if (p.lse != nullptr)
          p.lse[orow] = none ? -INFINITY : (top + log2f(all)) * 0.6931471805599453f;
      }
      tc_fence_before_sync();
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ converting warps (8-bit)
    if constexpr (C::kRaw) {
      if constexpr (C::kSplitRegs) regs_lower<C::kConvRegs>();
      const int cw = warp - 4 - C::kSoftWarps, tid = cw * 32 + lane;
      constexpr int kStepRows = 8 * 4 / C::kHalves;       // rows between a warp's steps
      constexpr int kSteps = KT / 8 * C::kHalves / 4, kBatch = 4;
      const int half = cw % C::kHalves, x = lane & 3, r7 = (lane >> 3) ^ (((lane >> 2) & 1) * 5);
      const int row = cw / C::kHalves * 8 + r7;
      const uint32_t src_at = C::kRawBox == 128
                                  ? (half >> 1) * (KT * 128) + row * 128 + ((((4 * half + x) & 7) ^ r7) << 4)
                                  : row * 64 + ((x ^ ((row >> 1) & 3)) << 4);
      const uint32_t dst_at0 = half * (KT * 128) + row * 128 + (((2 * x) ^ r7) << 4);
      const uint32_t dst_at1 = half * (KT * 128) + row * 128 + (((2 * x + 1) ^ r7) << 4);
      uint32_t idx = 0;
      bool ok = true;
      while (ok && walk.next(p, w)) {
        const int low = lowest_seen(p, w);
        int most = -1000;                            // the largest eV so far
        for (int j = w.ja; ok && j < w.jb; ++j) {
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv, ++idx) {
            const int rs = idx % RS, st = idx % ST;
            ok = attn_wait(rfull_bar(rs), (idx / RS) & 1u, abort_flag, p);
            if (ok) ok = attn_wait(empty_bar(st), ((idx / ST) & 1u) ^ 1u, abort_flag, p);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const int live = w.s.kv - j * KT;        // positions of the sequence from the tile's first on
            const uint32_t sc = (idx >> 1) % C::kScaleSlots;
            float* slot = reinterpret_cast<float*>(smem + C::kOffScales + sc * C::kSlotBytes);
            // four 16-byte pieces (64 codes) of eight rows a step; of eight lanes four take
            // row r and four row r ^ 5, which keeps both the raw pieces they read and the
            // (even or odd) f16 pieces they write in eight different bank groups
            const uint32_t src = sbase + C::kOffRaw + rs * C::kRawTile + src_at, dst = ring + st * C::kTile;
            // Compiled apart for K, which is the codes alone, and V; the loop stays rolled, for
            // the softmax warps need the instruction cache (512 new tokens over fp8 caches:
            // one unrolled piece of code for both took 13% longer, unrolled and apart 5%).
            auto convert = [&](auto v_tile) {
              constexpr bool kV = decltype(v_tile)::value;
              const int ev = kV ? __float_as_int(slot[KT]) : 0;
              const bool apart = ev == kApart;
              const float unit = apart ? 1.0f : exp2_int(-ev);
#pragma unroll 1
              for (int k0 = 0; k0 < kSteps; k0 += kBatch) {
                uint4 v[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) v[k] = ld_shared_v4(src + (k0 + k) * kStepRows * C::kRawBox);
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                  const uint32_t to = dst + (k0 + k) * kStepRows * 128;
                  __half2 f1, f0;
                  if constexpr (kV) {
                    // (rows past the sequence hold anything: a NaN is not silenced by a zero weight)
                    const int r = row + (k0 + k) * kStepRows;
                    if (r >= live) v[k] = make_uint4(0, 0, 0, 0);
                    // the row's factor as a sum of two f16 numbers, so that a product is rounded once
                    const float f = r >= live ? 0.0f : apart ? 1.0f : slot[KT + 4 + r] * unit;
                    const __half hi = __float2half_rn(f);
                    f1 = __half2half2(hi), f0 = __half2half2(__float2half_rn(f - __half2float(hi)));
                  }
                  auto two = [&](uint32_t codes) {
                    if constexpr (!kV) return codes;
                    const __half2 x = *reinterpret_cast<const __half2*>(&codes);
                    const __half2 y = __hfma2(x, f1, __hmul2(x, f0));
                    return *reinterpret_cast<const uint32_t*>(&y);
                  };
                  st_shared_v4(to + dst_at0, make_uint4(two(codes01_to_f16x2<C::FMT>(v[k].x)), two(codes23_to_f16x2<C::FMT>(v[k].x)),
                                                        two(codes01_to_f16x2<C::FMT>(v[k].y)), two(codes23_to_f16x2<C::FMT>(v[k].y))));
                  st_shared_v4(to + dst_at1, make_uint4(two(codes01_to_f16x2<C::FMT>(v[k].z)), two(codes23_to_f16x2<C::FMT>(v[k].z)),
                                                        two(codes01_to_f16x2<C::FMT>(v[k].w)), two(codes23_to_f16x2<C::FMT>(v[k].w))));
                }
              }
            };
            if (kv == 0) {
              // The tile's scales and eV into its slot, which was last read for the tile kScaleSlots
              // before, whose V tile has left the ring.  (The softmax needs them after the K tile:
              // the search for eV runs beside its conversion.)
              const float* scales = reinterpret_cast<const float*>(smem + C::kOffRawScales) + rs * 2 * KT;
              // (positions that no row sees, whose scales may be anything, count as 0)
              const int from = max(0, low - j * KT);
              unsigned big = 0, small = 0xffffffffu;
#pragma unroll
              for (int x = 0; x < KT / 32; ++x) {
                const unsigned bits = __float_as_uint(scales[KT + 32 * x + lane]);
                if (32 * x + lane >= from && 32 * x + lane < live) {
                  big = max(big, bits);
                  small = min(small, bits);
                }
              }
              if (tid < KT) {
                slot[tid] = scales[tid];
                slot[KT + 4 + tid] = tid >= from ? scales[KT + tid] : 0.0f;
              }
              big = __reduce_max_sync(0xffffffffu, big);
              small = __reduce_min_sync(0xffffffffu, small);
              convert(std::false_type{});
              const bool alike = scales_alike(small, big, most);
              most = max(most, scale_exponent(big));
              if (tid == 0) slot[KT] = __int_as_float(alike ? scale_exponent(big) : kApart);
              if (!alike && tid < KT) slot[KT + 4 + tid] = log2_approx(slot[KT + 4 + tid]);
              __syncwarp();
              if (lane == 0) mbar_arrive(scale_bar(sc));
            } else {
              // (the slot is whole: other warps wrote parts of it)
              ok = attn_wait(scale_bar(sc), ((idx >> 1) / C::kScaleSlots) & 1u, abort_flag, p);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              convert(std::true_type{});
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(full_bar(st));
              mbar_arrive(rempty_bar(rs));
            }
          }
        }
      }
    }
  }

  // an item that starts here and goes on in the next CTAs: its parts, for the joining launch
  __syncthreads();
  if (threadIdx.x == 0) {
    JoinDesc d = {};
    Walker<KT, C::kItem> again(p, plan);
    while (again.next(p, w))
      if (w.starts && !w.ends) {
        d.parts = 1 + static_cast<int>((w.after + plan.quota - 1) / plan.quota);
        d.q0 = w.s.q0;
        d.n = w.s.n;
        d.kv = w.s.kv;
        d.slice = w.slice;
        d.rt = w.rt;
      }
    p.join[blockIdx.x] = d;
  }
  if (*abort_flag) settle_after_abort();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

template <class C>
static lora_status_t launch_many(AttnParams& p, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  if (!encode_pages(p, C::D, C::kRaw ? 1 : 2, C::kRaw ? C::kRawBox : 128, C::KT)) return LORA_ERR_CUDA;
  if (ensure_smem_limit(attn_many_kernel<C>, C::kSmem, done) != cudaSuccess) return LORA_ERR_CUDA;
  if constexpr (C::kSplitRegs) {
    // the warpgroups' shares must fit what the block is launched with: checked once
    static const bool fits = [] {
      cudaFuncAttributes a;
      return cudaFuncGetAttributes(&a, attn_many_kernel<C>) == cudaSuccess && a.numRegs >= C::kRegs;
    }();
    if (!fits) return LORA_ERR_CUDA;
  }
  int grid = num_sms();
  grid = grid > kMaxManyCtas ? kMaxManyCtas : grid;
  set_tiles(p, 128, C::NQ);
  if (!encode_map_3d(&p.qmap, p.q.x, C::D, p.hq, p.M, p.q.hs, p.q.ts, 64, p.hs, p.th)) return LORA_ERR_CUDA;
  LGB_TRY(launch_counted(attn_many_kernel<C>, dim3(grid), dim3(C::kThreads), C::kSmem, LORA_KIND_ATTN, st, p));
  return launch_counted(join_kernel<C::D, C::R>, dim3(grid, 16), dim3(128), 0, LORA_KIND_ATTN, st, p);
}

template <int D, int NQ>
static lora_status_t launch_many_d(AttnParams& p, int format, cudaStream_t st) {
  return format == LORA_KV_BF16 ? launch_many<ManyCfg<D, LORA_KV_BF16, NQ>>(p, st)
                                : format == LORA_KV_FP8 ? launch_many<ManyCfg<D, LORA_KV_FP8, NQ>>(p, st)
                                                        : launch_many<ManyCfg<D, LORA_KV_INT8, NQ>>(p, st);
}

lora_status_t launch_attn_many(AttnParams& p, int halves, int head_dim, int format, cudaStream_t st) {
  if (head_dim == 256) return launch_many_d<256, 1>(p, format, st);
  if (head_dim == 128) return halves == 2 ? launch_many_d<128, 2>(p, format, st) : launch_many_d<128, 1>(p, format, st);
  return halves == 2 ? launch_many_d<64, 2>(p, format, st) : launch_many_d<64, 1>(p, format, st);
}

}  // namespace lgb
