// Attention over the paged cache for few query rows per cache head (a decode step: one
// token's heads).  Every K and V row is read once for at most 16 query rows, so memory
// bounds it; the products run on the warp-level matrix units (m16n8k16), whose 16 rows
// these few rows fill, straight from the tiles in shared memory.
//
// A CTA: one producer warp fills a ring of K/V tiles of 64 positions by TMA (128- or 64-byte
// swizzle, one box per page), four warps take a quarter of each tile's positions
// and keep a running maximum, sum and output of their own in registers, merged when the
// item's part ends.  bf16 weights go to the matrix units in two parts, P V is issued twice
// (beside the waits for memory this costs 1%).  Measured: one token of four sequences of 50,000 to 65,536 positions, 8
// cache heads of 128 features: 948 MB in 148 us (6.4 TB/s, 94% of a copy's rate).
//
// 8-bit caches run in f16, which holds both formats' codes exactly and to which they turn
// in fewer instructions than to bf16 (the conversions, not memory, set the pace: 64
// sequences of 200 to 8192 int8 positions, 569 MB in 131 us, 4.3 TB/s).  A row of
// Q is scaled by a power of two to f16's upper range (exact for features down to 2^-29 of
// the row's largest).  A position's K scale multiplies its score in f32; its V scale joins
// the weight as an exponent, 2^(s + log2 vs - m'), with a running maximum m' of its own, so
// that the f16 weights stay at the top of their range whatever the scales are, while the
// sum of the weights without it keeps the scores' maximum m.
#include <type_traits>

#include "paged_attn.cuh"
#include "codes.cuh"

namespace lgb {

template <int D_, int FMT_>
struct FewCfg {
  static constexpr int D = D_, FMT = FMT_;
  static constexpr int kEl = FMT == LORA_KV_BF16 ? 2 : 1;
  static constexpr int kRow = D * kEl;                        // bytes of a cached row
  static constexpr int kBox = kRow < 128 ? kRow : 128;        // bytes of a row that one box holds
  static constexpr int kBoxes = kRow / kBox;
  static constexpr int kKT = 64;                              // 16 positions for each of four warps
  // An item's own cost, in tiles: measured 1, 2, 3, 4, 6 at 152, 141, 136, 131, 136 us for 64
  // sequences of 200 to 8192 int8 positions.
  static constexpr int kItem = 4;
  static constexpr int kTile = kKT * kRow;
  static constexpr int kStage = 2 * kTile;
  // CTAs of an SM, 160 threads each: D = 256 needs the registers of one alone.  Two and three
  // took 171 and 201 us (bf16; shorter rings), 141 and 132 us (int8), 150 and 149 us (fp8) for
  // 64 sequences of 200 to 8192 positions with 128 features.
  static constexpr int kCtas = D == 256 ? 1 : D == 128 && FMT == LORA_KV_BF16 ? 2 : 3;
  static constexpr int kStagesFit = (kCtas == 1 ? 192 * 1024 : kCtas == 2 ? 96 * 1024 : 62 * 1024) / kStage;
  static constexpr int kStages = kStagesFit > 8 ? 8 : kStagesFit;
  static constexpr int kScales = FMT == LORA_KV_BF16 ? 0 : 2 * kKT * 4;    // bytes per stage
  static constexpr int kMergeLd = D + 4;
  static constexpr int kMerge = kFewRows * kMergeLd * 4;
  static constexpr int kThreads = 160;
  static constexpr int kOffScales = kStages * kStage;
  static constexpr int kOffMerge = kOffScales + kStages * kScales;
  static constexpr int kOffMl = kOffMerge + kMerge;                        // [4 warps][16 rows] float2
  static constexpr int kOffBars = kOffMl + 4 * kFewRows * 8;
  static constexpr int kOffPlan = kOffBars + 2 * kStages * 8 + 16;
  static constexpr int kSmem = kOffPlan + static_cast<int>(sizeof(PlanScratch<kThreads>)) + 1024;
};

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kCtas) attn_few_kernel(const __grid_constant__ AttnParams p) {
  constexpr int D = C::D, FMT = C::FMT, R = kFewRows, KT = C::kKT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 2 * C::kStages);
  auto& scratch = *reinterpret_cast<PlanScratch<C::kThreads>*>(smem + C::kOffPlan);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (C::kStages + s); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 4);
    }
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_map(&p.kmap);
    tma_prefetch_map(&p.vmap);
  }
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  make_plan<KT, C::kItem, C::kThreads>(p, scratch);
  const Plan plan = scratch.plan;
  if (threadIdx.x == 0) p.join[blockIdx.x].parts = 0;     // set below by the item that starts here and goes on
  if (plan.units == 0) return;

  Walker<KT, C::kItem> walk(p, plan);
  Span w;
  int stage = 0;
  uint32_t phase = 0;

  if (warp == 4) {
    // ------------------------------------------------------------ producer
    const int ps = 1 << p.cache.page_shift;
    const int box_rows = ps < KT ? ps : KT, boxes = KT / box_rows;
    int armed = 0;                        // stages filled so far, all drained if a wait runs out
    bool ok = true, first = true;
    while (ok && walk.next(p, w)) {
      const int kvh = w.slice / p.spg;
      const int* row = p.table + static_cast<long long>(w.b) * p.max_pages;
      const int pages = (w.s.kv + ps - 1) >> p.cache.page_shift;
      const int low = lowest_seen(p, w);
      int held = -64, page = 0;           // lane l holds the table's entry held + l
      for (int j = w.ja; j < w.jb; ++j) {
        ok = attn_wait(empty_bar(stage), phase ^ 1u, abort_flag, p);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
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
        const int left = w.s.kv - j * KT;                      // positions from the tile's first on
        const int live = left <= 0 ? 0 : min(boxes, (left + box_rows - 1) / box_rows);
        const int skip = max(0, low - j * KT) / box_rows;      // boxes that no row sees, below `live`
        const uint32_t fb = full_bar(stage);
        if (p.inject_stall && first) {                         // leave this stage empty
          first = false;
        } else {
          first = false;
          if (lane == 0) {
            if (live > 0)
              mbar_arrive_expect_tx(fb, box_rows * (live * 2u * C::kRow + (FMT == LORA_KV_BF16 ? 0u : (live - skip) * 8u)));
            else
              mbar_arrive(fb);
          }
          __syncwarp();
          if (lane < live) {
            const int r0 = lane * box_rows;
            const long long src = lane < skip ? -box_rows
                                              : ((static_cast<long long>(mine) * p.cache.heads + kvh) << p.cache.page_shift) +
                                                    ((j * KT + r0) & (ps - 1));
            const uint32_t kt = sbase + stage * C::kStage, vt = kt + C::kTile;
#pragma unroll
            for (int x = 0; x < C::kBoxes; ++x) {
              tma_load_2d(kt + x * (KT * C::kBox) + r0 * C::kBox, &p.kmap, fb, x * (C::kBox / C::kEl),
                          static_cast<int>(src));
              tma_load_2d(vt + x * (KT * C::kBox) + r0 * C::kBox, &p.vmap, fb, x * (C::kBox / C::kEl),
                          static_cast<int>(src));
            }
            if (FMT != LORA_KV_BF16 && lane >= skip) {
              const uint32_t sc = sbase + C::kOffScales + stage * C::kScales + r0 * 4;
              bulk_load(sc, p.cache.ks + src, box_rows * 4, fb);
              bulk_load(sc + KT * 4, p.cache.vs + src, box_rows * 4, fb);
            }
          }
        }
        ++armed;
        if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
      }
    }
    if (!ok) {
      // the copies of the last kStages fills may be in flight: let them land
      for (int f = armed > C::kStages ? armed - C::kStages : (p.inject_stall ? 1 : 0); f < armed; ++f)
        attn_wait_drain(full_bar(f % C::kStages), (f / C::kStages) & 1, p);
    }
    return;
  }

  // -------------------------------------------------------------- the four product warps
  constexpr bool k8 = FMT != LORA_KV_BF16;
  const int t = lane & 3, r0 = lane >> 2;         // fragment column pair and row (rows r0, r0 + 8)
  float* merge = reinterpret_cast<float*>(smem + C::kOffMerge);
  float2* ml = reinterpret_cast<float2*>(smem + C::kOffMl);
  // Shared-memory offsets of this lane's ldmatrix rows in a tile (its warp's first rows).  A
  // 16-byte piece is permuted within its row by the row's low bits (TMA's swizzle), so that
  // piece x + 4 lies at an offset that differs in one bit, and other rows of the same lane
  // at a constant distance.
  const int first = warp * 16;
  const uint32_t k_at = C::kBox == 128 ? (first + (lane & 7)) * 128 + (((lane >> 3) ^ (lane & 7)) << 4)
                                       : (first + (lane & 7)) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
  const uint32_t v_at = C::kBox == 128 ? (first + (lane & 15)) * 128 + (((lane >> 4) ^ (lane & 7)) << 4)
                                       : (first + (lane & 15)) * 64 + (((lane >> 4) ^ ((lane >> 1) & 3)) << 4);
  // a negative scale turns Q's signs; a scale of 0 becomes the smallest normal one (finite
  // scores weigh the same, a hidden one stays -inf)
  const float scale = fmaxf(fabsf(p.scale_log2), 1.17549435e-38f);
  const uint32_t flip = p.scale_log2 < 0.0f ? 0x80008000u : 0u;
  bool ok = true;
  while (walk.next(p, w)) {
    int tok[2], head[2], lo[2], hi[2];
    bool own[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      own[h] = row_owner(p, w.s, w.slice, w.rt, 0, r0 + 8 * h, tok[h], head[h]);
      if (own[h]) row_range(p, w.s, tok[h], lo[h], hi[h]); else lo[h] = 0, hi[h] = 0;
    }
    // the tile rows' common range: tiles inside it need no mask
    int lo_max = own[0] ? lo[0] : 0, hi_min = own[0] ? hi[0] : 0x7fffffff;
    if (own[1]) lo_max = max(lo_max, lo[1]), hi_min = min(hi_min, hi[1]);
    lo_max = __reduce_max_sync(0xffffffffu, lo_max);
    hi_min = __reduce_min_sync(0xffffffffu, hi_min);
    // Q fragments.  A step multiplies 16 features; which ones a fragment column stands for
    // is free as long as Q and K agree, so 8-bit K takes four neighbouring bytes a lane.
    uint32_t q[D / 16][4];
    float c[2] = {scale, scale};
    unsigned big[2] = {0, 0};
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bf16* x = p.q.x + static_cast<long long>(w.s.q0 + tok[h]) * p.q.ts + head[h] * p.q.hs + 16 * s;
        if (!k8) {
          q[s][h] = own[h] ? __ldg(reinterpret_cast<const uint32_t*>(x + 2 * t)) : 0u;
          q[s][2 + h] = own[h] ? __ldg(reinterpret_cast<const uint32_t*>(x + 2 * t + 8)) : 0u;
        } else {
          const uint2 v = own[h] ? __ldg(reinterpret_cast<const uint2*>(x + 4 * t)) : make_uint2(0u, 0u);
          q[s][h] = v.x;
          q[s][2 + h] = v.y;
          big[h] = max(max(big[h], max(v.x & 0x7FFFu, (v.x >> 16) & 0x7FFFu)), max(v.y & 0x7FFFu, (v.y >> 16) & 0x7FFFu));
        }
        q[s][h] ^= flip;
        q[s][2 + h] ^= flip;
      }
    }
    if (k8) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        big[h] = max(big[h], __shfl_xor_sync(0xffffffffu, big[h], 1));
        big[h] = max(big[h], __shfl_xor_sync(0xffffffffu, big[h], 2));
        // the row times 2^(14 - exponent of its largest), and the score scale without it
        const float f = __uint_as_float(static_cast<unsigned>(min(254, 268 - static_cast<int>(big[h] >> 7))) << 23);
        c[h] = fmaxf(scale / f, 1.17549435e-38f);
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
          for (int x = h; x < 4; x += 2)
            q[s][x] = pack_f16x2(__uint_as_float(q[s][x] << 16) * f, __uint_as_float(q[s][x] & 0xFFFF0000u) * f);
      }
    }
    float o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.0f;
    float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.0f, 0.0f};
    float vtop[2] = {-INFINITY, -INFINITY};       // 8-bit: of the scores with log2 of the V scales

    for (int j = w.ja; j < w.jb; ++j) {
      if (ok) ok = attn_wait(full_bar(stage), phase, abort_flag, p);
      ok = __all_sync(0xffffffffu, ok);
      // after an expired wait the warp walks on without data, so that the merge's barriers
      // below still meet
      if (ok) {
        const int k0 = j * KT + first;
        // compiled twice: for tiles that all rows see whole (nearly all), and for the others
        auto tile = [&](auto at_edge) {
        constexpr bool kEdge = decltype(at_edge)::value;
        const uint32_t ka = sbase + stage * C::kStage + k_at, va = sbase + stage * C::kStage + C::kTile + v_at;
        const float* ks = reinterpret_cast<const float*>(smem + C::kOffScales + stage * C::kScales) + first;
        const float* vs = ks + KT;
        float s[2][4];                            // positions k0 + 8 g + 2 t + {0, 1}, rows r0 and r0 + 8
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[g][e] = 0.0f;
#pragma unroll
        for (int x = 0; x < C::kRow / 16; x += 4) {          // four 16-byte pieces of a row
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint32_t b[4];
            ldmatrix_x4((ka ^ ((x & 7) << 4)) + (x >> 3) * (KT * 128) + 8 * g * C::kBox, b);
            if (!k8) {
              mma_m16n8k16_bf16(s[g], q[x / 2], b[0], b[1]);
              mma_m16n8k16_bf16(s[g], q[x / 2 + 1], b[2], b[3]);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                mma_m16n8k16_f16(s[g], q[k8 ? x + e : 0], codes01_to_f16x2<FMT>(b[e]), codes23_to_f16x2<FMT>(b[e]));
            }
          }
        }
        float most[2] = {-INFINITY, -INFINITY}, vmost[2] = {-INFINITY, -INFINITY};
        float2 lv[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (k8) {
            const float2 sc = *reinterpret_cast<const float2*>(ks + 8 * g + 2 * t);
            s[g][0] *= sc.x, s[g][1] *= sc.y, s[g][2] *= sc.x, s[g][3] *= sc.y;
            const float2 v = *reinterpret_cast<const float2*>(vs + 8 * g + 2 * t);
            lv[g] = make_float2(log2_approx(v.x), log2_approx(v.y));
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (kEdge) {
              const int key = k0 + 8 * g + 2 * t + (e & 1);
              if (key < lo[e >> 1] || key >= hi[e >> 1]) s[g][e] = -INFINITY;
            }
            most[e >> 1] = fmaxf(most[e >> 1], s[g][e]);
            if (k8) vmost[e >> 1] = fmaxf(vmost[e >> 1], fmaf(s[g][e], c[e >> 1], (e & 1) ? lv[g].y : lv[g].x));
          }
        }
        bool rise = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          most[h] = fmaxf(most[h], __shfl_xor_sync(0xffffffffu, most[h], 1));
          most[h] = fmaxf(most[h], __shfl_xor_sync(0xffffffffu, most[h], 2)) * c[h];
          rise = rise || most[h] > top[h] + kMaxSlack;
          if (k8) {
            vmost[h] = fmaxf(vmost[h], __shfl_xor_sync(0xffffffffu, vmost[h], 1));
            vmost[h] = fmaxf(vmost[h], __shfl_xor_sync(0xffffffffu, vmost[h], 2));
            rise = rise || vmost[h] > vtop[h] + kMaxSlack;
          }
        }
        if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float next = fmaxf(top[h], most[h]), vnext = fmaxf(vtop[h], vmost[h]);
            const float f = next == -INFINITY ? 1.0f : exp2_approx(top[h] - next);
            const float fo = !k8 ? f : vnext == -INFINITY ? 1.0f : exp2_approx(vtop[h] - vnext);
            top[h] = next;
            vtop[h] = vnext;
            sum[h] *= f;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) o[n][2 * h] *= fo, o[n][2 * h + 1] *= fo;
          }
        }
        const float m[2] = {top[0] == -INFINITY ? 0.0f : top[0], top[1] == -INFINITY ? 0.0f : top[1]};
        const float vm[2] = {vtop[0] == -INFINITY ? 0.0f : vtop[0], vtop[1] == -INFINITY ? 0.0f : vtop[1]};
        // A weight's 16 bits; bf16 ones carry 16 bits of significand in two parts, the second
        // rounded by 2^-16 of the weight.  (Parts of the same sign, and neither 0 unless both
        // are: they take an infinity of V to the same infinity.)
        uint32_t a[4], rest[4];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int h = e >> 1;
            x[e] = exp2_approx(fmaf(s[g][e], c[h], -m[h]));
            sum[h] += x[e];
            if (k8) {
              x[e] = exp2_approx(fmaf(s[g][e], c[h], ((e & 1) ? lv[g].y : lv[g].x) - vm[h]));
              if (kEdge && s[g][e] == -INFINITY) x[e] = 0.0f;        // a hidden position's scale is not looked at
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t& w = a[2 * g + h];
            if (k8) {
              w = pack_f16x2(x[2 * h], x[2 * h + 1]);
            } else {
              w = __byte_perm(__float_as_uint(x[2 * h]), __float_as_uint(x[2 * h + 1]), 0x7632);
              float r[2];
#pragma unroll
              for (int d = 0; d < 2; ++d)
                r[d] = fmaxf(x[2 * h + d] - __uint_as_float(__float_as_uint(x[2 * h + d]) & 0xFFFF0000u), x[2 * h + d] * 0x1p-24f);
              rest[2 * g + h] = pack_bf16x2(r[0], r[1]);
            }
          }
        }
        // rows of V past the sequence hold anything: zero weights do not silence a NaN
        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
        if (kEdge) {
          const int a0 = w.s.kv - k0 - 2 * t, a1 = a0 - 8;      // positions left from this lane's first
          keep0 = a0 >= 2 ? 0xffffffffu : a0 == 1 ? 0x0000ffffu : 0u;
          keep1 = a1 >= 2 ? 0xffffffffu : a1 == 1 ? 0x0000ffffu : 0u;
        }
#pragma unroll
        for (int x = 0; x < C::kRow / 16; x += 2) {        // two 16-byte pieces of 16 rows
          uint32_t b[4];
          ldmatrix_x4_trans((va ^ ((x & 7) << 4)) + (x >> 3) * (KT * 128), b);
          if (kEdge) {
            // (8-bit: a 16-bit element of the transposed tile is two features' codes)
            b[0] &= keep0, b[1] &= keep1, b[2] &= keep0, b[3] &= keep1;
          }
          if (!k8) {
            mma_m16n8k16_bf16(o[x], a, b[0], b[1]);
            mma_m16n8k16_bf16(o[x + 1], a, b[2], b[3]);
            mma_m16n8k16_bf16(o[x], rest, b[0], b[1]);
            mma_m16n8k16_bf16(o[x + 1], rest, b[2], b[3]);
          } else {
            // o[2 x] holds features 16 x + 2 n, o[2 x + 1] features 16 x + 2 n + 1
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              mma_m16n8k16_f16(o[k8 ? 2 * (x + e) : 0], a, codes02_to_f16x2<FMT>(b[2 * e]),
                               codes02_to_f16x2<FMT>(b[2 * e + 1]));
              mma_m16n8k16_f16(o[k8 ? 2 * (x + e) + 1 : 0], a, codes13_to_f16x2<FMT>(b[2 * e]),
                               codes13_to_f16x2<FMT>(b[2 * e + 1]));
            }
          }
        }
        };
        if (k0 >= lo_max && k0 + 16 <= hi_min)
          tile(std::false_type{});
        else
          tile(std::true_type{});
        __syncwarp();
        if (lane == 0) mbar_arrive(empty_bar(stage));
      }
      if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
    }
    if (k8) {
      // the outputs back to the scores' maximum (in two factors: 2^(vtop - top) may leave f32's
      // range where the product does not)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float f = vtop[h] == -INFINITY ? 0.0f : exp2_approx(0.5f * (vtop[h] - top[h]));
#pragma unroll
        for (int n = 0; n < D / 8; ++n) o[n][2 * h] = o[n][2 * h] * f * f, o[n][2 * h + 1] = o[n][2 * h + 1] * f * f;
      }
    }

    // The four warps' parts, four rows at a time: each warp lays its outputs down as they
    // are, and a thread joins four features of a row under the common maximum.  (Adding
    // them up in turn, one warp after the other, took 13 thousand cycles an item.)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
      sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
      if (t == 0) ml[warp * R + r0 + 8 * h] = make_float2(top[h], sum[h]);
    }
    const bool whole = w.starts && w.ends;
    const int slot = 2 * blockIdx.x + (w.starts ? 1 : 0);
    const int used = p.th * p.hs;                 // rows of the tile
#pragma unroll 1
    for (int pass = 0; 4 * pass < used; ++pass) {
      if ((r0 >> 2) == (pass & 1)) {
        float* line = merge + (4 * warp + (r0 & 3)) * C::kMergeLd + 2 * t;
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
          *reinterpret_cast<float2*>(line + 8 * n) = pass < 2 ? make_float2(o[n][0], o[n][1]) : make_float2(o[n][2], o[n][3]);
      }
      named_barrier(1, 128);
#pragma unroll
      for (int i0 = 0; i0 < D; i0 += 128) {
        const int i = i0 + threadIdx.x, r = 4 * pass + i / (D / 4), f = i % (D / 4) * 4;
        int tk, hd;
        if (!ok || i >= D || !row_owner(p, w.s, w.slice, w.rt, 0, r, tk, hd)) continue;
        float2 v[4];
        float m = -INFINITY;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          v[x] = ml[x * R + r];
          m = fmaxf(m, v[x].x);
        }
        const float ref = m == -INFINITY ? 0.0f : m;
        float l = 0.0f;
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float* line = merge + (4 * x + (r & 3)) * C::kMergeLd;
          float4 u;
          if (!k8) {
            u = *reinterpret_cast<const float4*>(line + f);
          } else {
            // features 16 c + 4 t + {0, 1, 2, 3} are columns 2 t, 2 t + 1 of o[2c] and of o[2c + 1]
            const float2 even = *reinterpret_cast<const float2*>(line + f / 16 * 16 + f % 16 / 2);
            const float2 odd = *reinterpret_cast<const float2*>(line + f / 16 * 16 + 8 + f % 16 / 2);
            u = make_float4(even.x, odd.x, even.y, odd.y);
          }
          const float g = exp2_approx(v[x].x - ref);
          l += g * v[x].y;
          y.x += g * u.x;
          y.y += g * u.y;
          y.z += g * u.z;
          y.w += g * u.w;
        }
        if (whole) {
          const bool none = m == -INFINITY && l == 0.0f;
          const float inv = none ? 0.0f : 1.0f / l;
          const long long row = static_cast<long long>(w.s.q0 + tk) * p.hq + hd;
          uint2 u;
          u.x = pack_bf16x2(y.x * inv, y.y * inv);
          u.y = pack_bf16x2(y.z * inv, y.w * inv);
          *reinterpret_cast<uint2*>(p.out + row * D + f) = u;
          if (p.lse != nullptr && f == 0) p.lse[row] = none ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
        } else {
          *reinterpret_cast<float4*>(p.part_o + (static_cast<long long>(slot) * R + r) * D + f) = y;
          if (f == 0) p.part_ml[static_cast<long long>(slot) * R + r] = make_float2(m, l);
        }
      }
      named_barrier(1, 128);            // `merge` is free again (after the last pass `ml` too)
    }
    if (ok && threadIdx.x == 0 && w.starts && !w.ends) {
      JoinDesc d;
      d.parts = 1 + static_cast<int>((w.after + plan.quota - 1) / plan.quota);
      d.q0 = w.s.q0;
      d.n = w.s.n;
      d.kv = w.s.kv;
      d.slice = w.slice;
      d.rt = w.rt;
      p.join[blockIdx.x] = d;
    }
  }
}

template <class C>
static lora_status_t launch_few(AttnParams& p, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  if (!encode_pages(p, C::D, C::kEl, C::kBox, C::kKT)) return LORA_ERR_CUDA;
  if (ensure_smem_limit(attn_few_kernel<C>, C::kSmem, done) != cudaSuccess) return LORA_ERR_CUDA;
  int grid = C::kCtas * num_sms();
  grid = grid > kMaxFewCtas ? kMaxFewCtas : grid;
  LGB_TRY(launch_counted(attn_few_kernel<C>, dim3(grid), dim3(C::kThreads), C::kSmem, LORA_KIND_ATTN, st, p));
  constexpr int kRowsPerBlock = 128 / (C::D / 4);
  return launch_counted(join_kernel<C::D, kFewRows>, dim3(grid, kFewRows / kRowsPerBlock), dim3(128), 0, LORA_KIND_ATTN,
                        st, p);
}

template <int D>
static lora_status_t launch_few_d(AttnParams& p, int format, cudaStream_t st) {
  return format == LORA_KV_BF16 ? launch_few<FewCfg<D, LORA_KV_BF16>>(p, st)
                                : format == LORA_KV_FP8 ? launch_few<FewCfg<D, LORA_KV_FP8>>(p, st)
                                                        : launch_few<FewCfg<D, LORA_KV_INT8>>(p, st);
}

lora_status_t launch_attn_few(AttnParams& p, int head_dim, int format, cudaStream_t st) {
  set_tiles(p, kFewRows, 1);
  return head_dim == 64 ? launch_few_d<64>(p, format, st) : head_dim == 128 ? launch_few_d<128>(p, format, st)
                                                                            : launch_few_d<256>(p, format, st);
}

}  // namespace lgb
