// Attention over the paged cache for few query rows per cache head (a decode step: one
// token's heads).  Every K and V row is read once for at most 16 query rows, so memory
// bounds it; the products run on the warp-level matrix units (m16n8k16), whose 16 rows
// these few rows fill, straight from the tiles in shared memory.
//
// A CTA: one producer warp fills a ring of K/V tiles of 64 positions by TMA (128- or
// 64-byte swizzle, one box per page), four warps take 16 positions of each tile and keep
// a running maximum, sum and output of their own in registers, merged when the item's
// part ends.  8-bit codes become bf16 exactly in registers (both formats' values fit
// bf16), the row scales multiply the scores and the weights in f32.
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
  static constexpr int kKT = 64;
  static constexpr int kTile = kKT * kRow;
  static constexpr int kStage = 2 * kTile;
  // D = 256 needs the registers of a whole SM for 160 threads; otherwise two CTAs share one
  static constexpr int kCtas = D == 256 ? 1 : 2;
  static constexpr int kStagesFit = (kCtas == 1 ? 192 * 1024 : 96 * 1024) / kStage;
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

// Shared-memory address of 16-byte piece c of row r of a tile: boxes of kBox-byte rows, the
// pieces of a row permuted as TMA's swizzle of that row width does.
template <class C>
__device__ __forceinline__ uint32_t piece_addr(uint32_t tile, int r, int c) {
  if (C::kBox == 128) return tile + (c >> 3) * (C::kKT * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
  return tile + r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

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
  make_plan<KT, C::kThreads>(p, scratch);
  const Plan plan = scratch.plan;
  if (threadIdx.x == 0) p.join[blockIdx.x].parts = 0;     // set below by the item that starts here and goes on
  if (plan.units == 0) return;

  Walker<KT> walk(p, plan);
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
      int held = -64, page = 0;           // lane l holds the table's entry held + l
      for (int j = w.ja; j < w.jb; ++j) {
        ok = attn_wait(empty_bar(stage), phase ^ 1u, abort_flag, p);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int at = (j * KT) >> p.cache.page_shift;
        if (at + boxes > held + 32) {
          held = at;
          page = 0;
          if (at + lane < pages) {
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
        const uint32_t fb = full_bar(stage);
        if (p.inject_stall && first) {                         // leave this stage empty
          first = false;
        } else {
          first = false;
          if (lane == 0) {
            if (live > 0)
              mbar_arrive_expect_tx(fb, live * box_rows * (2u * C::kRow + (FMT == LORA_KV_BF16 ? 0u : 8u)));
            else
              mbar_arrive(fb);
          }
          __syncwarp();
          if (lane < live) {
            const int r0 = lane * box_rows;
            const long long src = ((static_cast<long long>(mine) * p.cache.heads + kvh) << p.cache.page_shift) +
                                  ((j * KT + r0) & (ps - 1));
            const uint32_t kt = sbase + stage * C::kStage, vt = kt + C::kTile;
#pragma unroll
            for (int x = 0; x < C::kBoxes; ++x) {
              tma_load_2d(kt + x * (KT * C::kBox) + r0 * C::kBox, &p.kmap, fb, x * (C::kBox / C::kEl),
                          static_cast<int>(src));
              tma_load_2d(vt + x * (KT * C::kBox) + r0 * C::kBox, &p.vmap, fb, x * (C::kBox / C::kEl),
                          static_cast<int>(src));
            }
            if (FMT != LORA_KV_BF16) {
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
  const int t = lane & 3, r0 = lane >> 2;         // fragment column pair and row (rows r0, r0 + 8)
  float* merge = reinterpret_cast<float*>(smem + C::kOffMerge);
  float2* ml = reinterpret_cast<float2*>(smem + C::kOffMl);
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
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bf16* x = p.q.x + static_cast<long long>(w.s.q0 + tok[h]) * p.q.ts + head[h] * p.q.hs + 16 * s;
        if (FMT == LORA_KV_BF16) {
          q[s][h] = own[h] ? __ldg(reinterpret_cast<const uint32_t*>(x + 2 * t)) : 0u;
          q[s][2 + h] = own[h] ? __ldg(reinterpret_cast<const uint32_t*>(x + 2 * t + 8)) : 0u;
        } else {
          const uint2 v = own[h] ? __ldg(reinterpret_cast<const uint2*>(x + 4 * t)) : make_uint2(0u, 0u);
          q[s][h] = v.x;
          q[s][2 + h] = v.y;
        }
      }
    }
    float o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.0f;
    float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.0f, 0.0f};

    for (int j = w.ja; j < w.jb; ++j) {
      if (ok) ok = attn_wait(full_bar(stage), phase, abort_flag, p);
      ok = __all_sync(0xffffffffu, ok);
      // after an expired wait the warp walks on without data, so that the merge's barriers
      // below still meet
      if (ok) {
        const int k0 = j * KT + warp * 16;
        const uint32_t kt = sbase + stage * C::kStage, vt = kt + C::kTile;
        const float* ks = reinterpret_cast<const float*>(smem + C::kOffScales + stage * C::kScales) + warp * 16;
        const float* vs = ks + KT;
        float s[2][4] = {};                       // positions k0 + 8 g + 2 t + {0, 1}, rows r0 and r0 + 8
        if (FMT == LORA_KV_BF16) {
#pragma unroll
          for (int c = 0; c < D / 16; c += 2) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              uint32_t b[4];
              ldmatrix_x4(piece_addr<C>(kt, warp * 16 + 8 * g + (lane & 7), 2 * c + (lane >> 3)), b);
              mma_m16n8k16_bf16(s[g], q[c], b[0], b[1]);
              mma_m16n8k16_bf16(s[g], q[c + 1], b[2], b[3]);
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < D / 16; c += 4) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              uint32_t b[4];
              ldmatrix_x4(piece_addr<C>(kt, warp * 16 + 8 * g + (lane & 7), c + (lane >> 3)), b);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                mma_m16n8k16_bf16(s[g], q[c + e], codes01_to_bf16x2<FMT>(b[e]), codes23_to_bf16x2<FMT>(b[e]));
            }
          }
        }
        const bool edge = k0 < lo_max || k0 + 16 > hi_min;
        float tile_top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          float f0 = p.scale_log2, f1 = p.scale_log2;
          if (FMT != LORA_KV_BF16) {
            const float2 sc = *reinterpret_cast<const float2*>(ks + 8 * g + 2 * t);
            f0 *= sc.x;
            f1 *= sc.y;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[g][e] *= (e & 1) ? f1 : f0;
            if (edge) {
              const int key = k0 + 8 * g + 2 * t + (e & 1);
              if (key < lo[e >> 1] || key >= hi[e >> 1]) s[g][e] = -INFINITY;
            }
            tile_top[e >> 1] = fmaxf(tile_top[e >> 1], s[g][e]);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          tile_top[h] = fmaxf(tile_top[h], __shfl_xor_sync(0xffffffffu, tile_top[h], 1));
          tile_top[h] = fmaxf(tile_top[h], __shfl_xor_sync(0xffffffffu, tile_top[h], 2));
        }
        const bool rise = tile_top[0] > top[0] + kMaxSlack || tile_top[1] > top[1] + kMaxSlack;
        if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float next = fmaxf(top[h], tile_top[h]);
            const float f = next == -INFINITY ? 1.0f : exp2_approx(top[h] - next);
            top[h] = next;
            sum[h] *= f;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) o[n][2 * h] *= f, o[n][2 * h + 1] *= f;
          }
        }
        const float m0 = top[0] == -INFINITY ? 0.0f : top[0], m1 = top[1] == -INFINITY ? 0.0f : top[1];
        uint32_t a[4];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[e] = exp2_approx(s[g][e] - (e < 2 ? m0 : m1));
            sum[e >> 1] += x[e];
          }
          if (FMT != LORA_KV_BF16) {
            const float2 sc = *reinterpret_cast<const float2*>(vs + 8 * g + 2 * t);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float y = x[e] * ((e & 1) ? sc.y : sc.x);
              x[e] = edge && s[g][e] == -INFINITY ? 0.0f : y;       // a hidden position's scale is not looked at
            }
          }
          a[2 * g] = pack_bf16x2(x[0], x[1]);
          a[2 * g + 1] = pack_bf16x2(x[2], x[3]);
        }
        if (FMT == LORA_KV_BF16) {
          // rows of V past the sequence hold anything: zero weights do not silence a NaN
          uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
          const bool past = k0 + 16 > w.s.kv;
          if (past) {
            const int a0 = w.s.kv - k0 - 2 * t, a1 = a0 - 8;        // positions left from this lane's first
            keep0 = a0 >= 2 ? 0xffffffffu : a0 == 1 ? 0x0000ffffu : 0u;
            keep1 = a1 >= 2 ? 0xffffffffu : a1 == 1 ? 0x0000ffffu : 0u;
          }
#pragma unroll
          for (int n = 0; n < D / 8; n += 2) {
            uint32_t b[4];
            ldmatrix_x4_trans(piece_addr<C>(vt, warp * 16 + (lane & 15), n + (lane >> 4)), b);
            if (past) b[0] &= keep0, b[1] &= keep1, b[2] &= keep0, b[3] &= keep1;
            mma_m16n8k16_bf16(o[n], a, b[0], b[1]);
            mma_m16n8k16_bf16(o[n + 1], a, b[2], b[3]);
          }
        } else {
          // a 16-bit element of the transposed tile is two features' codes: o[2c] holds
          // features 16 c + 2 n, o[2c + 1] features 16 c + 2 n + 1
#pragma unroll
          for (int c = 0; c < D / 16; c += 2) {
            uint32_t b[4];
            ldmatrix_x4_trans(piece_addr<C>(vt, warp * 16 + (lane & 15), c + (lane >> 4)), b);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              mma_m16n8k16_bf16(o[2 * (c + e)], a, codes02_to_bf16x2<FMT>(b[2 * e]),
                                codes02_to_bf16x2<FMT>(b[2 * e + 1]));
              mma_m16n8k16_bf16(o[2 * (c + e) + 1], a, codes13_to_bf16x2<FMT>(b[2 * e]),
                                codes13_to_bf16x2<FMT>(b[2 * e + 1]));
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty_bar(stage));
      }
      if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
    }

    // the four warps' parts: a common maximum, then the outputs one after the other
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
      sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
      if (t == 0) ml[warp * R + r0 + 8 * h] = make_float2(top[h], sum[h]);
    }
    named_barrier(1, 128);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float m = -INFINITY;
#pragma unroll
      for (int x = 0; x < 4; ++x) m = fmaxf(m, ml[x * R + r0 + 8 * h].x);
      const float f = exp2_approx(top[h] - (m == -INFINITY ? 0.0f : m));
#pragma unroll
      for (int n = 0; n < D / 8; ++n) o[n][2 * h] *= f, o[n][2 * h + 1] *= f;
    }
#pragma unroll 1
    for (int x = 0; x < 4; ++x) {
      if (warp == x) {
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float2* cell = reinterpret_cast<float2*>(merge + (r0 + 8 * h) * C::kMergeLd + 8 * n + 2 * t);
            float2 v = make_float2(o[n][2 * h], o[n][2 * h + 1]);
            if (!own[h]) continue;
            if (x > 0) {
              const float2 b = *cell;
              v.x += b.x;
              v.y += b.y;
            }
            *cell = v;
          }
      }
      named_barrier(1, 128);
    }
    // merged rows out: feature order in `merge` is the fragments' (see above)
    const bool whole = w.starts && w.ends;
    const int slot = 2 * blockIdx.x + (w.starts ? 1 : 0);
    if (ok) {
      constexpr int kLanes = D / 4;                 // threads of a row, four features each
      for (int r = threadIdx.x / kLanes; r < R; r += 128 / kLanes) {
        int tk, hd;
        if (!row_owner(p, w.s, w.slice, w.rt, 0, r, tk, hd)) continue;
        const int f = (threadIdx.x % kLanes) * 4;
        float4 v;
        if (FMT == LORA_KV_BF16) {
          v = *reinterpret_cast<const float4*>(merge + r * C::kMergeLd + f);
        } else {
          // features 16 c + 4 t + {0, 1, 2, 3} are columns 2 t, 2 t + 1 of o[2c] and of o[2c + 1]
          const int c = f / 16, tt = (f % 16) / 4;
          const float2 even = *reinterpret_cast<const float2*>(merge + r * C::kMergeLd + 16 * c + 2 * tt);
          const float2 odd = *reinterpret_cast<const float2*>(merge + r * C::kMergeLd + 16 * c + 8 + 2 * tt);
          v = make_float4(even.x, odd.x, even.y, odd.y);
        }
        float m = -INFINITY, l = 0.0f;
#pragma unroll
        for (int x = 0; x < 4; ++x) m = fmaxf(m, ml[x * R + r].x);
        const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int x = 0; x < 4; ++x) l += ml[x * R + r].y * exp2_approx(ml[x * R + r].x - ref);
        if (whole) {
          const bool none = m == -INFINITY && l == 0.0f;
          const float inv = none ? 0.0f : 1.0f / l;
          const long long row = static_cast<long long>(w.s.q0 + tk) * p.hq + hd;
          uint2 u;
          u.x = pack_bf16x2(v.x * inv, v.y * inv);
          u.y = pack_bf16x2(v.z * inv, v.w * inv);
          *reinterpret_cast<uint2*>(p.out + row * D + f) = u;
          if (p.lse != nullptr && f == 0) p.lse[row] = none ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
        } else {
          *reinterpret_cast<float4*>(p.part_o + (static_cast<long long>(slot) * R + r) * D + f) = v;
          if (f == 0) p.part_ml[static_cast<long long>(slot) * R + r] = make_float2(m, l);
        }
      }
      if (threadIdx.x == 0 && w.starts && !w.ends) {
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
    named_barrier(1, 128);            // `merge` and `ml` are free again
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
