// Attention over the paged cache for many query rows per cache head (prefill chunks): the
// products run on the tcgen05 tensor cores.
//
// A CTA takes tiles of NQ x 128 packed query rows (two row halves up to head_dim 128, one
// at 256, where the output alone fills half of the tensor memory) against KT positions:
//   S = Q K^T        operands in shared memory, S in tensor memory (two buffers)
//   P = 2^(c S - m)  one thread per row: maximum, exponential and sum without a shuffle;
//                    P replaces S in place as packed bf16
//   O += P V         P from tensor memory, V from shared memory as it lies (MN-major)
// Roles: warp 0 fills a ring of K and V tiles by TMA (one box per page), warp 1 issues the
// MMAs, eight warps (one row half each four) do the softmax.  The tensor cores work on one
// half's products while the other half's softmax runs.  An accumulator is rescaled, in
// tensor memory, only when a row's maximum rises by more than 2^8 (kMaxSlack).
//
// 8-bit caches: the ring's raw tiles are turned into bf16 tiles by four more warps, once
// for all the tile's rows (both formats' codes are bf16 numbers); a position's K scale
// multiplies its score and its V scale its weight, in f32.
#include "paged_attn.cuh"
#include "codes.cuh"

namespace lgb {

template <int D_, int FMT_>
struct ManyCfg {
  static constexpr int D = D_, FMT = FMT_;
  static constexpr bool kRaw = FMT != LORA_KV_BF16;
  static constexpr int NQ = D == 256 ? 1 : 2;
  static constexpr int R = 128 * NQ;
  static constexpr int KT = D == 256 ? 64 : 128;
  static constexpr int kHalves = D / 64;                     // 128-byte columns of a bf16 row
  static constexpr int kTile = KT * D * 2;                   // one bf16 K or V tile
  static constexpr int kQBytes = 128 * D * 2;                // one row half of Q
  static constexpr int kRawRow = D, kRawBox = D < 128 ? D : 128, kRawBoxes = D / kRawBox;
  static constexpr int kRawTile = kRaw ? KT * D : 0;
  static constexpr int kRawStages = kRaw ? 3 : 0;
  static constexpr int kStages = kRaw ? (D == 64 ? 6 : 3) : (D == 64 ? 8 : 5);
  static constexpr int kScaleSlots = (kStages + 2) / 2;      // see the converting warps
  static constexpr int kConvWarps = kRaw ? 4 : 0;
  static constexpr int kSoftWarps = 4 * NQ;
  static constexpr int kThreads = 32 * (2 + kSoftWarps + kConvWarps);
  static constexpr bool kHold = !kRaw;                       // scores stay in registers between the two passes
  static constexpr int kSCol0 = 0, kSCols = KT, kOCol0 = 256;
  static constexpr int kOffRing = NQ * kQBytes;
  static constexpr int kOffRaw = kOffRing + kStages * kTile;
  static constexpr int kOffRawScales = kOffRaw + kRawStages * kRawTile;
  static constexpr int kOffScales = kOffRawScales + (kRaw ? kRawStages * KT * 4 : 0);
  static constexpr int kOffBars = kOffScales + (kRaw ? kScaleSlots * 2 * KT * 4 : 0);
  static constexpr int kNumBars = 2 * kStages + 2 * kRawStages + 2 * NQ + 2 + NQ + NQ + 1;
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

// Row halves of an item that hold rows of the sequence.
template <class C>
__device__ __forceinline__ int halves_of(const AttnParams& p, const Span& w) {
  const long long rows = static_cast<long long>(w.s.n) * p.hs - static_cast<long long>(w.rt) * C::R;
  return C::NQ == 2 && rows > 128 ? 2 : 1;
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
  auto full_bar = [&](int s) { return bar0 + 8u * s; };                          // a bf16 tile is in the ring
  auto empty_bar = [&](int s) { return bar0 + 8u * (ST + s); };
  auto rfull_bar = [&](int s) { return bar0 + 8u * (2 * ST + s); };              // a raw tile
  auto rempty_bar = [&](int s) { return bar0 + 8u * (2 * ST + RS + s); };
  constexpr int kB = 2 * ST + 2 * RS;
  // scores of half q are in buffer b (a barrier for each pair: a half that an item does not
  // use must not see phases go by)
  auto sfull_bar = [&](int q, int b) { return bar0 + 8u * (kB + 2 * q + b); };
  auto pready_bar = [&](int b) { return bar0 + 8u * (kB + 2 * C::NQ + b); };         // weights ready
  auto odone_bar = [&](int q) { return bar0 + 8u * (kB + 2 * C::NQ + 2 + q); };      // a half's O += P V is done
  auto qready_bar = [&](int q) { return bar0 + 8u * (kB + 3 * C::NQ + 2 + q); };
  const uint32_t drain_bar = bar0 + 8u * (kB + 4 * C::NQ + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(full_bar(s), C::kRaw ? C::kConvWarps : 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int s = 0; s < RS; ++s) {
      mbar_init(rfull_bar(s), 1);
      mbar_init(rempty_bar(s), C::kConvWarps);
    }
    for (int b = 0; b < 2; ++b) {
      for (int q = 0; q < C::NQ; ++q) mbar_init(sfull_bar(q, b), 1);
      mbar_init(pready_bar(b), 4);
    }
    for (int q = 0; q < C::NQ; ++q) {
      mbar_init(odone_bar(q), 1);
      mbar_init(qready_bar(q), 4);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_map(&p.kmap);
    tma_prefetch_map(&p.vmap);
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
  make_plan<R, KT, C::kThreads>(p, scratch);
  const Plan plan = scratch.plan;
  Walker<R, KT> walk(p, plan);
  Span w;

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
      int held = -64, page = 0;           // lane l holds the table's entry held + l
      for (int j = w.ja; ok && j < w.jb; ++j) {
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
        const int left = w.s.kv - j * KT;
        const int live = left <= 0 ? 0 : min(boxes, (left + box_rows - 1) / box_rows);
        const int r0 = lane * box_rows;
        const long long src = ((static_cast<long long>(mine) * p.cache.heads + kvh) << p.cache.page_shift) +
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
                mbar_arrive_expect_tx(fb, live * box_rows * (static_cast<uint32_t>(D * kEl) + (C::kRaw ? 4u : 0u)));
              else
                mbar_arrive(fb);
            }
            __syncwarp();
            if (lane < live) {
              const uint32_t dst = dst0 + stage * kDstTile + r0 * kBox;
#pragma unroll
              for (int x = 0; x < kBoxes; ++x)
                tma_load_2d(dst + x * (KT * kBox), kv ? &p.vmap : &p.kmap, fb, x * (kBox / kEl), static_cast<int>(src));
              if (C::kRaw)
                bulk_load(sbase + C::kOffRawScales + stage * (KT * 4) + r0 * 4, (kv ? p.cache.vs : p.cache.ks) + src,
                          box_rows * 4, fb);
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
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, KT, 0, 0);
      constexpr uint32_t idesc_o = idesc_bf16_f32(128, D, 0, 1);
      const uint64_t qdesc0 = smem_desc_sw128(sbase, 16u, 1024u);
      const uint64_t kdesc0 = smem_desc_sw128(ring, 16u, 1024u);
      const uint64_t vdesc0 = smem_desc_sw128(ring, KT * 128u, 1024u);
      constexpr uint64_t kTileStep = C::kTile >> 4;
      uint32_t tile = 0;              // ring tiles consumed before this item: K at tile + 2 i, V at tile + 2 i + 1
      uint32_t T = 0;                 // score tiles of this CTA so far: buffer T & 1
      uint32_t items[2] = {0, 0};     // items that used each half
      bool ok = true;
      while (ok && walk.next(p, w)) {
        const int nq = halves_of<C>(p, w), n = w.jb - w.ja, total = n * nq;
        for (int q = 0; q < nq && ok; ++q) {
          ok = attn_wait(qready_bar(q), items[q] & 1u, abort_flag, p);
          ++items[q];
        }
        if (!ok) break;
        auto issue_s = [&](int t) {   // scores of (position tile t / nq, half t % nq)
          const int i = nq == 2 ? t >> 1 : t, q = nq == 2 ? t & 1 : 0;
          const uint32_t idx = tile + 2u * i, st = idx % ST;
          if (q == 0 && !attn_wait(full_bar(st), (idx / ST) & 1u, abort_flag, p)) return false;
          tc_fence_after_sync();
          const uint32_t d = tmem + C::kSCol0 + ((T + t) & 1u) * C::kSCols;
          const uint64_t a = qdesc0 + static_cast<uint64_t>(q) * (C::kQBytes >> 4), b = kdesc0 + st * kTileStep;
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tc_mma_bf16(d, a + (k >> 2) * (128 * 128 >> 4) + (k & 3) * 2, b + (k >> 2) * (KT * 128 >> 4) + (k & 3) * 2,
                        idesc_s, k > 0 ? 1u : 0u);
          tc_commit(sfull_bar(q, (T + t) & 1u));
          if (q == nq - 1) tc_commit(empty_bar(st));
          return true;
        };
        ok = issue_s(0);
        for (int t = 0; t < total && ok; ++t) {
          if (t + 1 < total) ok = issue_s(t + 1);
          if (!ok) break;
          const int i = nq == 2 ? t >> 1 : t, q = nq == 2 ? t & 1 : 0;
          const uint32_t idx = tile + 2u * i + 1u, st = idx % ST, buf = (T + t) & 1u;
          if (q == 0) ok = attn_wait(full_bar(st), (idx / ST) & 1u, abort_flag, p);
          if (ok) ok = attn_wait(pready_bar(buf), ((T + t) >> 1) & 1u, abort_flag, p);
          if (!ok) break;
          tc_fence_after_sync();
          const uint32_t d = tmem + C::kOCol0 + q * D, a = tmem + C::kSCol0 + buf * C::kSCols;
          const uint64_t b = vdesc0 + st * kTileStep;
#pragma unroll
          for (int k = 0; k < KT / 16; ++k)
            tc_mma_bf16_ts(d, a + 8 * k, b + k * (2048 >> 4), idesc_o, (i > 0 || k > 0) ? 1u : 0u);
          tc_commit(odone_bar(q));
          if (q == nq - 1) tc_commit(empty_bar(st));
        }
        T += total;
        tile += 2u * n;
      }
      if (!ok) {
        tc_commit(drain_bar);
        attn_wait_drain(drain_bar, 0, p);
      }
    }
  } else if (warp < 2 + C::kSoftWarps) {
    // ------------------------------------------------------------ softmax
    const int q = (warp - 2) >> 2;                // row half
    const int quarter = warp & 3;                 // TMEM lanes of this warp
    const int r = quarter * 32 + lane;            // row of the half
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t o_tmem = tmem + lanes + C::kOCol0 + q * D;
    const float c = fabsf(p.scale_log2);
    const uint32_t flip = p.scale_log2 < 0.0f ? 0x80008000u : 0u;    // a negative scale turns Q's signs
    uint32_t T = 0, tile = 0, done = 0;           // done: O += P V steps of this half so far
    uint32_t sphase = 0;                          // bit b: phase of this half's score buffer b
    bool ok = true;
    while (ok && walk.next(p, w)) {
      const int nq = halves_of<C>(p, w), n = w.jb - w.ja;
      if (q >= nq) {
        T += n * nq;
        tile += 2u * n;
        continue;
      }
      int tok, head, lo, hi;
      const bool own = row_owner(p, w.s, w.slice, static_cast<long long>(w.rt) * R + q * 128 + r, tok, head);
      if (own) row_range(p, w.s, tok, lo, hi); else lo = 0, hi = 0x7fffffff;
      const int lo_max = __reduce_max_sync(0xffffffffu, lo), hi_min = __reduce_min_sync(0xffffffffu, hi);
      // this row of Q into shared memory, K-major with the 128-byte swizzle
      {
        const bf16* x = p.q.x + static_cast<long long>(w.s.q0 + tok) * p.q.ts + head * p.q.hs;
        const uint32_t dst = sbase + q * C::kQBytes + r * 128;
#pragma unroll
        for (int e = 0; e < D / 8; ++e) {
          uint4 v = own ? __ldg(reinterpret_cast<const uint4*>(x) + e) : make_uint4(0, 0, 0, 0);
          v.x ^= flip, v.y ^= flip, v.z ^= flip, v.w ^= flip;
          st_shared_v4(dst + (e >> 3) * (128 * 128) + (((e & 7) ^ (r & 7)) << 4), v);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(qready_bar(q));
      }
      float top = -INFINITY, sum = 0.0f;
      for (int i = 0; i < n; ++i) {
        const uint32_t t = T + (nq == 2 ? 2 * i + q : i), buf = t & 1u;
        const int k0 = (w.ja + i) * KT;
        const uint32_t s_tmem = tmem + lanes + C::kSCol0 + buf * C::kSCols;
        const uint32_t vidx = tile + 2u * i + 1u;
        const float* ks = nullptr;
        const float* vs = nullptr;
        ok = attn_wait(sfull_bar(q, buf), (sphase >> buf) & 1u, abort_flag, p);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        sphase ^= 1u << buf;
        if (C::kRaw) {
          // the tile's scales were written before its V tile was handed over (its stage is
          // not reused before these weights are)
          ok = attn_wait(full_bar(vidx % ST), (vidx / ST) & 1u, abort_flag, p);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          ks = reinterpret_cast<const float*>(smem + C::kOffScales) + ((vidx >> 1) % C::kScaleSlots) * 2 * KT;
          vs = ks + KT;
        }
        tc_fence_after_sync();
        const bool edge = k0 < lo_max || k0 + KT > hi_min;
        // scores of columns [x, x + 32) of this row: K scales, mask
        auto scores = [&](int x, float (&s)[32]) {
          uint32_t v[32];
          tmem_ld32(s_tmem + x, v);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) s[e] = __uint_as_float(v[e]);
          if (C::kRaw) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 f = *reinterpret_cast<const float4*>(ks + x + e);
              s[e] *= f.x, s[e + 1] *= f.y, s[e + 2] *= f.z, s[e + 3] *= f.w;
            }
          }
          if (edge) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int key = k0 + x + e;
              s[e] = key >= lo && key < hi ? s[e] : -INFINITY;
            }
          }
        };
        float held[C::kHold ? KT / 32 : 1][32];
        float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int x = 0; x < KT / 32; ++x) {
          float(&s)[32] = held[C::kHold ? x : 0];
          scores(32 * x, s);
#pragma unroll
          for (int e = 0; e < 32; ++e) m[e & 3] = fmaxf(m[e & 3], s[e]);
        }
        const float tile_top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * c;
        // (0 * -inf is NaN: with a scale of 0 a hidden row's maximum must stay -inf)
        const float cand = tile_top != tile_top ? (c == 0.0f ? -INFINITY : tile_top) : tile_top;
        if (__any_sync(0xffffffffu, cand > top + kMaxSlack)) {
          const float next = fmaxf(top, cand);
          const float f = next == -INFINITY ? 1.0f : exp2_approx(top - next);
          top = next;
          sum *= f;
          if (i > 0) {
            ok = attn_wait(odone_bar(q), (done - 1u) & 1u, abort_flag, p);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
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
          }
        }
        const float ref = top == -INFINITY ? 0.0f : top;
        float l[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int x = 0; x < KT / 32; ++x) {
          float(&s)[32] = held[C::kHold ? x : 0];
          if (!C::kHold) scores(32 * x, s);
          uint32_t u[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              // a hidden score is -inf: its weight is 0 for every finite scale but 0
              y[k] = exp2_approx(fmaf(s[e + k], c, -ref));
              if (edge && s[e + k] == -INFINITY) y[k] = 0.0f;
              l[k] += y[k];
            }
            if (C::kRaw) {
              const float4 f = *reinterpret_cast<const float4*>(vs + 32 * x + e);
              const float g[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) y[k] = edge && s[e + k] == -INFINITY ? 0.0f : y[k] * g[k];
            }
            u[e / 2] = pack_bf16x2(y[0], y[1]);
            u[e / 2 + 1] = pack_bf16x2(y[2], y[3]);
          }
          tmem_st16(s_tmem + 16 * x, u);
        }
        sum += (l[0] + l[1]) + (l[2] + l[3]);
        tmem_st_wait();
        if (!C::kRaw && k0 + KT > w.s.kv) {
          // rows of V past the sequence hold anything, and zero weights do not silence a
          // NaN: they are cleared here (both halves' warps may, with the same zeros)
          ok = attn_wait(full_bar(vidx % ST), (vidx / ST) & 1u, abort_flag, p);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          const uint32_t vt = ring + (vidx % ST) * C::kTile;
          for (int row = max(w.s.kv - k0, 0) + quarter; row < KT; row += 4)
            for (int e = lane; e < D / 8; e += 32)
              st_shared_v4(vt + (e >> 3) * (KT * 128) + row * 128 + ((e & 7) << 4), make_uint4(0, 0, 0, 0));
          fence_proxy_async_smem();
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(pready_bar(buf));
        ++done;
      }
      T += n * nq;
      tile += 2u * n;
      if (!ok) break;
      ok = attn_wait(odone_bar(q), (done - 1u) & 1u, abort_flag, p);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      tc_fence_after_sync();
      const bool whole = w.starts && w.ends;
      const long long slot = 2ll * blockIdx.x + (w.starts ? 1 : 0);
      const bool none = top == -INFINITY && sum == 0.0f;
      const float inv = whole ? (none ? 0.0f : 1.0f / sum) : 1.0f;
      const long long orow = static_cast<long long>(w.s.q0 + tok) * p.hq + head;
      const long long prow = slot * R + q * 128 + r;
#pragma unroll 1
      for (int x = 0; x < D; x += 32) {
        uint32_t v[32];
        __syncwarp();
        tmem_ld32(o_tmem + x, v);
        tmem_ld_wait();
        if (!own) continue;
        if (whole) {
          uint32_t u[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            u[e] = none ? 0u : pack_bf16x2(__uint_as_float(v[2 * e]) * inv, __uint_as_float(v[2 * e + 1]) * inv);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4*>(p.out + orow * D + x + 8 * e) = make_uint4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]);
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 8) st_global_v8(p.part_o + prow * D + x + e, v + e);
        }
      }
      if (own) {
        if (!whole)
          p.part_ml[prow] = make_float2(top, sum);
        else if (p.lse != nullptr)
          p.lse[orow] = none ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
      }
      tc_fence_before_sync();
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ converting warps (8-bit)
    if constexpr (C::kRaw) {
      const int cw = warp - 2 - C::kSoftWarps, tid = cw * 32 + lane;
      uint32_t idx = 0;
      bool ok = true;
      while (ok && walk.next(p, w)) {
        for (int j = w.ja; ok && j < w.jb; ++j) {
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv, ++idx) {
            const int rs = idx % RS, st = idx % ST;
            ok = attn_wait(rfull_bar(rs), (idx / RS) & 1u, abort_flag, p);
            if (ok) ok = attn_wait(empty_bar(st), ((idx / ST) & 1u) ^ 1u, abort_flag, p);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            // scales of K tile and V tile of position tile idx / 2: the slot was last read by
            // the softmax of kScaleSlots tiles before, whose V tile has left the ring
            if (tid < KT)
              reinterpret_cast<float*>(smem + C::kOffScales)[((idx >> 1) % C::kScaleSlots * 2 + kv) * KT + tid] =
                  reinterpret_cast<const float*>(smem + C::kOffRawScales)[rs * KT + tid];
            const uint32_t src = sbase + C::kOffRaw + rs * C::kRawTile, dst = ring + st * C::kTile;
            constexpr int kPieces = D / 16;          // 16-byte pieces of a raw row
#pragma unroll 2
            for (int e = tid; e < KT * kPieces; e += 128) {
              const int row = e / kPieces, x = e % kPieces;
              const uint32_t at = C::kRawBox == 128
                                      ? src + (x >> 3) * (KT * 128) + row * 128 + (((x & 7) ^ (row & 7)) << 4)
                                      : src + row * 64 + ((x ^ ((row >> 1) & 3)) << 4);
              const uint4 v = ld_shared_v4(at);
              uint4 y[2];
              y[0] = make_uint4(codes_to_bf16x2<C::FMT>(__byte_perm(v.x, 0, 0x4140)),
                                codes_to_bf16x2<C::FMT>(__byte_perm(v.x, 0, 0x4342)),
                                codes_to_bf16x2<C::FMT>(__byte_perm(v.y, 0, 0x4140)),
                                codes_to_bf16x2<C::FMT>(__byte_perm(v.y, 0, 0x4342)));
              y[1] = make_uint4(codes_to_bf16x2<C::FMT>(__byte_perm(v.z, 0, 0x4140)),
                                codes_to_bf16x2<C::FMT>(__byte_perm(v.z, 0, 0x4342)),
                                codes_to_bf16x2<C::FMT>(__byte_perm(v.w, 0, 0x4140)),
                                codes_to_bf16x2<C::FMT>(__byte_perm(v.w, 0, 0x4342)));
              // the lanes of a row's second 64 features store their second piece first, so
              // that eight lanes always fill all banks
              const int odd = (x >> 2) & 1;
              const uint32_t base = dst + (x >> 2) * (KT * 128) + row * 128;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int piece = 2 * (x & 3) + (h ^ odd);
                st_shared_v4(base + ((piece ^ (row & 7)) << 4), (h ^ odd) ? y[1] : y[0]);
              }
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
    Walker<R, KT> again(p, plan);
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
  int grid = num_sms();
  grid = grid > kMaxManyCtas ? kMaxManyCtas : grid;
  p.spg = static_cast<int>(ceil_div(p.group, C::R));
  p.hs = static_cast<int>(ceil_div(p.group, p.spg));
  p.slices = p.cache.heads * p.spg;
  LGB_TRY(launch_counted(attn_many_kernel<C>, dim3(grid), dim3(C::kThreads), C::kSmem, LORA_KIND_ATTN, st, p));
  return launch_counted(join_kernel<C::D, C::R>, dim3(grid, 16), dim3(128), 0, LORA_KIND_ATTN, st, p);
}

template <int D>
static lora_status_t launch_many_d(AttnParams& p, int format, cudaStream_t st) {
  return format == LORA_KV_BF16 ? launch_many<ManyCfg<D, LORA_KV_BF16>>(p, st)
                                : format == LORA_KV_FP8 ? launch_many<ManyCfg<D, LORA_KV_FP8>>(p, st)
                                                        : launch_many<ManyCfg<D, LORA_KV_INT8>>(p, st);
}

lora_status_t launch_attn_many(AttnParams& p, int head_dim, int format, cudaStream_t st) {
  return head_dim == 64 ? launch_many_d<64>(p, format, st) : head_dim == 128 ? launch_many_d<128>(p, format, st)
                                                                             : launch_many_d<256>(p, format, st);
}

}  // namespace lgb
