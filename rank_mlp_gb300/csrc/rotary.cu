// Rotary positions of views of heads (lora_rotary) and their tables for long contexts
// (lora_rope_table_scaled); include/lora_gb300.h is the contract.
//
// The rotation reads 2 bytes and writes 2 bytes a feature for a handful of f32
// operations, so memory bounds it.  A thread owns the pairs that one 16-byte piece (half
// layout: two pieces, half a rotation apart) holds and walks several heads of its token
// with the same cos and sin in registers; owning whole pairs, it can write over its
// input.  Measured: 8192 tokens of 32 + 8 heads of 128 features, 172 MB in 30 us (5.7 TB/s,
// 84% of a copy's rate); 16 tokens 1.9 us in a graph.
#include "serve.cuh"

namespace lgb {

struct RotaryParams {
  HeadsView in[2];
  HeadsOut out[2];
  int heads0, heads;         // heads of q, of q and k
  long long M;
  RotaryArgs rot;
  float sign;                // -1: the inverse rotation
  int interleaved;
  int dim;                   // head_dim
  int items;                 // thread items of a head: rotated ones, then passed-through ones
  int turned;                // the rotated ones among them
  int per_group, groups;     // heads a thread walks; such groups of heads
  unsigned* status;
};

__device__ __forceinline__ const bf16* row_in(const RotaryParams& p, long long m, int h) {
  const int t = h >= p.heads0;
  return p.in[t].x + m * p.in[t].ts + (t ? h - p.heads0 : h) * p.in[t].hs;
}
__device__ __forceinline__ bf16* row_out(const RotaryParams& p, long long m, int h) {
  const int t = h >= p.heads0;
  return p.out[t].y + m * p.out[t].ts + (t ? h - p.heads0 : h) * p.out[t].hs;
}

// Item of a flat index: (token, group of heads, item); 32-bit division where it fits.
__device__ __forceinline__ void split_index(const RotaryParams& p, unsigned long long idx, long long& m, int& g, int& it) {
  if (idx <= 0xffffffffull) {
    const unsigned u = static_cast<unsigned>(idx) / static_cast<unsigned>(p.items);
    it = static_cast<int>(static_cast<unsigned>(idx) - u * p.items);
    const unsigned t = u / static_cast<unsigned>(p.groups);
    g = static_cast<int>(u - t * p.groups);
    m = t;
  } else {
    const unsigned long long u = idx / static_cast<unsigned>(p.items);
    it = static_cast<int>(idx - u * p.items);
    m = static_cast<long long>(u / static_cast<unsigned>(p.groups));
    g = static_cast<int>(u - static_cast<unsigned long long>(m) * p.groups);
  }
}

// How a thread's items look (rot_dim a multiple of 16 but for kScalar):
//   kHalves       two 16-byte pieces of a head: half a rotation apart, or neighbours that pass
//   kInterleaved  one piece
//   kScalar       one pair of features, or one that passes
enum RotaryMode : int { kHalves = 0, kInterleaved = 1, kScalar = 2 };

// At most 64 registers a thread: the loads in flight come from many resident threads (with
// the loads of four heads held by twice as many registers the kernel was 1.2 to 1.7 times
// slower).
template <int MODE>
__global__ void __launch_bounds__(256, 4) rotary_kernel(const __grid_constant__ RotaryParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const unsigned long long total = static_cast<unsigned long long>(p.M) * p.groups * p.items;
  const int half = p.rot.half;
  for (unsigned long long idx = blockIdx.x * 256ull + threadIdx.x; idx < total; idx += 256ull * gridDim.x) {
    long long m;
    int g, it;
    split_index(p, idx, m, g, it);
    const int h0 = g * p.per_group, h1 = min(h0 + p.per_group, p.heads);
    const bool turned = it < p.turned;
    // The position, the first heads' pieces and then the table entries, which wait for the
    // position: two memory latencies in a row instead of three.
    const int at = turned ? __ldg(p.rot.pos + m) : 0;
    if constexpr (MODE == kScalar) {
      const long long tab = turned ? static_cast<long long>(checked_position(p.rot, at, p.status)) * half : 0;
      if (!turned) {
        const int f = 2 * half + it - p.turned;
        for (int h = h0; h < h1; ++h) row_out(p, m, h)[f] = row_in(p, m, h)[f];
        continue;
      }
      const float c = __ldg(p.rot.cos + tab + it), s = p.sign * __ldg(p.rot.sin + tab + it);
      const int fa = p.interleaved ? 2 * it : it, fb = p.interleaved ? 2 * it + 1 : it + half;
      for (int h = h0; h < h1; ++h) {
        const bf16* x = row_in(p, m, h);
        float a, b;
        turn(__bfloat162float(x[fa]), __bfloat162float(x[fb]), c, s, a, b);
        bf16* y = row_out(p, m, h);
        y[fa] = __float2bfloat16_rn(a);
        y[fb] = __float2bfloat16_rn(b);
      }
    } else if constexpr (MODE == kInterleaved) {
      // features [8 it, 8 it + 8), table columns [4 it, 4 it + 4)
      float4 c = make_float4(0.0f, 0.0f, 0.0f, 0.0f), s = c;
      for (int hb = h0; hb < h1; hb += 4) {
        uint4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (hb + i < h1) w[i] = *reinterpret_cast<const uint4*>(row_in(p, m, hb + i) + 8 * it);
        if (turned && hb == h0) {
          const long long tab = static_cast<long long>(checked_position(p.rot, at, p.status)) * half;
          c = __ldg(reinterpret_cast<const float4*>(p.rot.cos + tab) + it);
          s = __ldg(reinterpret_cast<const float4*>(p.rot.sin + tab) + it);
          s.x *= p.sign, s.y *= p.sign, s.z *= p.sign, s.w *= p.sign;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (hb + i >= h1) break;
          if (turned) {
            float x[8];
            unpack8(w[i], x);
            turn(x[0], x[1], c.x, s.x, x[0], x[1]);
            turn(x[2], x[3], c.y, s.y, x[2], x[3]);
            turn(x[4], x[5], c.z, s.z, x[4], x[5]);
            turn(x[6], x[7], c.w, s.w, x[6], x[7]);
            w[i] = pack8(x);
          }
          *reinterpret_cast<uint4*>(row_out(p, m, hb + i) + 8 * it) = w[i];
        }
      }
    } else {
      const int fa = turned ? 8 * it : 2 * half + 16 * (it - p.turned);
      const int fb = turned ? fa + half : fa + 8;
      const bool two = turned || fb < p.dim;              // the last passed piece may be alone
      float c[8], s[8];
      for (int hb = h0; hb < h1; hb += 2) {
        uint4 wa[2], wb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (hb + i >= h1) break;
          const bf16* x = row_in(p, m, hb + i);
          wa[i] = *reinterpret_cast<const uint4*>(x + fa);
          if (two) wb[i] = *reinterpret_cast<const uint4*>(x + fb);
        }
        if (turned && hb == h0) {
          const long long tab = static_cast<long long>(checked_position(p.rot, at, p.status)) * half;
          load8f(p.rot.cos + tab + 8 * it, c);
          load8f(p.rot.sin + tab + 8 * it, s);
#pragma unroll
          for (int e = 0; e < 8; ++e) s[e] *= p.sign;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (hb + i >= h1) break;
          if (turned) {
            const uint32_t va[4] = {wa[i].x, wa[i].y, wa[i].z, wa[i].w}, vb[4] = {wb[i].x, wb[i].y, wb[i].z, wb[i].w};
            uint32_t oa[4], ob[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float a0, a1, b0, b1;
              turn(__uint_as_float(va[e] << 16), __uint_as_float(vb[e] << 16), c[2 * e], s[2 * e], a0, b0);
              turn(__uint_as_float(va[e] & 0xFFFF0000u), __uint_as_float(vb[e] & 0xFFFF0000u), c[2 * e + 1], s[2 * e + 1],
                   a1, b1);
              oa[e] = pack_bf16x2(a0, a1);
              ob[e] = pack_bf16x2(b0, b1);
            }
            wa[i] = make_uint4(oa[0], oa[1], oa[2], oa[3]);
            wb[i] = make_uint4(ob[0], ob[1], ob[2], ob[3]);
          }
          bf16* y = row_out(p, m, hb + i);
          *reinterpret_cast<uint4*>(y + fa) = wa[i];
          if (two) *reinterpret_cast<uint4*>(y + fb) = wb[i];
        }
      }
    }
  }
}

struct ScaledTableParams {
  float* cos;
  float* sin;
  long long npos;
  int half;
  double base;
  int kind;
  double factor, len, low, high, mag;
};

// Angular frequency of table column c under the scaling.
__device__ double scaled_frequency(const ScaledTableParams& p, int c) {
  const double d = 2.0 * p.half;
  const double base = p.kind == LORA_ROPE_NTK ? p.base * pow(p.factor, d / (d - 2.0)) : p.base;
  const double w = pow(base, -2.0 * c / d);
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  if (p.kind == LORA_ROPE_LINEAR) return w / p.factor;
  if (p.kind == LORA_ROPE_YARN) {
    // the (fractional) column that turns r times in len positions: base^(-2c/d) len = 2 pi r
    const double lb = 2.0 * log(p.base);
    double c0 = floor(d * log(p.len / (p.high * kTwoPi)) / lb), c1 = ceil(d * log(p.len / (p.low * kTwoPi)) / lb);
    c0 = fmax(c0, 0.0);
    c1 = fmin(c1, d - 1.0);
    const double g = c1 > c0 ? fmin(fmax((c - c0) / (c1 - c0), 0.0), 1.0) : (c >= c0 ? 1.0 : 0.0);
    return (1.0 - g) * w + g * (w / p.factor);
  }
  if (p.kind == LORA_ROPE_WAVELENGTH) {
    const double turns = p.len * w / kTwoPi;                   // len / wavelength
    const double g = fmin(fmax((turns - p.low) / (p.high - p.low), 0.0), 1.0);
    return g * w + (1.0 - g) * (w / p.factor);
  }
  return w;
}

__global__ void __launch_bounds__(256) scaled_table_kernel(const __grid_constant__ ScaledTableParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const long long total = p.npos * p.half;
  for (long long it = blockIdx.x * 256ll + threadIdx.x; it < total; it += 256ll * gridDim.x) {
    const long long pos = it / p.half;
    const double w = scaled_frequency(p, static_cast<int>(it - pos * p.half));
    double sn, cs;
    sincos(static_cast<double>(pos) * w, &sn, &cs);
    p.cos[it] = static_cast<float>(p.mag * cs);
    p.sin[it] = static_cast<float>(p.mag * sn);
  }
}

}  // namespace lgb

using namespace lgb;

extern "C" lora_status_t lora_rotary(int64_t M, int head_dim, const lora_heads_t* q, const lora_heads_t* yq,
                                     const lora_heads_t* k, const lora_heads_t* yk, const lora_rotary_t* rot,
                                     int inverse, void* ws, size_t ws_bytes, cudaStream_t stream) {
  NvtxRange nvtx_range("lora_rotary");
  const bool two = k != nullptr && k->data != nullptr;
  if (M < 0 || !q || !yq || !rot || (two && !yk)) return LORA_ERR_INVALID_ARG;
  if (M > 0 && (!rot->pos || !q->data || !yq->data || (two && !yk->data))) return LORA_ERR_INVALID_ARG;
  if (head_dim < 1) return LORA_ERR_INVALID_ARG;
  if (head_dim > 1024 || M > kMaxExtent) return LORA_ERR_UNSUPPORTED;
  if (head_dim % 8) return LORA_ERR_ALIGNMENT;
  LGB_TRY(check_rotary(rot, head_dim));
  LGB_TRY(check_heads_in(q));
  LGB_TRY(check_heads_out(yq, M, head_dim));
  if (yq->heads != q->heads) return LORA_ERR_INVALID_ARG;
  if (two) {
    LGB_TRY(check_heads_in(k));
    LGB_TRY(check_heads_out(yk, M, head_dim));
    if (yk->heads != k->heads) return LORA_ERR_INVALID_ARG;
  }
  LGB_TRY(check_ws(ws, ws_bytes, kWsHeader));
  if (M == 0) return LORA_OK;
  RotaryParams p;
  auto same = [](const lora_heads_t* a, const lora_heads_t* b) {
    return a->data == b->data && a->token_stride == b->token_stride && a->head_stride == b->head_stride;
  };
  const lora_heads_t* in[2] = {q, two ? k : q};
  const lora_heads_t* out[2] = {yq, two ? yk : yq};
  bool in_place = true;
  for (int t = 0; t < 2; ++t) {
    p.in[t] = HeadsView{static_cast<const bf16*>(in[t]->data), in[t]->token_stride, in[t]->head_stride};
    p.out[t] = HeadsOut{static_cast<bf16*>(out[t]->data), out[t]->token_stride, out[t]->head_stride};
    in_place = in_place && same(in[t], out[t]);
  }
  p.heads0 = static_cast<int>(q->heads);
  p.heads = p.heads0 + (two ? static_cast<int>(k->heads) : 0);
  p.M = M;
  p.rot = rotary_args(rot);
  p.sign = inverse ? -1.0f : 1.0f;
  p.interleaved = rot->layout == LORA_ROTARY_INTERLEAVED;
  const bool vec = rot->rot_dim % 16 == 0;
  const int passed = head_dim - rot->rot_dim;
  p.dim = head_dim;
  p.turned = !vec ? rot->rot_dim / 2 : p.interleaved ? rot->rot_dim / 8 : rot->rot_dim / 16;
  p.items = p.turned;
  if (!in_place) p.items += static_cast<int>(!vec ? passed : p.interleaved ? passed / 8 : ceil_div(passed, 16));
  p.per_group = heads_per_group(M, p.items, p.heads);
  p.groups = static_cast<int>(ceil_div(p.heads, p.per_group));
  p.status = static_cast<unsigned*>(ws);
  // M, groups and items are below 2^31, 2^17 and 2^10: the product fits 64 bits
  const int64_t blocks = ceil_div(M * p.groups * p.items, 256);
  const unsigned grid = static_cast<unsigned>(blocks < (1 << 30) ? blocks : (1 << 30));
  return launch_counted(!vec ? rotary_kernel<kScalar> : p.interleaved ? rotary_kernel<kInterleaved> : rotary_kernel<kHalves>,
                        dim3(grid), dim3(256), 0, LORA_KIND_ROPE, stream, p);
}

extern "C" lora_status_t lora_rope_table_scaled(float* cos, float* sin, int64_t n_pos, int rot_dim, double base,
                                                const lora_rope_scaling_t* scaling, cudaStream_t stream) {
  NvtxRange nvtx_range("lora_rope_table_scaled");
  const lora_rope_scaling_t* sc = scaling;
  if (!cos || !sin || !sc || n_pos < 1 || rot_dim < 2 || rot_dim % 2 || !(base > 0.0) || !std::isfinite(base))
    return LORA_ERR_INVALID_ARG;
  if (sc->kind < LORA_ROPE_PLAIN || sc->kind > LORA_ROPE_WAVELENGTH || !std::isfinite(sc->magnitude) ||
      sc->magnitude < 0.0)
    return LORA_ERR_INVALID_ARG;
  if (sc->kind != LORA_ROPE_PLAIN && !(sc->factor >= 1.0 && std::isfinite(sc->factor))) return LORA_ERR_INVALID_ARG;
  if (sc->kind == LORA_ROPE_NTK && rot_dim < 4) return LORA_ERR_INVALID_ARG;
  if (sc->kind == LORA_ROPE_YARN && !(base > 1.0)) return LORA_ERR_INVALID_ARG;
  if ((sc->kind == LORA_ROPE_YARN || sc->kind == LORA_ROPE_WAVELENGTH) &&
      !(sc->original_len > 0.0 && std::isfinite(sc->original_len) && sc->low > 0.0 && sc->high > sc->low &&
        std::isfinite(sc->high)))
    return LORA_ERR_INVALID_ARG;
  if (n_pos > kMaxExtent || rot_dim > 65536) return LORA_ERR_UNSUPPORTED;
  if (!aligned(cos, 16) || !aligned(sin, 16)) return LORA_ERR_ALIGNMENT;
  ScaledTableParams p;
  p.cos = cos;
  p.sin = sin;
  p.npos = n_pos;
  p.half = rot_dim / 2;
  p.base = base;
  p.kind = sc->kind;
  p.factor = sc->factor;
  p.len = sc->original_len;
  p.low = sc->low;
  p.high = sc->high;
  p.mag = sc->magnitude > 0.0 ? sc->magnitude : sc->kind == LORA_ROPE_YARN ? 0.1 * std::log(sc->factor) + 1.0 : 1.0;
  int64_t gx = ceil_div(n_pos * p.half, 256);
  gx = gx > 4 * num_sms() ? 4 * num_sms() : gx;
  return launch_counted(scaled_table_kernel, dim3(static_cast<unsigned>(gx)), dim3(256), 0, LORA_KIND_ROPE, stream, p);
}
