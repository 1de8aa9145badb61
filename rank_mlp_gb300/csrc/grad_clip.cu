// Gradient norms and clipping over lists of tensors: lora_grad_norm, lora_clip_grads and, for
// per-example gradients, lora_clip_examples; include/lora_gb300.h is the contract.
//
// A list travels in the launch's parameters (up to kListMax tensors a launch), so nothing is
// copied to the device ahead of a call and a captured call keeps its own.  Tensors are cut
// into chunks of kChunk elements; blocks take chunks in turn and find a chunk's tensor by
// bisection of the chunks' running count.  All is bound by memory.
#include "serve.cuh"

namespace lgb {

constexpr int kListMax = 960;             // tensors of a launch: 30 KB of parameters
constexpr int kChunk = 8192;              // elements
constexpr int kClipThreads = 256;

struct ListEntry {
  const void* in;
  void* out;
  long long count;
  int first;                              // chunks of the launch before this tensor's
  int f32;
};
struct ListArgs {
  ListEntry t[kListMax];
  int n;
  int chunks;
};

struct NormPassArgs {
  ListArgs list;
  double* part;                           // [gridDim.x]
  int inf_norm;
};
struct ScalePassArgs {
  ListArgs list;
  const double* part;                     // all launches' partial results
  int parts;
  int inf_norm;
  float max_norm;
  float* norm;                            // written by the first launch's first block, or NULL
};

// The tensor that holds chunk c.
__device__ __forceinline__ int find_tensor(const ListArgs& l, int c) {
  int lo = 0, hi = l.n;                   // t[lo].first <= c < t[hi].first
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (l.t[mid].first <= c) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ float load_one(const void* p, long long i, int f32) {
  return f32 ? static_cast<const float*>(p)[i] : __bfloat162float(static_cast<const bf16*>(p)[i]);
}

// Elements [a, b) of a tensor, shared among the block's threads: f(value) for each.  The
// 16-byte pieces of the aligned middle, then the ends, element by element.
template <typename F>
__device__ __forceinline__ void each_value(const void* base, long long a, long long b, int f32, F&& f) {
  const int size = f32 ? 4 : 2, per = 16 / size;
  const uintptr_t at = reinterpret_cast<uintptr_t>(base) + a * size;
  const long long lead = min(static_cast<long long>(((16 - (at & 15)) & 15) / size), b - a);
  const long long pieces = (b - a - lead) / per, tail = a + lead + pieces * per;
  const uint4* v = reinterpret_cast<const uint4*>(at + lead * size);
#pragma unroll 4
  for (long long j = threadIdx.x; j < pieces; j += kClipThreads) {
    const uint4 w = __ldg(v + j);
    if (f32) {
      f(__uint_as_float(w.x)), f(__uint_as_float(w.y)), f(__uint_as_float(w.z)), f(__uint_as_float(w.w));
    } else {
      float x[8];
      unpack8(w, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) f(x[e]);
    }
  }
  if (threadIdx.x < lead) f(load_one(base, a + threadIdx.x, f32));
  if (tail + threadIdx.x < b) f(load_one(base, tail + threadIdx.x, f32));      // fewer than 8
}

// Sum (or NaN-keeping maximum) of a block's values, in a fixed order; for all threads.
__device__ __forceinline__ double block_total(double v, int inf_norm, double* slots) {
  auto join = [&](double a, double b) {
    return !inf_norm ? a + b : static_cast<double>(max_abs_nan(static_cast<float>(a), static_cast<float>(b)));
  };
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = join(v, __shfl_xor_sync(0xffffffffu, v, d));
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  v = slots[0];
#pragma unroll
  for (int k = 1; k < kClipThreads / 32; ++k) v = join(v, slots[k]);
  return v;
}

__global__ void __launch_bounds__(kClipThreads) list_norm_kernel(const __grid_constant__ NormPassArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ double slots[kClipThreads / 32];
  float acc = 0.0f;
  for (int c = blockIdx.x; c < p.list.chunks; c += gridDim.x) {
    const ListEntry& t = p.list.t[find_tensor(p.list, c)];
    const long long a = static_cast<long long>(c - t.first) * kChunk, b = min(a + kChunk, t.count);
    if (p.inf_norm) {
      each_value(t.in, a, b, t.f32, [&](float g) { acc = max_abs_nan(acc, g); });
    } else {
      each_value(t.in, a, b, t.f32, [&](float g) { acc = fmaf(g, g, acc); });
    }
  }
  const double v = block_total(acc, p.inf_norm, slots);
  if (threadIdx.x == 0) p.part[blockIdx.x] = v;
}

// The norm of the partial results, in a fixed order; for all threads of the block.
__device__ __forceinline__ float whole_norm(const double* part, int parts, int inf_norm, double* slots) {
  double v = 0.0;
  for (int i = threadIdx.x; i < parts; i += kClipThreads) {
    const double o = __ldcg(part + i);
    v = !inf_norm ? v + o : static_cast<double>(max_abs_nan(static_cast<float>(v), static_cast<float>(o)));
  }
  v = block_total(v, inf_norm, slots);
  return inf_norm ? static_cast<float>(v) : static_cast<float>(sqrt(v));
}

__global__ void __launch_bounds__(kClipThreads) list_scale_kernel(const __grid_constant__ ScalePassArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ double slots[kClipThreads / 32];
  const float norm = whole_norm(p.part, p.parts, p.inf_norm, slots);
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.norm != nullptr) *p.norm = norm;
  float k = p.max_norm / (norm + 1e-6f);
  if (isinf(p.max_norm)) k = 1.0f;                  // whatever the norm
  if (k > 1.0f) k = 1.0f;                           // a NaN stays
  for (int c = blockIdx.x; c < p.list.chunks; c += gridDim.x) {
    const ListEntry& t = p.list.t[find_tensor(p.list, c)];
    if (k == 1.0f && t.in == t.out) continue;
    const long long a = static_cast<long long>(c - t.first) * kChunk, b = min(a + kChunk, t.count);
    const int size = t.f32 ? 4 : 2, per = 16 / size;
    const uintptr_t from = reinterpret_cast<uintptr_t>(t.in) + a * size, to = reinterpret_cast<uintptr_t>(t.out) + a * size;
    auto one = [&](long long i) {
      if (t.f32) {
        static_cast<float*>(t.out)[i] = static_cast<const float*>(t.in)[i] * k;
      } else {
        static_cast<bf16*>(t.out)[i] = __float2bfloat16_rn(__bfloat162float(static_cast<const bf16*>(t.in)[i]) * k);
      }
    };
    if ((from ^ to) & 15) {                         // no common alignment
      for (long long i = a + threadIdx.x; i < b; i += kClipThreads) one(i);
      continue;
    }
    const long long lead = min(static_cast<long long>(((16 - (from & 15)) & 15) / size), b - a);
    const long long pieces = (b - a - lead) / per, tail = a + lead + pieces * per;
    const uint4* v = reinterpret_cast<const uint4*>(from + lead * size);
    uint4* o = reinterpret_cast<uint4*>(to + lead * size);
#pragma unroll 4
    for (long long j = threadIdx.x; j < pieces; j += kClipThreads) {
      uint4 w = v[j];
      if (t.f32) {
        w.x = __float_as_uint(__uint_as_float(w.x) * k);
        w.y = __float_as_uint(__uint_as_float(w.y) * k);
        w.z = __float_as_uint(__uint_as_float(w.z) * k);
        w.w = __float_as_uint(__uint_as_float(w.w) * k);
      } else {
        float x[8];
        unpack8(w, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= k;
        w = pack8(x);
      }
      o[j] = w;
    }
    if (threadIdx.x < lead) one(a + threadIdx.x);
    if (tail + threadIdx.x < b) one(tail + threadIdx.x);
  }
}

struct FinishArgs {
  const double* part;
  int parts;
  int inf_norm;
  float* out;
};
__global__ void __launch_bounds__(kClipThreads) norm_finish_kernel(const __grid_constant__ FinishArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ double slots[kClipThreads / 32];
  const float norm = whole_norm(p.part, p.parts, p.inf_norm, slots);
  if (threadIdx.x == 0) *p.out = norm;
}

// ---------------------------------------------------------------- per-example gradients

struct ExamplePassArgs {
  ListArgs list;                          // count: elements of one example; chunks of one example
  double* part;                           // [n_examples][gridDim.x of all launches]
  int parts, part0;                       // partial results of an example, this launch's first
};
struct ExampleSumArgs {
  ListArgs list;                          // chunks of kSumChunk elements of one example
  const float* sq;
  int n_examples;
  float max_norm, scale;
};
constexpr int kSumChunk = 8 * kClipThreads;

// Squared norms: block (x, example).
__global__ void __launch_bounds__(kClipThreads) example_norm_kernel(const __grid_constant__ ExamplePassArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ double slots[kClipThreads / 32];
  const long long e = blockIdx.y;
  float acc = 0.0f;
  for (int c = blockIdx.x; c < p.list.chunks; c += gridDim.x) {
    const ListEntry& t = p.list.t[find_tensor(p.list, c)];
    const long long a = static_cast<long long>(c - t.first) * kChunk, b = min(a + kChunk, t.count);
    each_value(t.in, e * t.count + a, e * t.count + b, t.f32, [&](float g) { acc = fmaf(g, g, acc); });
  }
  const double v = block_total(acc, 0, slots);
  if (threadIdx.x == 0) p.part[e * p.parts + p.part0 + blockIdx.x] = v;
}
// sq[e] of the partial results: a block for each example.
struct ExampleFinishArgs {
  const double* part;
  int parts;
  float* sq;
};
__global__ void __launch_bounds__(kClipThreads) example_finish_kernel(const __grid_constant__ ExampleFinishArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ double slots[kClipThreads / 32];
  double v = 0.0;
  for (int i = threadIdx.x; i < p.parts; i += kClipThreads) v += __ldcg(p.part + static_cast<long long>(blockIdx.x) * p.parts + i);
  v = block_total(v, 0, slots);
  if (threadIdx.x == 0) p.sq[blockIdx.x] = static_cast<float>(v);
}

// One thread owns eight neighbouring elements (or, where rows are not aligned, every 256th
// element) of the result and walks the examples in order.
__global__ void __launch_bounds__(kClipThreads) example_sum_kernel(const __grid_constant__ ExampleSumArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float keep[kClipThreads];
  for (int c = blockIdx.x; c < p.list.chunks; c += gridDim.x) {
    const ListEntry& t = p.list.t[find_tensor(p.list, c)];
    const long long a = static_cast<long long>(c - t.first) * kSumChunk, b = min(a + kSumChunk, t.count);
    const int per = t.f32 ? 4 : 8, size = t.f32 ? 4 : 2;
    const bool vec = ((reinterpret_cast<uintptr_t>(t.in) | static_cast<uintptr_t>(t.count * size) |
                       reinterpret_cast<uintptr_t>(t.out)) & 15) == 0;
    float acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
    const long long col = a + 8 * threadIdx.x;
    for (int e0 = 0; e0 < p.n_examples; e0 += kClipThreads) {
      __syncthreads();
      if (e0 + threadIdx.x < p.n_examples) {
        float k = p.max_norm / sqrtf(__ldcg(p.sq + e0 + threadIdx.x));
        if (isinf(p.max_norm) || k > 1.0f) k = 1.0f;                 // a NaN stays
        keep[threadIdx.x] = k;
      }
      __syncthreads();
      const int n = min(kClipThreads, p.n_examples - e0);
      if (vec) {
        if (col >= b) continue;                                      // count is a multiple of per
        const char* src = static_cast<const char*>(t.in) + (e0 * t.count + col) * size;
        const bool two = t.f32 && col + 4 < b;
#pragma unroll 4
        for (int e = 0; e < n; ++e) {
          const uint4 w = __ldg(reinterpret_cast<const uint4*>(src + e * t.count * size));
          if (t.f32) {
            const float x[4] = {__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w)};
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] = fmaf(keep[e], x[j], acc[j]);
            if (two) {
              const uint4 u = __ldg(reinterpret_cast<const uint4*>(src + e * t.count * size) + 1);
              const float z[4] = {__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w)};
#pragma unroll
              for (int j = 0; j < 4; ++j) acc[4 + j] = fmaf(keep[e], z[j], acc[4 + j]);
            }
          } else {
            float x[8];
            unpack8(w, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] = fmaf(keep[e], x[j], acc[j]);
          }
        }
      } else {
        for (int e = 0; e < n; ++e)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const long long i = a + threadIdx.x + j * kClipThreads;
            if (i < b) acc[j] = fmaf(keep[e], load_one(t.in, (e0 + e) * t.count + i, t.f32), acc[j]);
          }
      }
    }
    float* out = static_cast<float*>(t.out);
    if (vec) {
      if (col < b) {
        *reinterpret_cast<float4*>(out + col) = make_float4(p.scale * acc[0], p.scale * acc[1], p.scale * acc[2], p.scale * acc[3]);
        if (per == 8 || col + 4 < b)
          *reinterpret_cast<float4*>(out + col + 4) = make_float4(p.scale * acc[4], p.scale * acc[5], p.scale * acc[6], p.scale * acc[7]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const long long i = a + threadIdx.x + j * kClipThreads;
        if (i < b) out[i] = p.scale * acc[j];
      }
    }
  }
}

// ---------------------------------------------------------------- host

constexpr int64_t kListTensors = int64_t(1) << 20;
constexpr int kNormBlocks = 1216;         // partial results of a launch, whatever the device

static int64_t list_launches(int64_t n) { return ceil_div(n, kListMax); }

static lora_status_t check_list(int64_t n, const lora_tensor_t* t, int64_t parts) {
  for (int64_t i = 0; i < n; ++i) {
    if (t[i].count < 0 || (t[i].dtype != LORA_BF16 && t[i].dtype != LORA_F32) || (t[i].count > 0 && !t[i].data))
      return LORA_ERR_INVALID_ARG;
    if (t[i].count % parts) return LORA_ERR_INVALID_ARG;
    // chunks are counted in 32 bits, in all tensors of a launch
    if (t[i].count > (int64_t(1) << 40)) return LORA_ERR_UNSUPPORTED;
    if (!aligned(t[i].data, t[i].dtype == LORA_F32 ? 4 : 2)) return LORA_ERR_ALIGNMENT;
  }
  return LORA_OK;
}

// Fills `list` with tensors [i, ...) of the call; returns the next one.  Empty tensors and
// those past the launch's room are left out.
static int64_t fill_list(ListArgs& list, int64_t i, int64_t n, const lora_tensor_t* in, const lora_tensor_t* out,
                         int64_t parts, int chunk) {
  list.n = 0;
  int64_t chunks = 0;
  for (; i < n && list.n < kListMax; ++i) {
    const int64_t count = in[i].count / parts;
    if (count == 0) continue;
    const int64_t more = ceil_div(count, chunk);
    if (list.n > 0 && chunks + more > kMaxExtent) break;
    ListEntry& t = list.t[list.n++];
    t.in = in[i].data;
    t.out = out != nullptr ? out[i].data : in[i].data;
    t.count = count;
    t.first = static_cast<int>(chunks);
    t.f32 = in[i].dtype == LORA_F32;
    chunks += more;
  }
  list.chunks = static_cast<int>(chunks);
  return i;
}

static unsigned list_grid(int chunks, int most) { return static_cast<unsigned>(chunks < most ? chunks : most); }

// Norms of the list's launches into part; returns the number of partial results.
static lora_status_t norm_passes(int64_t n, const lora_tensor_t* grads, int norm_type, double* part, int* parts,
                                 cudaStream_t st) {
  *parts = 0;
  NormPassArgs p;
  for (int64_t i = 0; i < n;) {
    i = fill_list(p.list, i, n, grads, nullptr, 1, kChunk);
    if (p.list.n == 0) break;
    const unsigned grid = list_grid(p.list.chunks, kNormBlocks);
    p.part = part + *parts;
    p.inf_norm = norm_type == LORA_GRAD_NORM_INF;
    LGB_TRY(launch_counted(list_norm_kernel, dim3(grid), dim3(kClipThreads), 0, LORA_KIND_CLIP, st, p));
    *parts += static_cast<int>(grid);
  }
  return LORA_OK;
}

}  // namespace lgb

using namespace lgb;

extern "C" size_t lora_grad_norm_workspace_bytes(int64_t n) {
  if (n < 0 || n > kListTensors) return 0;
  Carve c(nullptr);
  c.take(kWsHeader);
  // a launch holds kListMax tensors, fewer where their chunks pass 2^31 (one of the largest each)
  c.take_n<double>(kNormBlocks * (list_launches(n) + 1));
  return c.off;
}

static lora_status_t check_norm_call(int64_t n, const lora_tensor_t* grads, int norm_type, const float* norm, const void* ws,
                                     size_t ws_bytes) {
  if (n < 0 || (n > 0 && !grads) || !norm || (norm_type != LORA_GRAD_NORM_2 && norm_type != LORA_GRAD_NORM_INF))
    return LORA_ERR_INVALID_ARG;
  if (n > kListTensors) return LORA_ERR_UNSUPPORTED;
  int64_t elements = 0;
  for (int64_t i = 0; i < n; ++i) {
    LGB_TRY(check_list(1, grads + i, 1));
    elements += ceil_div(grads[i].count, kChunk);
    if (elements > kMaxExtent) return LORA_ERR_UNSUPPORTED;
  }
  if (!aligned(norm, 4)) return LORA_ERR_ALIGNMENT;
  return check_ws(ws, ws_bytes, lora_grad_norm_workspace_bytes(n));
}

extern "C" lora_status_t lora_grad_norm(int64_t n, const lora_tensor_t* grads, int norm_type, float* norm, void* ws,
                                        size_t ws_bytes, cudaStream_t stream) {
  NvtxRange nvtx_range("lora_grad_norm");
  LGB_TRY(check_norm_call(n, grads, norm_type, norm, ws, ws_bytes));
  Carve c(ws);
  c.take(kWsHeader);
  FinishArgs f;
  double* part = c.take_n<double>(kNormBlocks * (list_launches(n) + 1));
  LGB_TRY(norm_passes(n, grads, norm_type, part, &f.parts, stream));
  f.part = part;
  f.inf_norm = norm_type == LORA_GRAD_NORM_INF;
  f.out = norm;
  return launch_counted(norm_finish_kernel, dim3(1), dim3(kClipThreads), 0, LORA_KIND_CLIP, stream, f);
}

extern "C" lora_status_t lora_clip_grads(int64_t n, const lora_tensor_t* grads, const lora_tensor_t* out, int norm_type,
                                         float max_norm, float* norm, void* ws, size_t ws_bytes, cudaStream_t stream) {
  NvtxRange nvtx_range("lora_clip_grads");
  if (!(max_norm > 0.0f)) return LORA_ERR_INVALID_ARG;
  LGB_TRY(check_norm_call(n, grads, norm_type, norm, ws, ws_bytes));
  if (out != nullptr) {
    LGB_TRY(check_list(n, out, 1));
    for (int64_t i = 0; i < n; ++i)
      if (out[i].count != grads[i].count || out[i].dtype != grads[i].dtype) return LORA_ERR_INVALID_ARG;
  }
  Carve c(ws);
  c.take(kWsHeader);
  double* part = c.take_n<double>(kNormBlocks * (list_launches(n) + 1));
  int parts = 0;
  LGB_TRY(norm_passes(n, grads, norm_type, part, &parts, stream));
  ScalePassArgs p;
  p.part = part;
  p.parts = parts;
  p.inf_norm = norm_type == LORA_GRAD_NORM_INF;
  p.max_norm = max_norm;
  p.norm = norm;
  int64_t i = 0;
  do {
    i = fill_list(p.list, i, n, grads, out, 1, kChunk);
    if (p.list.n == 0 && p.norm == nullptr) break;
    const unsigned grid = list_grid(p.list.chunks, 8 * num_sms());
    LGB_TRY(launch_counted(list_scale_kernel, dim3(grid > 0 ? grid : 1), dim3(kClipThreads), 0, LORA_KIND_CLIP, stream, p));
    p.norm = nullptr;
  } while (i < n);
  return LORA_OK;
}

// Partial results of an example's norm in one launch.
static int example_parts(int64_t n_examples) {
  const int64_t want = ceil_div(kNormBlocks, n_examples);
  return static_cast<int>(want);
}

extern "C" size_t lora_clip_examples_workspace_bytes(int64_t n, int64_t n_examples) {
  if (n < 0 || n > kListTensors || n_examples < 1 || n_examples > 65535) return 0;
  Carve c(nullptr);
  c.take(kWsHeader);
  c.take_n<double>(n_examples * example_parts(n_examples) * (list_launches(n) + 1));
  return c.off;
}

extern "C" lora_status_t lora_clip_examples(int64_t n, const lora_tensor_t* grads, int64_t n_examples,
                                            const lora_tensor_t* out, float max_norm, float scale, float* sq_norms,
                                            int norms_given, void* ws, size_t ws_bytes, cudaStream_t stream) {
  NvtxRange nvtx_range("lora_clip_examples");
  if (n < 0 || (n > 0 && (!grads || !out)) || n_examples < 1 || !sq_norms || !(max_norm > 0.0f) || !std::isfinite(scale))
    return LORA_ERR_INVALID_ARG;
  if (n > kListTensors || n_examples > 65535) return LORA_ERR_UNSUPPORTED;
  LGB_TRY(check_list(n, grads, n_examples));
  LGB_TRY(check_list(n, out, 1));
  int64_t chunks = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (out[i].dtype != LORA_F32 || out[i].count != grads[i].count / n_examples) return LORA_ERR_INVALID_ARG;
    chunks += ceil_div(out[i].count, kSumChunk);
    if (chunks > kMaxExtent) return LORA_ERR_UNSUPPORTED;
  }
  if (!aligned(sq_norms, 4)) return LORA_ERR_ALIGNMENT;
  LGB_TRY(check_ws(ws, ws_bytes, lora_clip_examples_workspace_bytes(n, n_examples)));
  if (!norms_given) {
    Carve c(ws);
    c.take(kWsHeader);
    const int per = example_parts(n_examples);
    ExamplePassArgs p;
    ExampleFinishArgs f;
    p.part = c.take_n<double>(n_examples * per * (list_launches(n) + 1));
    // the launches' widths first: a row of partial results holds all of them
    f.parts = 0;
    for (int64_t i = 0; i < n;) {
      i = fill_list(p.list, i, n, grads, nullptr, n_examples, kChunk);
      f.parts += p.list.n > 0 ? static_cast<int>(list_grid(p.list.chunks, per)) : 0;
    }
    p.parts = f.parts;
    p.part0 = 0;
    for (int64_t i = 0; i < n;) {
      i = fill_list(p.list, i, n, grads, nullptr, n_examples, kChunk);
      if (p.list.n == 0) break;
      const unsigned grid = list_grid(p.list.chunks, per);
      LGB_TRY(launch_counted(example_norm_kernel, dim3(grid, static_cast<unsigned>(n_examples)), dim3(kClipThreads), 0,
                             LORA_KIND_CLIP, stream, p));
      p.part0 += static_cast<int>(grid);
    }
    f.part = p.part;
    f.sq = sq_norms;
    LGB_TRY(launch_counted(example_finish_kernel, dim3(static_cast<unsigned>(n_examples)), dim3(kClipThreads), 0,
                           LORA_KIND_CLIP, stream, f));
  }
  ExampleSumArgs p;
  p.sq = sq_norms;
  p.n_examples = static_cast<int>(n_examples);
  p.max_norm = max_norm;
  p.scale = scale;
  for (int64_t i = 0; i < n;) {
    i = fill_list(p.list, i, n, grads, out, n_examples, kSumChunk);
    if (p.list.n == 0) break;
    const unsigned grid = static_cast<unsigned>(p.list.chunks);
    LGB_TRY(launch_counted(example_sum_kernel, dim3(grid), dim3(kClipThreads), 0, LORA_KIND_CLIP, stream, p));
  }
  return LORA_OK;
}
