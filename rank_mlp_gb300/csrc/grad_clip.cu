// Gradient norms and clipping over lists of tensors: lora_grad_norm, lora_clip_grads and, for
// per-example gradients, lora_clip_examples; include/lora_gb300.h is the contract.
//
// A list travels in the launch's parameters (up to kListMax tensors a launch), so nothing is
// copied to the device ahead of a call and a captured call keeps its own.  Tensors are cut
// into chunks of chunk_of() elements and every block takes an equal share of neighbouring chunks: the host
// writes which tensor it begins with into the parameters, and it walks on from there.  (A block of the examples'
// sum has one chunk and finds its tensor by bisection.)  All is bound by memory.
//
// Sums are f32.  A thread adds up to 64 squares of a batch of loads (32 of f32 tensors), then its batches, one for
// each 10 million (5 million) elements of a launch; a block's threads join in 8 steps, the blocks' results in 3
// and 8.  So a square is rounded fewer than 256 times in lists of up to 10^9 elements a launch, and their sum is off by
// less than 256 * 2^-24 of itself.
#include "serve.cuh"

namespace lgb {

constexpr int kListMax = 920;             // tensors of a launch: 32 KB of parameters with the rest
constexpr int kListFew = 48;              // tensors of a launch with 4 KB of them
constexpr int kClipThreads = 256;
constexpr int kInFlight = 8;              // 16-byte pieces a thread has in flight
constexpr int kListBlocks = 608;          // blocks of a launch at most, whatever the device: four an SM of a GB300

// Elements of a chunk: a 16-byte piece for each thread.
__host__ __device__ constexpr int chunk_of(int f32) { return kClipThreads * (f32 ? 4 : 8); }

struct ListEntry {
  const void* in;
  void* out;
  long long count;
  int first;                              // chunks of the launch before this tensor's
  int f32;
};
template <int CAP>
struct ListArgs {
  int n;
  int chunks;
  uint16_t start[kListBlocks];            // each block's tensor to begin with (launches with shares)
  ListEntry t[CAP];
};

template <int CAP>
struct NormPassArgs {
  float* part;                           // [gridDim.x]
  int inf_norm;
  ListArgs<CAP> list;
};
template <int CAP>
struct ScalePassArgs {
  const float* part;                     // all launches' partial results
  int parts;
  int inf_norm;
  float max_norm;
  float* norm;                            // written by the first launch's first block, or NULL
  ListArgs<CAP> list;
};

// Chunks [c0, c1) of block b out of n.
__host__ __device__ inline int share_begin(int chunks, int b, int n) {
  return static_cast<int>(static_cast<long long>(chunks) * b / n);
}

// Calls f(tensor, a, b) for the spans [a, b) of the block's share of the list, the last ones first
// if `back`.
template <int CAP, typename F>
__device__ __forceinline__ void each_span(const ListArgs<CAP>& l, bool back, F&& f) {
  const int c0 = share_begin(l.chunks, blockIdx.x, gridDim.x), c1 = share_begin(l.chunks, blockIdx.x + 1, gridDim.x);
  if (c0 >= c1) return;
  for (int i = l.start[blockIdx.x]; i >= 0 && i < l.n; i += back ? -1 : 1) {
    const ListEntry& t = l.t[i];
    const long long from = static_cast<long long>(max(c0 - t.first, 0)) * chunk_of(t.f32);
    const long long to = min(static_cast<long long>(c1 - t.first) * chunk_of(t.f32), t.count);
    if (to <= 0) break;                   // (walking on) a tensor behind the share
    if (from >= t.count) break;           // (walking back) one before it
    f(t, from, to);
  }
}

template <typename T>
__device__ __forceinline__ float load_one(const T* p, long long i) {
  if constexpr (sizeof(T) == 4) return p[i]; else return __bfloat162float(p[i]);
}

// Elements [a, b) of a tensor, shared among the block's threads: f(value) for each, f.end() after each
// batch.  The 16-byte pieces of the aligned middle, then the ends, element by element.
template <typename T, typename F>
__device__ __forceinline__ void each_value(const T* base, long long a, long long b, F& f) {
  constexpr int per = 16 / sizeof(T);
  const uintptr_t at = reinterpret_cast<uintptr_t>(base + a);
  const long long lead = min(static_cast<long long>(((16 - (at & 15)) & 15) / sizeof(T)), b - a);
  const long long pieces = (b - a - lead) / per, tail = a + lead + pieces * per;
  const uint4* v = reinterpret_cast<const uint4*>(base + a + lead);
  auto one = [&](uint4 w) {
    if constexpr (sizeof(T) == 4) {
      f(__uint_as_float(w.x)), f(__uint_as_float(w.y)), f(__uint_as_float(w.z)), f(__uint_as_float(w.w));
    } else {
      float x[8];
      unpack8(w, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) f(x[e]);
    }
  };
  for (long long j = threadIdx.x; j < pieces; j += kInFlight * kClipThreads) {
    uint4 w[kInFlight];                   // past the end: the first piece, left out of the sum
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) w[k] = __ldg(v + (j + k * kClipThreads < pieces ? j + k * kClipThreads : 0));
#pragma unroll
    for (int k = 0; k < kInFlight; ++k)
      if (j + k * kClipThreads < pieces) one(w[k]);
    f.end();
  }
  if (threadIdx.x < lead) f(load_one(base, a + threadIdx.x));
  if (tail + threadIdx.x < b) f(load_one(base, tail + threadIdx.x));      // fewer than 8
  f.end();
}
template <typename F>
__device__ __forceinline__ void each_value(const ListEntry& t, long long a, long long b, F& f) {
  if (t.f32) {
    each_value(static_cast<const float*>(t.in), a, b, f);
  } else {
    each_value(static_cast<const bf16*>(t.in), a, b, f);
  }
}

// Sum (or NaN-keeping maximum) of a block's values, in a fixed order; for all threads.  (f64 has no
// place here: the eight blocks of an SM took 6 us for a tree of it.)
__device__ __forceinline__ float block_total(float v, int inf_norm, float* slots) {
  auto join = [&](float a, float b) { return inf_norm ? max_abs_nan(a, b) : a + b; };
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = join(v, __shfl_xor_sync(0xffffffffu, v, d));
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  v = slots[threadIdx.x & (kClipThreads / 32 - 1)];
#pragma unroll
  for (int d = kClipThreads / 64; d > 0; d >>= 1) v = join(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}

// The block's share of a list's squares (or its largest magnitude) for this thread.  Squares are summed
// a batch of loads at a time: chains stay short.
struct Squares {
  float total = 0.0f, batch = 0.0f;
  __device__ __forceinline__ void operator()(float g) { batch = fmaf(g, g, batch); }
  __device__ __forceinline__ void end() { total += batch, batch = 0.0f; }
};
struct Largest {
  float total = 0.0f;
  __device__ __forceinline__ void operator()(float g) { total = max_abs_nan(total, g); }
  __device__ __forceinline__ void end() {}
};

template <int CAP>
__global__ void __launch_bounds__(kClipThreads, 4) list_norm_kernel(const __grid_constant__ NormPassArgs<CAP> p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float slots[kClipThreads / 32];
  float v;
  if (p.inf_norm) {
    Largest f;
    each_span(p.list, false, [&](const ListEntry& t, long long a, long long b) { each_value(t, a, b, f); });
    v = f.total;
  } else {
    Squares f;
    each_span(p.list, false, [&](const ListEntry& t, long long a, long long b) { each_value(t, a, b, f); });
    v = f.total;
  }
  v = block_total(v, p.inf_norm, slots);
  if (threadIdx.x == 0) p.part[blockIdx.x] = v;
}

// The norm of the partial results, in a fixed order; for all threads of the block.
__device__ __forceinline__ float whole_norm(const float* part, int parts, int inf_norm, float* slots) {
  float v = 0.0f;
#pragma unroll 4
  for (int i = threadIdx.x; i < parts; i += kClipThreads) {
    const float o = __ldcg(part + i);
    v = inf_norm ? max_abs_nan(v, o) : v + o;
  }
  v = block_total(v, inf_norm, slots);
  return inf_norm ? v : sqrtf(v);
}

// Elements [a, b) of in times k, into out.  Where the two lie at unlike distances from 16-byte boundaries they go one
// by one: 126 million f32 in 506 us instead of 241, bf16 in 446 instead of 127.
template <typename T>
__device__ __forceinline__ void scale_span(const T* in, T* out, long long a, long long b, float k) {
  constexpr int per = 16 / sizeof(T);
  auto one = [&](long long i) {
    if constexpr (sizeof(T) == 4) out[i] = in[i] * k; else out[i] = __float2bfloat16_rn(__bfloat162float(in[i]) * k);
  };
  const uintptr_t from = reinterpret_cast<uintptr_t>(in + a);
  if ((from ^ reinterpret_cast<uintptr_t>(out + a)) & 15) {          // no common alignment
    for (long long i = a + threadIdx.x; i < b; i += kClipThreads) one(i);
    return;
  }
  const long long lead = min(static_cast<long long>(((16 - (from & 15)) & 15) / sizeof(T)), b - a);
  const long long pieces = (b - a - lead) / per, tail = a + lead + pieces * per;
  const uint4* v = reinterpret_cast<const uint4*>(in + a + lead);
  uint4* o = reinterpret_cast<uint4*>(out + a + lead);
  auto scaled = [&](uint4 w) {
    if constexpr (sizeof(T) == 4) {
      return make_uint4(__float_as_uint(__uint_as_float(w.x) * k), __float_as_uint(__uint_as_float(w.y) * k),
                        __float_as_uint(__uint_as_float(w.z) * k), __float_as_uint(__uint_as_float(w.w) * k));
    } else {
      float x[8];
      unpack8(w, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= k;
      return pack8(x);
    }
  };
  for (long long j = threadIdx.x; j < pieces; j += kInFlight * kClipThreads) {
    uint4 w[kInFlight];
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) w[i] = v[j + i * kClipThreads < pieces ? j + i * kClipThreads : 0];
#pragma unroll
    for (int i = 0; i < kInFlight; ++i)
      if (j + i * kClipThreads < pieces) o[j + i * kClipThreads] = scaled(w[i]);
  }
  if (threadIdx.x < lead) one(a + threadIdx.x);
  if (tail + threadIdx.x < b) one(tail + threadIdx.x);
}

// Walks each share backwards: what the norm's pass read last is still in L2.
template <int CAP>
__global__ void __launch_bounds__(kClipThreads, 4) list_scale_kernel(const __grid_constant__ ScalePassArgs<CAP> p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float slots[kClipThreads / 32];
  const float norm = whole_norm(p.part, p.parts, p.inf_norm, slots);
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.norm != nullptr) *p.norm = norm;
  float k = p.max_norm / (norm + 1e-6f);
  if (isinf(p.max_norm)) k = 1.0f;                  // whatever the norm
  if (k > 1.0f) k = 1.0f;                           // a NaN stays
  each_span(p.list, true, [&](const ListEntry& t, long long a, long long b) {
    if (k == 1.0f && t.in == t.out) return;
    if (t.f32) {
      scale_span(static_cast<const float*>(t.in), static_cast<float*>(t.out), a, b, k);
    } else {
      scale_span(static_cast<const bf16*>(t.in), static_cast<bf16*>(t.out), a, b, k);
    }
  });
}

struct FinishArgs {
  const float* part;
  int parts;
  int inf_norm;
  float* out;
};
__global__ void __launch_bounds__(kClipThreads) norm_finish_kernel(const __grid_constant__ FinishArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float slots[kClipThreads / 32];
  const float norm = whole_norm(p.part, p.parts, p.inf_norm, slots);
  if (threadIdx.x == 0) *p.out = norm;
}

// ---------------------------------------------------------------- per-example gradients

template <int CAP>
struct ExamplePassArgs {
  float* part;                           // [n_examples][parts]
  int parts, part0;                       // partial results of an example, this launch's first
  ListArgs<CAP> list;                     // count: elements of one example; chunks of one example
};
template <int CAP>
struct ExampleSumArgs {
  const float* sq;
  int n_examples;
  int shares;                             // blocks that shared out an example's chunks for its norm; 0: none
  float max_norm, scale;
  ListArgs<CAP> list;
};

// Squared norms: block (x, example).
template <int CAP>
__global__ void __launch_bounds__(kClipThreads, 4) example_norm_kernel(const __grid_constant__ ExamplePassArgs<CAP> p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float slots[kClipThreads / 32];
  const long long e = blockIdx.y;
  Squares f;
  each_span(p.list, false, [&](const ListEntry& t, long long a, long long b) { each_value(t, e * t.count + a, e * t.count + b, f); });
  const float v = block_total(f.total, 0, slots);
  if (threadIdx.x == 0) p.part[e * p.parts + p.part0 + blockIdx.x] = v;
}
// sq[e] of the partial results: a block for each example.
struct ExampleFinishArgs {
  const float* part;
  int parts;
  float* sq;
};
__global__ void __launch_bounds__(kClipThreads) example_finish_kernel(const __grid_constant__ ExampleFinishArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float slots[kClipThreads / 32];
  float v = 0.0f;
  for (int i = threadIdx.x; i < p.parts; i += kClipThreads) v += __ldcg(p.part + static_cast<long long>(blockIdx.x) * p.parts + i);
  v = block_total(v, 0, slots);
  if (threadIdx.x == 0) p.sq[blockIdx.x] = v;
}

// A span of the sum, one chunk: a thread owns a 16-byte piece's elements (or, where rows are not
// aligned, every 256th element) and walks the examples in order, four loads ahead.
template <typename T, int CAP>
__device__ __forceinline__ void sum_span(const ExampleSumArgs<CAP>& p, const ListEntry& t, long long a, long long b, float* keep) {
  constexpr int per = 16 / sizeof(T), kAhead = 4;
  const T* in = static_cast<const T*>(t.in);
  float* out = static_cast<float*>(t.out);
  const bool vec = ((reinterpret_cast<uintptr_t>(in) | static_cast<uintptr_t>(t.count * sizeof(T)) |
                     reinterpret_cast<uintptr_t>(out)) & 15) == 0;
  const long long col = a + per * threadIdx.x;
  const bool mine = col < b;                         // (vec: all of the piece is)
  float acc[per];
#pragma unroll
  for (int j = 0; j < per; ++j) acc[j] = 0.0f;
  for (int e0 = 0; e0 < p.n_examples; e0 += kClipThreads) {
    __syncthreads();
    if (e0 + threadIdx.x < p.n_examples) {
      float k = p.max_norm / sqrtf(__ldcg(p.sq + e0 + threadIdx.x));
      if (isinf(p.max_norm) || k > 1.0f) k = 1.0f;   // a NaN stays
      keep[threadIdx.x] = k;
    }
    __syncthreads();
    const int n = min(kClipThreads, p.n_examples - e0);
    if (vec) {
      const T* src = in + e0 * t.count + (mine ? col : a);
      for (int e = 0; e < n; e += kAhead) {
        uint4 w[kAhead];                          // past the end: the first one's, left out
#pragma unroll
        for (int k = 0; k < kAhead; ++k) w[k] = __ldg(reinterpret_cast<const uint4*>(src + (e + k < n ? e + k : e) * t.count));
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          if (e + k >= n) break;
          float x[8];
          if constexpr (per == 4) {
            x[0] = __uint_as_float(w[k].x), x[1] = __uint_as_float(w[k].y), x[2] = __uint_as_float(w[k].z), x[3] = __uint_as_float(w[k].w);
          } else {
            unpack8(w[k], x);
          }
#pragma unroll
          for (int j = 0; j < per; ++j) acc[j] = fmaf(keep[e + k], x[j], acc[j]);
        }
      }
    } else {
      for (int e = 0; e < n; ++e)
#pragma unroll
        for (int j = 0; j < per; ++j) {
          const long long i = a + threadIdx.x + j * kClipThreads;
          if (i < b) acc[j] = fmaf(keep[e], load_one(in, (e0 + e) * t.count + i), acc[j]);
        }
    }
  }
  if (vec) {
    if (!mine) return;
#pragma unroll
    for (int j = 0; j < per; j += 4)
      *reinterpret_cast<float4*>(out + col + j) = make_float4(p.scale * acc[j], p.scale * acc[j + 1], p.scale * acc[j + 2], p.scale * acc[j + 3]);
  } else {
#pragma unroll
    for (int j = 0; j < per; ++j) {
      const long long i = a + threadIdx.x + j * kClipThreads;
      if (i < b) out[i] = p.scale * acc[j];
    }
  }
}

template <int CAP>
__global__ void __launch_bounds__(kClipThreads, 6) example_sum_kernel(const __grid_constant__ ExampleSumArgs<CAP> p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float keep[kClipThreads];
  // A block has one chunk.  After the norms' launch: the last chunk of each of its shares, then the
  // chunks before them, and so on: what was read last is still in L2.
  int c = blockIdx.x;
  if (p.shares > 0) {
    const int k = blockIdx.x / p.shares, s = blockIdx.x - k * p.shares;
    c = share_begin(p.list.chunks, s + 1, p.shares) - 1 - k;
    if (c < share_begin(p.list.chunks, s, p.shares)) return;
  }
  int lo = 0, hi = p.list.n;                         // its tensor: t[lo].first <= c < t[hi].first
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.list.t[mid].first <= c) lo = mid; else hi = mid;
  }
  const ListEntry& t = p.list.t[lo];
  const long long a = static_cast<long long>(c - t.first) * chunk_of(t.f32), b = min(a + chunk_of(t.f32), t.count);
  if (t.f32) {
    sum_span<float>(p, t, a, b, keep);
  } else {
    sum_span<bf16>(p, t, a, b, keep);
  }
}

// ---------------------------------------------------------------- host

constexpr int64_t kListTensors = int64_t(1) << 20;

static int64_t list_launches(int64_t n) { return n > 0 ? ceil_div(n, kListMax) : 1; }

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
template <int CAP>
static int64_t fill_list(ListArgs<CAP>& list, int64_t i, int64_t n, const lora_tensor_t* in, const lora_tensor_t* out,
                         int64_t parts) {
  list.n = 0;
  int64_t chunks = 0;
  for (; i < n && list.n < CAP; ++i) {
    const int64_t count = in[i].count / parts;
    if (count == 0) continue;
    const int64_t more = ceil_div(count, chunk_of(in[i].dtype == LORA_F32));
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

// The blocks' first tensors (their last ones if `back`) for a launch of `grid` blocks.
template <int CAP>
static void fill_starts(ListArgs<CAP>& list, unsigned grid, bool back) {
  int i = 0;
  for (unsigned b = 0; b < grid; ++b) {
    const int c = back ? share_begin(list.chunks, b + 1, grid) - 1 : share_begin(list.chunks, b, grid);
    while (i + 1 < list.n && list.t[i + 1].first <= c) ++i;
    list.start[b] = static_cast<uint16_t>(i);
  }
}

static unsigned list_grid(int chunks, int most) { return static_cast<unsigned>(chunks < most ? chunks : most); }

// Norms of the list's launches into part; *parts: the number of partial results.
template <int CAP>
static lora_status_t norm_passes(int64_t n, const lora_tensor_t* grads, int norm_type, float* part, int* parts,
                                 cudaStream_t st) {
  *parts = 0;
  NormPassArgs<CAP> p;
  for (int64_t i = 0; i < n;) {
    i = fill_list(p.list, i, n, grads, nullptr, 1);
    if (p.list.n == 0) break;
    const unsigned grid = list_grid(p.list.chunks, kListBlocks);
    fill_starts(p.list, grid, false);
    p.part = part + *parts;
    p.inf_norm = norm_type == LORA_GRAD_NORM_INF;
    LGB_TRY(launch_counted(list_norm_kernel<CAP>, dim3(grid), dim3(kClipThreads), 0, LORA_KIND_CLIP, st, p));
    *parts += static_cast<int>(grid);
  }
  return LORA_OK;
}

template <int CAP>
static lora_status_t norm_only(int64_t n, const lora_tensor_t* grads, int norm_type, float* norm, float* part, cudaStream_t st) {
  FinishArgs f;
  LGB_TRY(norm_passes<CAP>(n, grads, norm_type, part, &f.parts, st));
  f.part = part;
  f.inf_norm = norm_type == LORA_GRAD_NORM_INF;
  f.out = norm;
  return launch_counted(norm_finish_kernel, dim3(1), dim3(kClipThreads), 0, LORA_KIND_CLIP, st, f);
}

template <int CAP>
static lora_status_t clip_passes(int64_t n, const lora_tensor_t* grads, const lora_tensor_t* out, int norm_type, float max_norm,
                                 float* norm, float* part, cudaStream_t st) {
  ScalePassArgs<CAP> p;
  LGB_TRY(norm_passes<CAP>(n, grads, norm_type, part, &p.parts, st));
  p.part = part;
  p.inf_norm = norm_type == LORA_GRAD_NORM_INF;
  p.max_norm = max_norm;
  p.norm = norm;
  int64_t i = 0;
  do {
    i = fill_list(p.list, i, n, grads, out, 1);
    if (p.list.n == 0 && p.norm == nullptr) break;
    // (the grid of the norm's pass: what it read last of a share is read first here)
    const unsigned grid = list_grid(p.list.chunks, kListBlocks);
    fill_starts(p.list, grid, true);
    LGB_TRY(launch_counted(list_scale_kernel<CAP>, dim3(grid > 0 ? grid : 1), dim3(kClipThreads), 0, LORA_KIND_CLIP, st, p));
    p.norm = nullptr;
  } while (i < n);
  return LORA_OK;
}

// Partial results of an example's norm in one launch.
static int example_parts(int64_t n_examples) { return static_cast<int>(ceil_div(kListBlocks, n_examples)); }

template <int CAP>
static lora_status_t example_norms(int64_t n, const lora_tensor_t* grads, int64_t n_examples, float* sq, float* part,
                                   cudaStream_t st) {
  const int per = example_parts(n_examples);
  ExamplePassArgs<CAP> p;
  ExampleFinishArgs f;
  p.part = part;
  // the launches' widths first: a row of partial results holds all of them
  f.parts = 0;
  for (int64_t i = 0; i < n;) {
    i = fill_list(p.list, i, n, grads, nullptr, n_examples);
    f.parts += p.list.n > 0 ? static_cast<int>(list_grid(p.list.chunks, per)) : 0;
  }
  p.parts = f.parts;
  p.part0 = 0;
  for (int64_t i = 0; i < n;) {
    i = fill_list(p.list, i, n, grads, nullptr, n_examples);
    if (p.list.n == 0) break;
    const unsigned grid = list_grid(p.list.chunks, per);
    fill_starts(p.list, grid, false);
    LGB_TRY(launch_counted(example_norm_kernel<CAP>, dim3(grid, static_cast<unsigned>(n_examples)), dim3(kClipThreads), 0,
                           LORA_KIND_CLIP, st, p));
    p.part0 += static_cast<int>(grid);
  }
  f.part = p.part;
  f.sq = sq;
  return launch_counted(example_finish_kernel, dim3(static_cast<unsigned>(n_examples)), dim3(kClipThreads), 0, LORA_KIND_CLIP,
                        st, f);
}

template <int CAP>
static lora_status_t example_sums(int64_t n, const lora_tensor_t* grads, int64_t n_examples, const lora_tensor_t* out,
                                  float max_norm, float scale, const float* sq, bool read, cudaStream_t st) {
  ExampleSumArgs<CAP> p;
  p.sq = sq;
  p.n_examples = static_cast<int>(n_examples);
  p.max_norm = max_norm;
  p.scale = scale;
  for (int64_t i = 0; i < n;) {
    i = fill_list(p.list, i, n, grads, out, n_examples);
    if (p.list.n == 0) break;
    p.shares = read ? static_cast<int>(list_grid(p.list.chunks, example_parts(n_examples))) : 0;
    const int64_t grid = read ? ceil_div(p.list.chunks, p.shares) * p.shares : p.list.chunks;
    LGB_TRY(launch_counted(example_sum_kernel<CAP>, dim3(static_cast<unsigned>(grid)), dim3(kClipThreads), 0, LORA_KIND_CLIP,
                           st, p));
  }
  return LORA_OK;
}

}  // namespace lgb

using namespace lgb;

extern "C" size_t lora_grad_norm_workspace_bytes(int64_t n) {
  if (n < 0 || n > kListTensors) return 0;
  Carve c(nullptr);
  c.take(kWsHeader);
  c.take_n<float>(kListBlocks * list_launches(n));
  return c.off;
}

static lora_status_t check_norm_call(int64_t n, const lora_tensor_t* grads, int norm_type, const float* norm, const void* ws,
                                     size_t ws_bytes) {
  if (n < 0 || (n > 0 && !grads) || !norm || (norm_type != LORA_GRAD_NORM_2 && norm_type != LORA_GRAD_NORM_INF))
    return LORA_ERR_INVALID_ARG;
  if (n > kListTensors) return LORA_ERR_UNSUPPORTED;
  int64_t chunks = 0;
  for (int64_t i = 0; i < n; ++i) {
    LGB_TRY(check_list(1, grads + i, 1));
    chunks += ceil_div(grads[i].count, chunk_of(grads[i].dtype == LORA_F32));
    if (chunks > kMaxExtent) return LORA_ERR_UNSUPPORTED;
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
  float* part = c.take_n<float>(kListBlocks * list_launches(n));
  return n <= kListFew ? norm_only<kListFew>(n, grads, norm_type, norm, part, stream)
                       : norm_only<kListMax>(n, grads, norm_type, norm, part, stream);
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
  float* part = c.take_n<float>(kListBlocks * list_launches(n));
  return n <= kListFew ? clip_passes<kListFew>(n, grads, out, norm_type, max_norm, norm, part, stream)
                       : clip_passes<kListMax>(n, grads, out, norm_type, max_norm, norm, part, stream);
}

extern "C" size_t lora_clip_examples_workspace_bytes(int64_t n, int64_t n_examples) {
  if (n < 0 || n > kListTensors || n_examples < 1 || n_examples > 65535) return 0;
  Carve c(nullptr);
  c.take(kWsHeader);
  c.take_n<float>(n_examples * example_parts(n_examples) * list_launches(n));
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
    chunks += ceil_div(out[i].count, chunk_of(grads[i].dtype == LORA_F32));
    if (chunks > kMaxExtent) return LORA_ERR_UNSUPPORTED;
  }
  if (!aligned(sq_norms, 4)) return LORA_ERR_ALIGNMENT;
  LGB_TRY(check_ws(ws, ws_bytes, lora_clip_examples_workspace_bytes(n, n_examples)));
  if (!norms_given) {
    Carve c(ws);
    c.take(kWsHeader);
    float* part = c.take_n<float>(n_examples * example_parts(n_examples) * list_launches(n));
    LGB_TRY(n <= kListFew ? example_norms<kListFew>(n, grads, n_examples, sq_norms, part, stream)
                          : example_norms<kListMax>(n, grads, n_examples, sq_norms, part, stream));
  }
  return n <= kListFew ? example_sums<kListFew>(n, grads, n_examples, out, max_norm, scale, sq_norms, !norms_given, stream)
                       : example_sums<kListMax>(n, grads, n_examples, out, max_norm, scale, sq_norms, !norms_given, stream);
}
