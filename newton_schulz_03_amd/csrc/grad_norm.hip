// The global norm of a ragged batch of gradients, the clip factor, and the
// gradients times that factor.
//
//   n = sqrt(sum_i sum_j g_ij^2)   or   max_ij |g_ij|
//   s = min(1, max_norm / (n + eps)),   out_ij = s * g_ij  rounded to out's type
//
// Squares and sums are held in double: every finite fp32 gradient has its
// square there (fp32 loses |g| > 1.8e19 and < 1e-23), and the order of the sum
// does not show in the fp32 result.  Partials go through the workspace, one per
// block, and are summed in a fixed order: no atomics, the same bits every time.
// The maximum is taken over the bit patterns of |g|, in whose order infinities
// and then NaNs come last, so that a NaN reaches the norm.
//
// Bandwidth-bound: each block requests a whole part of its chunk before it
// uses the first value.
#include "device_common.hpp"

namespace muon {

namespace {

constexpr int kNormBatch = 4;  // 16-byte loads per thread in flight

// One chunk (kGradSpan elements) of a tensor, or what is left of it.
struct Chunk {
  int j;         // the tensor
  int64_t base;  // first element
  int64_t n;     // elements, 1 .. kGradSpan
};

// The chunk's tensor by binary search: prefix[j] <= c < prefix[j + 1].
template <typename Tab>
__device__ __forceinline__ Chunk find_chunk(const Tab& t, int32_t c) {
  int lo = 0, hi = t.batch();
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.prefix(mid) <= c)
      lo = mid;
    else
      hi = mid;
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  Chunk k;
  k.j = lo;
  k.base = static_cast<int64_t>(c - t.prefix(lo)) * kGradSpan;
  const int64_t left = t.desc(lo).numel - k.base;
  k.n = left < kGradSpan ? left : kGradSpan;
  return k;
}

// The table in the workspace, or among the kernel's arguments.
struct TabMem {
  GradCtx c;
  __device__ __forceinline__ int batch() const { return c.batch; }
  __device__ __forceinline__ int32_t prefix(int j) const { return load_const(c.prefix + j); }
  __device__ __forceinline__ GradDesc desc(int j) const { return load_const(c.desc + j); }
};
struct TabArg {
  GradInline t;
  __device__ __forceinline__ int batch() const { return t.batch; }
  __device__ __forceinline__ int32_t prefix(int j) const { return t.prefix[j]; }
  __device__ __forceinline__ GradDesc desc(int j) const { return t.desc[j]; }
};

struct SumSq {
  typedef double acc_t;
  static __device__ __forceinline__ void add(acc_t& a, float v) {
    const double d = static_cast<double>(v);
    a = __builtin_fma(d, d, a);
  }
  static __device__ __forceinline__ acc_t join(acc_t a, acc_t b) { return a + b; }
  static __device__ __forceinline__ double norm(acc_t a) { return sqrt(a); }
};
struct MaxAbs {
  typedef uint32_t acc_t;
  static __device__ __forceinline__ void add(acc_t& a, float v) {
    const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
    a = b > a ? b : a;
  }
  static __device__ __forceinline__ acc_t join(acc_t a, acc_t b) { return a > b ? a : b; }
  static __device__ __forceinline__ double norm(acc_t a) {
    return static_cast<double>(__uint_as_float(a));
  }
};

// Joins one value per thread of the block; every thread gets the result.
template <typename K>
__device__ __forceinline__ typename K::acc_t block_join(typename K::acc_t v,
                                                        typename K::acc_t* scratch) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = K::join(v, __shfl_xor(v, off, 64));
  if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = v;
  __syncthreads();
  v = scratch[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) v = K::join(v, scratch[w]);
  __syncthreads();
  return v;
}

template <typename K, typename T>
__device__ __forceinline__ void add_chunk(const T* g, int64_t n, typename K::acc_t& acc) {
  constexpr int V = Elt<T>::kVec;
  constexpr int kStep = kThreads * V * kNormBatch;
  const int64_t whole = n / kStep * kStep;
  for (int64_t i = 0; i < whole; i += kStep) {
    u32x4_t x[kNormBatch];
#pragma unroll
    for (int u = 0; u < kNormBatch; ++u) x[u] = ld16_nt(g + i + (u * kThreads + threadIdx.x) * V);
#pragma unroll
    for (int u = 0; u < kNormBatch; ++u) {
      float v[V];
      vec_to_f32<T>(x[u], v);
#pragma unroll
      for (int e = 0; e < V; ++e) K::add(acc, v[e]);
    }
  }
  int64_t i = whole + threadIdx.x * V;
  for (; i + V <= n; i += kThreads * V) {
    float v[V];
    vec_to_f32<T>(ld16(g + i), v);
#pragma unroll
    for (int e = 0; e < V; ++e) K::add(acc, v[e]);
  }
  for (; i < n; ++i) K::add(acc, Elt<T>::to_f32(g[i]));  // at most V - 1, in one thread
}

// The norm and the clip factor from the joined value.
template <typename K>
__device__ __forceinline__ void finish_norm(typename K::acc_t a, const GradNormArgs& p) {
  const double n = K::norm(a);
  double s = 1.0;
  if (p.clip) {
    const double d = n + static_cast<double>(p.eps);
    const double r = d == 0.0 ? 1.0 : static_cast<double>(p.max_norm) / d;
    s = r < 1.0 || r != r ? r : 1.0;  // NaN stays
  }
  p.result[0] = static_cast<float>(n);
  p.result[1] = static_cast<float>(s);
}

}  // namespace

// Block b joins chunks b, b + grid, ...: neighbouring blocks read neighbouring
// chunks.  A single block finishes the norm itself.
template <typename K, typename Tab>
__global__ __launch_bounds__(kThreads) void k_grad_norm(Tab tab, GradNormArgs p) {
  __shared__ typename K::acc_t scratch[kThreads / 64];
  typename K::acc_t acc = 0;
  for (int32_t c = blockIdx.x; c < p.chunks; c += gridDim.x) {
    const Chunk k = find_chunk(tab, c);
    const GradDesc d = tab.desc(k.j);
    if (d.in_bf16)
      add_chunk<K>(static_cast<const uint16_t*>(d.g) + k.base, k.n, acc);
    else
      add_chunk<K>(static_cast<const float*>(d.g) + k.base, k.n, acc);
  }
  acc = block_join<K>(acc, scratch);
  if (threadIdx.x != 0) return;
  if (gridDim.x == 1)
    finish_norm<K>(acc, p);
  else
    static_cast<typename K::acc_t*>(p.partials)[blockIdx.x] = acc;
}

// One block joins the partials in a fixed order.
template <typename K>
__global__ __launch_bounds__(kThreads) void k_grad_finish(GradNormArgs p, int32_t n) {
  __shared__ typename K::acc_t scratch[kThreads / 64];
  const typename K::acc_t* part = static_cast<const typename K::acc_t*>(p.partials);
  typename K::acc_t acc = 0;
  for (int32_t i = threadIdx.x; i < n; i += kThreads) acc = K::join(acc, part[i]);
  acc = block_join<K>(acc, scratch);
  if (threadIdx.x == 0) finish_norm<K>(acc, p);
}

namespace {

template <typename Ti, typename To>
__device__ __forceinline__ void scale_chunk(const Ti* g, To* o, int64_t n, float s) {
  constexpr int V = 8;
  const int64_t whole = n / V * V;
  for (int64_t i = static_cast<int64_t>(threadIdx.x) * V; i < whole; i += kThreads * V) {
    float v[V];
    vec_to_f32<Ti>(ld16(g + i), v);
    if constexpr (sizeof(Ti) == 4) vec_to_f32<Ti>(ld16(g + i + 4), v + 4);
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] *= s;
    st16(o + i, f32_to_vec<To>(v));
    if constexpr (sizeof(To) == 4) st16(o + i + 4, f32_to_vec<To>(v + 4));
  }
  const int64_t i = whole + threadIdx.x;
  if (i < n) o[i] = Elt<To>::from_f32(Elt<Ti>::to_f32(g[i]) * s);
}

}  // namespace

// One block per chunk.  A factor of exactly 1 leaves a tensor scaled in place
// as it is.
template <typename Tab>
__global__ __launch_bounds__(kThreads) void k_grad_scale(Tab tab, const float* scale) {
  const float s = *scale;
  const Chunk k = find_chunk(tab, blockIdx.x);
  const GradDesc d = tab.desc(k.j);
  if (s == 1.f && d.out == d.g) return;
  const uint16_t* gh = static_cast<const uint16_t*>(d.g) + k.base;
  const float* gf = static_cast<const float*>(d.g) + k.base;
  uint16_t* oh = static_cast<uint16_t*>(d.out) + k.base;
  float* of = static_cast<float*>(d.out) + k.base;
  if (d.in_bf16) {
    if (d.out_bf16)
      scale_chunk(gh, oh, k.n, s);
    else
      scale_chunk(gh, of, k.n, s);
  } else {
    if (d.out_bf16)
      scale_chunk(gf, oh, k.n, s);
    else
      scale_chunk(gf, of, k.n, s);
  }
}

namespace {

template <typename K, typename Tab>
hipError_t norm_launches(const Tab& tab, const GradNormArgs& p, hipStream_t s) {
  const int32_t grid = p.chunks < kNormBlocks ? (p.chunks > 0 ? p.chunks : 1) : kNormBlocks;
  hipLaunchKernelGGL((k_grad_norm<K, Tab>), dim3(grid), dim3(kThreads), 0, s, tab, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || grid == 1) return e;
  hipLaunchKernelGGL(k_grad_finish<K>, dim3(1), dim3(kThreads), 0, s, p, grid);
  return hipGetLastError();
}

template <typename Tab>
hipError_t norm_of(const Tab& tab, const GradNormArgs& p, int32_t kind, hipStream_t s) {
  return kind == 0 ? norm_launches<SumSq>(tab, p, s) : norm_launches<MaxAbs>(tab, p, s);
}

template <typename Tab>
hipError_t scale_of(const Tab& tab, int32_t chunks, const float* scale, hipStream_t s) {
  if (chunks <= 0) return hipSuccess;
  hipLaunchKernelGGL(k_grad_scale<Tab>, dim3(chunks), dim3(kThreads), 0, s, tab, scale);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grad_norm(const GradTable& t, const GradNormArgs& p, int32_t kind,
                            hipStream_t s) {
  return t.in_args ? norm_of(TabArg{t.args}, p, kind, s) : norm_of(TabMem{t.mem}, p, kind, s);
}

hipError_t launch_grad_scale(const GradTable& t, int32_t chunks, const float* scale,
                             hipStream_t s) {
  return t.in_args ? scale_of(TabArg{t.args}, chunks, scale, s)
                   : scale_of(TabMem{t.mem}, chunks, scale, s);
}

}  // namespace muon
