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
#include "grad_chunks.hpp"

namespace muon {

namespace {

constexpr int kNormBatch = 4;  // 16-byte loads per thread in flight

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

template <typename K, bool NT, typename T>
__device__ __forceinline__ void add_chunk(const T* g, int64_t n, typename K::acc_t& acc) {
  constexpr int V = Elt<T>::kVec;
  constexpr int kStep = kThreads * V * kNormBatch;
  const int64_t whole = n / kStep * kStep;
  for (int64_t i = 0; i < whole; i += kStep) {
    u32x4_t x[kNormBatch];
#pragma unroll
    for (int u = 0; u < kNormBatch; ++u) {
      const T* const at = g + i + (u * kThreads + threadIdx.x) * V;
      x[u] = NT ? ld16_nt(at) : ld16(at);
    }
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

// The factor from up to 64 partials, joined in a fixed order by every wave for
// itself; block 0 stores the norm and the factor.
template <typename K>
__device__ __forceinline__ float factor_of_few(const GradNormArgs& p, int32_t n) {
  const int lane = threadIdx.x & 63;
  typename K::acc_t v = lane < n ? static_cast<const typename K::acc_t*>(p.partials)[lane] : 0;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = K::join(v, __shfl_xor(v, off, 64));
  GradNormArgs q = p;
  float r[2];
  q.result = r;
  finish_norm<K>(v, q);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    p.result[0] = r[0];
    p.result[1] = r[1];
  }
  return r[1];
}

}  // namespace

// Block b joins chunks b, b + grid, ...: neighbouring blocks read neighbouring
// chunks.  A single block finishes the norm itself.
template <typename K, bool NT>
__global__ __launch_bounds__(kThreads) void k_grad_norm(ArgTable, GradCtx ctx, GradNormArgs p) {
  __shared__ typename K::acc_t scratch[kThreads / 64];
  typename K::acc_t acc = 0;
  for (int32_t c = blockIdx.x; c < p.chunks; c += gridDim.x) {
    const Chunk k = find_chunk(ctx, c);
    if (k.in_bf16)
      add_chunk<K, NT>(static_cast<const uint16_t*>(k.g) + k.base, k.n, acc);
    else
      add_chunk<K, NT>(static_cast<const float*>(k.g) + k.base, k.n, acc);
  }
  acc = block_join<K>(acc, scratch);
  if (threadIdx.x != 0) return;
  if (gridDim.x == 1 && !p.keep_partials)
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

constexpr int kScaleVec = 4;    // elements per thread and iteration: 16 bytes of fp32, 8 of bf16
constexpr int kScaleIters = 4;  // iterations per block
constexpr int64_t kScaleSpan = static_cast<int64_t>(kThreads) * kScaleVec * kScaleIters;

template <typename Ti, typename To, bool NT>
__device__ __forceinline__ void scale_span(const Ti* g, To* o, int64_t n, float s) {
  if (n >= kScaleSpan) {
    float x[kScaleIters][kScaleVec];
#pragma unroll
    for (int u = 0; u < kScaleIters; ++u)
      load4<Ti, NT>(g + (u * kThreads + threadIdx.x) * kScaleVec, x[u]);
#pragma unroll
    for (int u = 0; u < kScaleIters; ++u) {
#pragma unroll
      for (int e = 0; e < kScaleVec; ++e) x[u][e] *= s;
      store4<To, NT>(o + (u * kThreads + threadIdx.x) * kScaleVec, x[u]);
    }
    return;
  }
  for (int64_t i = static_cast<int64_t>(threadIdx.x) * kScaleVec; i < n; i += kThreads * kScaleVec) {
    if (i + kScaleVec <= n) {
      float x[kScaleVec];
      load4<Ti, false>(g + i, x);
#pragma unroll
      for (int e = 0; e < kScaleVec; ++e) x[e] *= s;
      store4<To, false>(o + i, x);
    } else {
      for (int64_t k = i; k < n; ++k) o[k] = Elt<To>::from_f32(Elt<Ti>::to_f32(g[k]) * s);
    }
  }
}

}  // namespace

// One block per kScaleSpan elements of a chunk.  A factor of exactly 1 leaves a
// tensor scaled in place as it is.  nparts > 0: the norm's partials are joined
// here (a call of few blocks saves the launch that would join them).
template <bool NT>
__global__ __launch_bounds__(kThreads) void k_grad_scale(ArgTable, GradCtx ctx, const float* scale,
                                                         GradNormArgs p, int32_t kind,
                                                         int32_t nparts, int32_t chunks) {
  constexpr int kPer = static_cast<int>(kGradSpan / kScaleSpan);  // blocks per chunk
  const int32_t b = block_number();
  if (b / kPer >= chunks) return;
  float s;
  if (nparts == 0)
    s = *scale;
  else
    s = kind == 0 ? factor_of_few<SumSq>(p, nparts) : factor_of_few<MaxAbs>(p, nparts);
  const Chunk k = find_chunk(ctx, b / kPer);
  const int64_t off = static_cast<int64_t>(b % kPer) * kScaleSpan;
  const int64_t left = k.n - off, n = left < kScaleSpan ? left : kScaleSpan;
  if (n <= 0 || (s == 1.f && k.out == k.g)) return;
  const uint16_t* gh = static_cast<const uint16_t*>(k.g) + k.base + off;
  const float* gf = static_cast<const float*>(k.g) + k.base + off;
  uint16_t* oh = static_cast<uint16_t*>(k.out) + k.base + off;
  float* of = static_cast<float*>(k.out) + k.base + off;
  if (k.in_bf16) {
    if (k.out_bf16)
      scale_span<uint16_t, uint16_t, NT>(gh, oh, n, s);
    else
      scale_span<uint16_t, float, NT>(gh, of, n, s);
  } else {
    if (k.out_bf16)
      scale_span<float, uint16_t, NT>(gf, oh, n, s);
    else
      scale_span<float, float, NT>(gf, of, n, s);
  }
}

namespace {

// The hint pays once the data is larger than the caches keep: norms of 20 fp32
// tensors of 100003 elements (8 MB) 5.8 us without it and 6.8 with, of 74 bf16
// router gradients (349 MB) 64 and 58 us; scaling 201 MB into 101 MB 48 and 46 us,
// 1.2 GB into 0.6 GB 315 and 285 us.
constexpr int64_t kNtNormBytes = 64ll << 20, kNtScaleBytes = 256ll << 20;

int32_t norm_grid(int32_t chunks) {
  return chunks < 1 ? 1 : chunks < kNormBlocks ? chunks : kNormBlocks;
}

template <typename K>
hipError_t run_norm(const ArgTable& t, const GradCtx& c, const GradNormArgs& p, int64_t bytes) {
  const int32_t grid = norm_grid(p.chunks);
  if (bytes > kNtNormBytes)
    hipLaunchKernelGGL((k_grad_norm<K, true>), dim3(grid), dim3(kThreads), 0, c.stream, t, c, p);
  else
    hipLaunchKernelGGL((k_grad_norm<K, false>), dim3(grid), dim3(kThreads), 0, c.stream, t, c, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || grid == 1 || p.keep_partials) return e;
  hipLaunchKernelGGL(k_grad_finish<K>, dim3(1), dim3(kThreads), 0, c.stream, p, grid);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grad_norm(const ArgTable& t, const GradCtx& c, const GradNormArgs& p,
                            int32_t kind, int64_t bytes) {
  return kind == 0 ? run_norm<SumSq>(t, c, p, bytes) : run_norm<MaxAbs>(t, c, p, bytes);
}

bool grad_few_blocks(int32_t chunks) { return chunks > 0 && chunks <= 64; }

hipError_t launch_grad_scale(const ArgTable& t, const GradCtx& c, int32_t chunks,
                             const float* scale, const GradNormArgs* joined, int32_t kind,
                             int64_t bytes) {
  if (chunks <= 0) return hipSuccess;
  const dim3 grid = block_grid(chunks * (kGradSpan / kScaleSpan));
  const GradNormArgs p = joined != nullptr ? *joined : GradNormArgs{};
  const int32_t nparts = joined != nullptr ? norm_grid(chunks) : 0;
  if (bytes > kNtScaleBytes)
    hipLaunchKernelGGL(k_grad_scale<true>, grid, dim3(kThreads), 0, c.stream, t, c, scale, p, kind,
                       nparts, chunks);
  else
    hipLaunchKernelGGL(k_grad_scale<false>, grid, dim3(kThreads), 0, c.stream, t, c, scale, p, kind,
                       nparts, chunks);
  return hipGetLastError();
}

}  // namespace muon
