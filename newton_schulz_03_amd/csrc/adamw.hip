// Fused AdamW step over a ragged batch of flat tensors (the parameters that
// Muon does not cover: norms, routers, embeddings).
//
// Per element, in fp32 (p and g stored as T, the moments m and v as fp32):
//   p <- p * (1 - lr * wd)
//   m <- beta1 * m + (1 - beta1) * g
//   v <- beta2 * v + (1 - beta2) * g^2
//   p <- p - (lr / (1 - beta1^t)) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
// SCALED: g is first multiplied by a factor in device memory (the clip factor
// of the global norm), so that clipping costs no pass of its own.
// Bandwidth-bound (22 bytes an element in bf16, 28 in fp32): each block reads
// its whole span (p, g, m, v) before the first store.  Every load and store of a
// wave covers whole 128-byte lines, 4 elements a lane, with the nontemporal
// hint: 223 bf16 tensors of 175.5 M elements in 639 us, 6.0 TB/s (633 to 675 us by
// where the tensors lie).  (8 elements a lane, which covers each fp32 line in two
// halves: 705 us with the hint, 731 without; 4 elements without the hint 710; more
// spans per block are slower, 687 us with two.)  Blocks find their tensor through
// the prefix table, in one round of loads for up to kAdamScan tensors.
#include "device_common.hpp"

namespace muon {

namespace {

constexpr int kAdamVec = 4;  // elements per thread: 16 bytes of each moment
constexpr int64_t kAdamSpan = static_cast<int64_t>(kThreads) * kAdamVec;  // per block
// Most tensors for the scan of the prefixes, which every block of 1024 elements
// reads whole (2000 tensors of 5000 elements, bf16: 68 us with it, 61 with the search;
// 700: 37 both ways).
constexpr int kAdamScan = 1024;

// Four elements: 16 bytes of fp32, 8 of bf16.
template <typename T>
__device__ __forceinline__ void load_vec(const T* p, float* v) {
  if constexpr (sizeof(T) == 2) {
    const u32x2_t w = __builtin_nontemporal_load((const GLOBAL_AS u32x2_t*)(p));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    vec_to_f32<T>(ld16_nt(p), v);
  }
}

template <typename T>
__device__ __forceinline__ void store_vec(T* p, const float* v) {
  if constexpr (sizeof(T) == 2) {
    u32x2_t w;
    w[0] = Elt<uint16_t>::pack2(v[0], v[1]);
    w[1] = Elt<uint16_t>::pack2(v[2], v[3]);
    __builtin_nontemporal_store(w, (GLOBAL_AS u32x2_t*)(p));
  } else {
    st16_nt(p, f32_to_vec<T>(v));
  }
}

__device__ __forceinline__ void adamw_update(const AdamParams& a, float& p, float g, float& m,
                                             float& v) {
  p *= a.decay;
  m = a.beta1 * m + a.one_minus_beta1 * g;
  v = a.beta2 * v + a.one_minus_beta2 * (g * g);
  const float denom = sqrtf(v) * a.inv_bc2_sqrt + a.eps;
  p -= a.step_size * (m / denom);
}

template <typename T, bool SCALED>
__global__ __launch_bounds__(kThreads) void k_adamw(ArgTable, AdamCtx c, AdamParams a,
                                                    int32_t nblocks) {
  __shared__ int slot;
  const int32_t b = block_number();
  if (b >= nblocks) return;
  const float gs = SCALED ? *a.g_scale : 1.f;
  const char* const table = table_base(c.table);
  const int32_t* const prefix = reinterpret_cast<const int32_t*>(table + c.prefix_off);
  const int j = __builtin_amdgcn_readfirstlane(locate_matrix(prefix, c.batch, b, &slot, kAdamScan));
  const AdamDesc d = load_const(reinterpret_cast<const AdamDesc*>(table) + j);
  const int64_t numel = d.numel;
  const int64_t base = static_cast<int64_t>(b - load_const(prefix + j)) * kAdamSpan;
  T* __restrict__ pp = static_cast<T*>(d.p) + base;
  const T* __restrict__ gp = static_cast<const T*>(d.g) + base;
  float* __restrict__ mp = d.m + base;
  float* __restrict__ vp = d.v + base;
  if (base + kAdamSpan <= numel) {
    float p[kAdamVec], g[kAdamVec], m[kAdamVec], v[kAdamVec];
    const int off = threadIdx.x * kAdamVec;
    load_vec<T>(pp + off, p);
    load_vec<T>(gp + off, g);
    load_vec<float>(mp + off, m);
    load_vec<float>(vp + off, v);
#pragma unroll
    for (int e = 0; e < kAdamVec; ++e)
      adamw_update(a, p[e], SCALED ? gs * g[e] : g[e], m[e], v[e]);
    store_vec<T>(pp + off, p);
    store_vec<float>(mp + off, m);
    store_vec<float>(vp + off, v);
  } else {
    // the tensor's last, partial span: element by element
    const int64_t n = numel - base;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) {
      float p = Elt<T>::to_f32(pp[i]);
      float m = mp[i], v = vp[i];
      const float g = Elt<T>::to_f32(gp[i]);
      adamw_update(a, p, SCALED ? gs * g : g, m, v);
      pp[i] = Elt<T>::from_f32(p);
      mp[i] = m;
      vp[i] = v;
    }
  }
}

}  // namespace

int64_t adamw_blocks(int64_t numel) {
  return (numel + kAdamSpan - 1) / kAdamSpan;
}

namespace {

template <typename T, bool SCALED>
hipError_t run_adamw(const ArgTable& t, const AdamCtx& c, int32_t nblocks, const AdamParams& a) {
  hipLaunchKernelGGL((k_adamw<T, SCALED>), block_grid(nblocks), dim3(kThreads), 0, c.stream,
                     t, c, a, nblocks);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_adamw(const AdamCtx& c, int32_t nblocks, bool is_bf16, const AdamParams& a) {
  if (nblocks <= 0) return hipSuccess;
  const ArgTable& t = *c.args;
  if (a.g_scale != nullptr)
    return is_bf16 ? run_adamw<uint16_t, true>(t, c, nblocks, a) : run_adamw<float, true>(t, c, nblocks, a);
  return is_bf16 ? run_adamw<uint16_t, false>(t, c, nblocks, a) : run_adamw<float, false>(t, c, nblocks, a);
}

}  // namespace muon
