// Dropout over a ragged batch of flat tensors, its mask from a counter-based
// generator and never stored:
//
//   y_j = u_j < t ? 0 : x_j * 2^16 / (2^16 - t),   t = round(p * 2^16)
//
// u_j is 16 bits of Philox 4x32 with 7 rounds (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", SC 2011): eight elements share
// the block of counter (j / 8, tensor, offset) and key (seed), so that the mask
// depends on the element's place alone and the gradient is the same call on the
// gradients.  What is dropped is 0 whatever it held.
#include "grad_chunks.hpp"

namespace muon {

namespace {

// The four words of a block.
__device__ __forceinline__ void philox(uint32_t (&c)[4], uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int r = 0; r < kDropRounds; ++r) {
    const uint64_t p = static_cast<uint64_t>(0xD2511F53u) * c[0];
    const uint64_t q = static_cast<uint64_t>(0xCD9E8D57u) * c[2];
    const uint32_t c1 = c[1], c3 = c[3];
    c[0] = static_cast<uint32_t>(q >> 32) ^ c1 ^ k0;
    c[1] = static_cast<uint32_t>(q);
    c[2] = static_cast<uint32_t>(p >> 32) ^ c3 ^ k1;
    c[3] = static_cast<uint32_t>(p);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}

struct DropKey {
  uint64_t seed, offset;
  int32_t tensor;
  uint32_t threshold;
  float scale;
};

// Elements j .. j + N - 1 of a tensor, j a multiple of N (4 or 8).
template <int N>
__device__ __forceinline__ void drop(const DropKey& k, int64_t j, float* v) {
  uint32_t c[4] = {static_cast<uint32_t>(j / 8), static_cast<uint32_t>(k.tensor),
                   static_cast<uint32_t>(k.offset), static_cast<uint32_t>(k.offset >> 32)};
  philox(c, static_cast<uint32_t>(k.seed), static_cast<uint32_t>(k.seed >> 32));
  if constexpr (N == 4) {  // the block's first or second half
    c[0] = (j & 4) != 0 ? c[2] : c[0];
    c[1] = (j & 4) != 0 ? c[3] : c[1];
  }
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const uint32_t u = e & 1 ? c[e / 2] >> 16 : c[e / 2] & 0xffffu;
    v[e] = u < k.threshold ? 0.f : v[e] * k.scale;
  }
}

constexpr int kDropSpan = 4096;  // elements of a block

// A lane takes 8 bf16 elements, a whole block of the generator's; where one side is
// fp32, 4, 16 bytes of it, and the block is formed twice.
template <typename Ti, typename To, bool NT>
__device__ __forceinline__ void drop_span(const Ti* x, To* y, int64_t at, int64_t n,
                                          const DropKey& k) {
  constexpr int N = sizeof(Ti) == 2 && sizeof(To) == 2 ? 8 : 4;
  constexpr int kIters = kDropSpan / (kThreads * N);
  if (n == kDropSpan) {
    float v[kIters][N];
#pragma unroll
    for (int u = 0; u < kIters; ++u) {
      const Ti* const from = x + (u * kThreads + threadIdx.x) * N;
      if constexpr (N == 8)
        vec_to_f32<Ti>(NT ? ld16_nt(from) : ld16(from), v[u]);
      else
        load4<Ti, NT>(from, v[u]);
    }
#pragma unroll
    for (int u = 0; u < kIters; ++u) {
      const int i = (u * kThreads + threadIdx.x) * N;
      drop<N>(k, at + i, v[u]);
      if constexpr (N == 4)
        store4<To, NT>(y + i, v[u]);
      else if constexpr (NT)
        st16_nt(y + i, f32_to_vec<To>(v[u]));
      else
        st16(y + i, f32_to_vec<To>(v[u]));
    }
    return;
  }
  for (int64_t i = static_cast<int64_t>(threadIdx.x) * 4; i < n; i += kThreads * 4) {
    float v[4];
    const bool whole = i + 4 <= n;
    if (whole)
      load4<Ti, false>(x + i, v);
    else
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = i + e < n ? Elt<Ti>::to_f32(x[i + e]) : 0.f;
    drop<4>(k, at + i, v);
    if (whole)
      store4<To, false>(y + i, v);
    else
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e < n) y[i + e] = Elt<To>::from_f32(v[e]);
  }
}

}  // namespace

template <bool NT>
__global__ __launch_bounds__(kThreads) void k_dropout(ArgTable, GradCtx ctx, DropArgs p,
                                                      int32_t chunks) {
  constexpr int kPer = static_cast<int>(kGradSpan / kDropSpan);  // blocks per chunk
  const int32_t b = block_number();
  if (b / kPer >= chunks) return;
  const Chunk c = find_chunk(ctx, b / kPer);
  const int64_t off = static_cast<int64_t>(b % kPer) * kDropSpan;
  const int64_t left = c.n - off, n = left < kDropSpan ? left : kDropSpan;
  if (n <= 0) return;
  DropKey k;
  k.seed = p.rng != nullptr ? load_const(p.rng) : p.seed;
  k.offset = p.rng != nullptr ? load_const(p.rng + 1) : p.offset;
  k.tensor = c.tensor;
  k.threshold = p.threshold;
  k.scale = p.scale;
  const int64_t at = c.base + off;
  const uint16_t* xh = static_cast<const uint16_t*>(c.g) + at;
  const float* xf = static_cast<const float*>(c.g) + at;
  uint16_t* yh = static_cast<uint16_t*>(c.out) + at;
  float* yf = static_cast<float*>(c.out) + at;
  if (c.in_bf16) {
    if (c.out_bf16)
      drop_span<uint16_t, uint16_t, NT>(xh, yh, at, n, k);
    else
      drop_span<uint16_t, float, NT>(xh, yf, at, n, k);
  } else {
    if (c.out_bf16)
      drop_span<float, uint16_t, NT>(xf, yh, at, n, k);
    else
      drop_span<float, float, NT>(xf, yf, at, n, k);
  }
}

namespace {

// Bytes read and written from which they pass the caches by.  A call by itself is
// faster that way from 48 MB on (bf16, inputs from memory: 48 MB 11.1 us, without the
// hint 12.8; 128 MB 23.8 and 25.6; 256 MB 44 and 48), but one that reads the result next
// finds it in the caches without it (with a copy of the result: 32 MB 16.0 us, without
// 14.3; 64 MB 26.9 and 24.5; 128 MB 48.5 and 44.3; 192 MB 69 and 70; 256 MB 91 and 118).
constexpr int64_t kNtDropBytes = 64ll << 20;

}  // namespace

hipError_t launch_dropout(const ArgTable& t, const GradCtx& c, int32_t chunks, const DropArgs& p,
                          int64_t bytes) {
  if (chunks <= 0) return hipSuccess;
  const dim3 grid = block_grid(chunks * (kGradSpan / kDropSpan));
  if (bytes > kNtDropBytes)
    hipLaunchKernelGGL(k_dropout<true>, grid, dim3(kThreads), 0, c.stream, t, c, p, chunks);
  else
    hipLaunchKernelGGL(k_dropout<false>, grid, dim3(kThreads), 0, c.stream, t, c, p, chunks);
  return hipGetLastError();
}

}  // namespace muon
