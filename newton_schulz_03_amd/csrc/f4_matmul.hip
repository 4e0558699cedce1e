// Rows times matrices of 4-bit weights with group scales (f4_operand.hip):
//
//   y[p][r] = sum_k x[p][k] W_e[r][k],   offsets[e] <= p < offsets[e + 1]
//
// bf16 rows, fp32 sums, rounded once.  A weight's value is a bf16 number, so that
// the products are exact in fp32: two weights and their scale are one conversion
// (v_cvt_scalef32_pk_bf16_fp4), and four 16x16x32 matrix instructions take a tile
// of 16 weight rows x 128 columns times up to 16 rows of x.
//
// Bound by the weights' bytes.  The waves of a block share the contracted side of
// one tile row; their sums are joined in a fixed order through LDS.
#include "device_common.hpp"

namespace muon {

namespace {

constexpr int kF4Waves = 8;

// The bf16 pairs that a word of four bytes stands for.
__device__ __forceinline__ bf16x8_t weights8(uint32_t q, float scale) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 0);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 1);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 2);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 3);
  return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// 2^(byte - 127); byte 255 is a NaN.
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7fc00000u : byte << 23);
}

// Eight values of a row from column k on, zero past its end.
template <bool VEC>
__device__ __forceinline__ bf16x8_t row8(const uint16_t* x, int32_t k, int32_t cols) {
  if constexpr (VEC) {
    u32x4_t v = {0, 0, 0, 0};
    if (k < cols) v = ld16(x + k);
    return __builtin_bit_cast(bf16x8_t, v);
  } else {
    uint16_t v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = k + e < cols ? x[k + e] : 0;
    bf16x8_t r;
    __builtin_memcpy(&r, v, 16);
    return r;
  }
}

}  // namespace

template <typename To, bool VEC>
__global__ __launch_bounds__(64 * kF4Waves) void k_f4_matmul(F4ProdArgs a) {
  __shared__ __attribute__((aligned(16))) f32x4_t part[kF4Waves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int32_t e = 0;
  int64_t p0 = 0, p1 = a.m;
  if (a.active != nullptr) {
    if (static_cast<int32_t>(blockIdx.y) >= a.active[0]) return;
    e = a.active[1 + blockIdx.y];
    if (e < 0 || e >= a.experts) return;
    p0 = max(a.offsets[e], 0);
    p1 = min(static_cast<int64_t>(a.offsets[e + 1]), a.m);
  }
  const int64_t strip = static_cast<int64_t>(e) * a.rtiles + blockIdx.x;
  const char* const q = a.q + (strip * a.ktiles * 64 + lane) * 16;
  const uint32_t* const s = reinterpret_cast<const uint32_t*>(a.s) +
                            (strip * ((a.ktiles + 3) / 4) * 16 + (lane & 15)) * 4;
  const int32_t t0 = a.ktiles * wave / kF4Waves, t1 = a.ktiles * (wave + 1) / kF4Waves;
  for (; p0 < p1; p0 += 16) {
    // lanes past the last row take that row's: their results are not stored
    int64_t row = min(p0 + (lane & 15), p1 - 1);
    if (a.slots != nullptr) {
      row = a.slots[row] / a.top_k;
      if (row < 0 || row >= a.x_rows) row = 0;
    }
    const uint16_t* const x = static_cast<const uint16_t*>(a.x) + row * a.cols;
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    for (int32_t t = t0; t < t1; ++t) {
      const u32x4_t w = ld16(q + static_cast<int64_t>(t) * 1024);
      const uint32_t sc = s[(t / 4) * 64 + t % 4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bf16x8_t b = row8<VEC>(x, t * kF4Tile + 32 * i + 8 * (lane >> 4), a.cols);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            weights8(w[i], scale_of(sc >> (8 * i) & 255u)), b, acc, 0, 0, 0);
      }
    }
    part[wave][lane] = acc;
    __syncthreads();
    if (wave == 0) {
      f32x4_t sum = part[0][lane];
#pragma unroll
      for (int w = 1; w < kF4Waves; ++w) sum += part[w][lane];
      const int64_t p = p0 + (lane & 15);
      const int32_t r = blockIdx.x * 16 + 4 * (lane >> 4);
      if (p < p1) {
        To* const y = static_cast<To*>(a.y) + p * a.rows + r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (r + i < a.rows) y[i] = Elt<To>::from_f32(sum[i]);
      }
    }
    __syncthreads();
  }
}

hipError_t launch_f4_matmul(const F4ProdArgs& a, bool is_bf16, hipStream_t s) {
  if (a.m <= 0 || a.rows <= 0) return hipSuccess;
  const int64_t most = a.active != nullptr ? (a.m < a.experts ? a.m : a.experts) : 1;
  const dim3 grid(a.rtiles, static_cast<uint32_t>(most)), block(64 * kF4Waves);
  const bool vec = a.cols % 8 == 0;
  if (is_bf16) {
    if (vec)
      hipLaunchKernelGGL((k_f4_matmul<uint16_t, true>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((k_f4_matmul<uint16_t, false>), grid, block, 0, s, a);
  } else {
    if (vec)
      hipLaunchKernelGGL((k_f4_matmul<float, true>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((k_f4_matmul<float, false>), grid, block, 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace muon
