// Block-scaled e4m3 operands of a ragged batch of matrices (F8QuantDesc in
// muon_internal.hpp): the matrix, its transpose, or both from one read.
//
// A block (1 x 128 along the contracted side, or 128 x 128) shares one scale
// 2^e: the smallest power of two, at least 2^-127, with the block's largest
// finite magnitude at most 448 * 2^e (448: e4m3's largest value), so that
// nothing saturates.  An element x is stored as the e4m3 rounding (to nearest
// even) of x * 2^-e; the product x * 2^-e is exact in fp32 wherever it is not
// below e4m3's smallest step.  Infinities and NaNs become NaN and take no part
// in the scale.
//
// Bandwidth-bound: one block per 128 x 128 tile reads it once, 16 bytes a lane
// and every load issued first, and writes whole 128-byte rows of values; the
// transpose goes through 16 KiB of LDS as bytes.
#include "device_common.hpp"

namespace muon {

namespace {

constexpr int kQ = kF8Block;

// Exponent of the scale of a block with largest finite magnitude amax = m * 2^E,
// 1 <= m < 2; 448 = 1.75 * 2^8.  Zero and subnormal blocks take -127.
__device__ __forceinline__ int scale_exp(uint32_t amax_bits) {
  const int field = static_cast<int>(amax_bits >> 23);
  if (field == 0) return -127;
  const int e = field - 127 - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -127 ? -127 : e;  // at most 120
}
__device__ __forceinline__ float inv_scale(int e) {  // 2^-e, e in [-127, 120]
  return __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}

__device__ __forceinline__ uint32_t finite_abs(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Four values as e4m3 bytes.  x - x is 0 for a finite value and NaN otherwise.
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  int x = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  x = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, x, true);
  return static_cast<uint32_t>(x);
}
__device__ __forceinline__ float scaled(float v, float inv) {
  const float s = v * inv;
  return (__float_as_uint(s) & 0x7f800000u) == 0x7f800000u ? __uint_as_float(0x7fc00000u) : s;
}

}  // namespace

// Thread t holds the 8 x 8 sub-block of rows 8 (t / 16) .. + 7 and columns
// 8 (t % 16) .. + 7 of the tile: 16 lanes cover a row's 128 columns, and the
// 8 rows of a column are 8 bytes of the transpose.
template <typename T, bool SQUARE>
__global__ __launch_bounds__(kThreads) void k_f8_quantize(F8QuantCtx c) {
  __shared__ __attribute__((aligned(16))) uint8_t tr[kQ * 144];  // [column][row], pitch 144
  __shared__ uint32_t part[4][kQ];
  __shared__ __attribute__((aligned(16))) uint8_t sc[kQ];
  __shared__ int slot;
  const int j = __builtin_amdgcn_readfirstlane(locate_matrix(c.prefix, c.batch, blockIdx.x, &slot));
  const F8QuantDesc d = load_const(c.desc + j);
  const int32_t t = blockIdx.x - load_const(c.prefix + j);
  const int32_t tpr = (d.cols + kQ - 1) / kQ;
  const int32_t r0 = t / tpr * kQ, c0 = t % tpr * kQ;
  const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;

  float v[8][8];
  const int32_t col = c0 + 8 * cg;
  constexpr int V = Elt<T>::kVec;
  const bool vec = d.cols % V == 0 && col + 8 <= d.cols;
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int32_t row = r0 + 8 * rg + p;
    const T* x = static_cast<const T*>(d.x) + static_cast<int64_t>(row) * d.cols + col;
    if (vec && row < d.rows) {
#pragma unroll
      for (int h = 0; h < 8 / V; ++h) vec_to_f32<T>(ld16_nt(x + h * V), v[p] + h * V);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[p][e] = row < d.rows && col + e < d.cols ? Elt<T>::to_f32(x[e]) : 0.f;
    }
  }

  int esq = -127;  // SQUARE: the tile's exponent
  if constexpr (SQUARE) {
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < 8; ++p)
#pragma unroll
      for (int e = 0; e < 8; ++e) m = umax(m, finite_abs(v[p][e]));
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = umax(m, __shfl_xor(m, off, 64));
    if (lane == 0) part[wave][0] = m;
    __syncthreads();
    esq = scale_exp(umax(umax(part[0][0], part[1][0]), umax(part[2][0], part[3][0])));
  }

  if (d.q != nullptr) {
    const int32_t kp = tpr * kQ;
    const int32_t rp = (d.rows + 15) / 16 * 16;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      int e = esq;
      if constexpr (!SQUARE) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = umax(m, finite_abs(v[p][i]));
#pragma unroll
        for (int off = 8; off >= 1; off >>= 1) m = umax(m, __shfl_xor(m, off, 64));
        e = scale_exp(m);
      }
      const float inv = inv_scale(e);
      const int32_t row = r0 + 8 * rg + p;
      if (cg == 0) sc[8 * rg + p] = row < d.rows ? static_cast<uint8_t>(e + 127) : 0;
      if (row < d.rows) {
        u32x2_t w;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[h] = pack4(scaled(v[p][4 * h], inv), scaled(v[p][4 * h + 1], inv),
                       scaled(v[p][4 * h + 2], inv), scaled(v[p][4 * h + 3], inv));
        *reinterpret_cast<u32x2_t*>(d.q + static_cast<int64_t>(row) * kp + col) = w;
      }
    }
    __syncthreads();
    if (threadIdx.x < kQ / 16 && r0 + 16 * static_cast<int>(threadIdx.x) < rp)
      st16(d.s + static_cast<int64_t>(c0 / kQ) * rp + r0 + 16 * threadIdx.x,
           *reinterpret_cast<const u32x4_t*>(sc + 16 * threadIdx.x));
    __syncthreads();
  }

  if (d.qt != nullptr) {
    const int32_t kp = (d.rows + kQ - 1) / kQ * kQ;
    const int32_t rp = (d.cols + 15) / 16 * 16;
    if constexpr (!SQUARE) {
      uint32_t m[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        m[e] = 0;
#pragma unroll
        for (int p = 0; p < 8; ++p) m[e] = umax(m[e], finite_abs(v[p][e]));
        m[e] = umax(m[e], __shfl_xor(m[e], 16, 64));
        m[e] = umax(m[e], __shfl_xor(m[e], 32, 64));
      }
      if (lane < 16) {
#pragma unroll
        for (int e = 0; e < 8; ++e) part[wave][8 * cg + e] = m[e];
      }
      __syncthreads();
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      int ex = esq;
      const int cc = 8 * cg + e;
      if constexpr (!SQUARE)
        ex = scale_exp(umax(umax(part[0][cc], part[1][cc]), umax(part[2][cc], part[3][cc])));
      const float inv = inv_scale(ex);
      if (rg == 0) sc[cc] = c0 + cc < d.cols ? static_cast<uint8_t>(ex + 127) : 0;
      u32x2_t w;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        w[h] = pack4(scaled(v[4 * h][e], inv), scaled(v[4 * h + 1][e], inv),
                     scaled(v[4 * h + 2][e], inv), scaled(v[4 * h + 3][e], inv));
      // 16-byte chunk i of a column sits at i ^ (cg / 2): the 16 lanes of a row
      // group then spread over the banks
      *reinterpret_cast<u32x2_t*>(tr + cc * 144 + (((rg >> 1) ^ (cg >> 1)) << 4) + 8 * (rg & 1)) = w;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int cc = (threadIdx.x >> 3) + 32 * u, i = threadIdx.x & 7;
      if (c0 + cc < d.cols)
        st16(d.qt + static_cast<int64_t>(c0 + cc) * kp + r0 + 16 * i,
             *reinterpret_cast<const u32x4_t*>(tr + cc * 144 + ((i ^ (cc >> 4)) << 4)));
    }
    if (threadIdx.x < kQ / 16 && c0 + 16 * static_cast<int>(threadIdx.x) < rp)
      st16(d.st + static_cast<int64_t>(r0 / kQ) * rp + c0 + 16 * threadIdx.x,
           *reinterpret_cast<const u32x4_t*>(sc + 16 * threadIdx.x));
  }
}

namespace {

template <typename T>
hipError_t run_quantize(const F8QuantCtx& c, int32_t nblocks, int32_t block_rows) {
  if (block_rows == kF8Block)
    hipLaunchKernelGGL((k_f8_quantize<T, true>), dim3(nblocks), dim3(kThreads), 0, c.stream, c);
  else
    hipLaunchKernelGGL((k_f8_quantize<T, false>), dim3(nblocks), dim3(kThreads), 0, c.stream, c);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_f8_quantize(const F8QuantCtx& c, int32_t nblocks, bool is_bf16,
                              int32_t block_rows) {
  if (nblocks <= 0) return hipSuccess;
  return is_bf16 ? run_quantize<uint16_t>(c, nblocks, block_rows)
                 : run_quantize<float>(c, nblocks, block_rows);
}

}  // namespace muon
