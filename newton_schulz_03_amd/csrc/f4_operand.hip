// 4-bit weights with group scales: operands of a list of equal matrices, or of
// their transposes, for the products of few rows in f4_matmul.hip.
//
// A group of 32 weights along the contracted side shares the scale 2^e, the
// smallest power of two, from 2^-125 to 2^125, with the group's largest magnitude
// at most 6 * 2^e (6: e2m1's largest value); a weight w is stored as the e2m1
// rounding (to nearest even) of w * 2^-e, in one conversion for two
// (v_cvt_scalef32_pk_fp4_f32).  The limits keep every value that an operand can
// stand for a normal bf16 number; magnitudes above 6 * 2^125 become that.  e2m1
// has no NaN: a group that holds an infinity or a NaN takes the scale byte 255,
// and all of it stands for NaN.
//
// Layout (F4 layout in muon_internal.hpp): tiles of 16 rows x 128 columns, a lane
// of the product's wave holding the 16 bytes that it feeds to four matrix
// instructions, so that a wave's load is 1024 bytes in a row.
#include "device_common.hpp"

namespace muon {

namespace {

constexpr float kF4Largest = 6.f * 0x1p125f;

// Exponent of the scale of a group with largest finite magnitude amax = m * 2^E,
// 1 <= m < 2; 6 = 1.5 * 2^2.
__device__ __forceinline__ int group_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - 2 + ((b & 0x7fffffu) > 0x400000u ? 1 : 0);
  return e < -125 ? -125 : e > 125 ? 125 : e;
}

// Quantizes and stores one tile, of tile row `strip` (over all matrices) and tile
// column kt: v[i] are columns 32 i + 8 c .. + 7 of this lane's row r (lane 16 c + r).
__device__ __forceinline__ void put_tile(const F4QuantArgs& a, int64_t strip, int32_t kt, bool live,
                                         float (&v)[4][8]) {
  const int lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
  u32x4_t codes = {0, 0, 0, 0};
  uint32_t scales = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float top = 0.f;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float m = fabsf(v[i][e]);
      bad = bad || !(m < __builtin_inff());
      top = fmaxf(top, m);
    }
    // over the four lanes that share the group
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    bad = (__ballot(bad) >> r & 0x0001000100010001ull) != 0;
    const int e = group_exp(bad ? 0.f : top);
    const float scale = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
#pragma unroll
    for (int x = 0; x < 8; ++x) v[i][x] = bad ? 0.f : fminf(fmaxf(v[i][x], -kF4Largest), kF4Largest);
    uint32_t q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[i][0], v[i][1], scale, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[i][2], v[i][3], scale, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[i][4], v[i][5], scale, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[i][6], v[i][7], scale, 3);
    codes[i] = q;
    scales |= static_cast<uint32_t>(bad ? 255 : live ? e + 127 : 127) << (8 * i);
  }
  st16(a.q + ((strip * a.ktiles + kt) * 64 + lane) * 16, codes);
  if (c == 0) {
    // the scales of four tiles lie together, those past the last are 1
    const int32_t quads = (a.ktiles + 3) / 4;
    uint32_t* const to = reinterpret_cast<uint32_t*>(a.s) + ((strip * quads + kt / 4) * 16 + r) * 4;
    to[kt % 4] = scales;
    if (kt + 1 == a.ktiles)
      for (int k = kt % 4 + 1; k < 4; ++k) to[k] = 0x7f7f7f7fu;
  }
}

template <typename T>
__device__ __forceinline__ const T* matrix(const F4QuantArgs& a, int32_t m) {
  typedef const void* ptr_t;
  return static_cast<const T*>(load_const(reinterpret_cast<const ptr_t*>(table_base(a.table)) + m));
}

}  // namespace

// A wave takes one tile.  Matrices whose rows are no multiple of 8 long are read
// element by element, and so are transposed ones that the kernel below does not
// take (16 of 2048 x 6145 bf16 418 us; 64 of 2048 x 6144 369, 5.5 TB/s).
template <typename T, bool TRANSPOSE>
__global__ __launch_bounds__(kThreads) void k_f4_quantize(ArgTable, F4QuantArgs a) {
  constexpr int kVec = 16 / sizeof(T);
  const int lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
  const int64_t tile = static_cast<int64_t>(block_number()) * (kThreads / 64) + (threadIdx.x >> 6);
  if (tile >= a.tiles) return;
  const int32_t kt = static_cast<int32_t>(tile % a.ktiles);
  const int64_t strip = tile / a.ktiles;
  const T* const w = matrix<T>(a, static_cast<int32_t>(strip / a.rtiles));
  const int32_t row = static_cast<int32_t>(strip % a.rtiles) * 16 + r;
  float v[4][8];
  if (!TRANSPOSE && a.cols % 8 == 0 && row < a.rows) {
    const T* const from = w + static_cast<int64_t>(row) * a.cols + kt * kF4Tile + 8 * c;
    u32x4_t raw[4][8 / kVec];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 8 / kVec; ++h) {
        raw[i][h] = u32x4_t{0, 0, 0, 0};
        if (kt * kF4Tile + 32 * i + 8 * c < a.cols) raw[i][h] = ld16(from + 32 * i + kVec * h);
      }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 8 / kVec; ++h) vec_to_f32<T>(raw[i][h], v[i] + kVec * h);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int32_t k = kt * kF4Tile + 32 * i + 8 * c + e;
        v[i][e] = 0.f;
        if (row < a.rows && k < a.cols)
          v[i][e] = Elt<T>::to_f32(TRANSPOSE ? w[static_cast<int64_t>(k) * a.rows + row]
                                             : w[static_cast<int64_t>(row) * a.cols + k]);
      }
  }
  put_tile(a, strip, kt, row < a.rows, v);
}

// Transposed bf16 matrices whose rows are a multiple of 8 long: a block reads 128
// of their rows, 64 columns of each, in 16-byte pieces, and its waves take a tile
// each from LDS (64 of 6144 x 2048: 378 us; element by element 952.  fp32 stays with
// that: 875 us, through LDS 1500, at 230 registers).
__global__ __launch_bounds__(kThreads) void k_f4_quantize_t(ArgTable, F4QuantArgs a) {
  typedef uint16_t T;
  constexpr int kVec = 16 / sizeof(T), kPieces = 64 / kVec;  // of a row's 64 columns
  constexpr int kPitch = 64 * sizeof(T) + 16;
  __shared__ __attribute__((aligned(16))) char rows[kF4Tile * kPitch];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, c = lane >> 4;
  const int32_t wide = (a.rtiles + 3) / 4;  // blocks over the operand's rows
  const int64_t b = block_number();
  const int32_t kt = static_cast<int32_t>(b % a.ktiles);
  const int64_t rest = b / a.ktiles;
  const int32_t r0 = static_cast<int32_t>(rest % wide) * 64, m = static_cast<int32_t>(rest / wide);
  if (static_cast<int64_t>(m) * a.rtiles * a.ktiles >= a.tiles) return;
  const T* const w = matrix<T>(a, m);
  constexpr int kEach = kF4Tile * kPieces / kThreads;
  u32x4_t raw[kEach];
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const int at = u * kThreads + threadIdx.x;
    const int32_t k = kt * kF4Tile + at / kPieces, col = r0 + at % kPieces * kVec;
    raw[u] = u32x4_t{0, 0, 0, 0};
    if (k < a.cols && col < a.rows) raw[u] = ld16(w + static_cast<int64_t>(k) * a.rows + col);
  }
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const int at = u * kThreads + threadIdx.x;
    *reinterpret_cast<u32x4_t*>(rows + at / kPieces * kPitch + at % kPieces * 16) = raw[u];
  }
  __syncthreads();
  const int32_t tr = r0 / 16 + wave;
  if (tr >= a.rtiles) return;
  float v[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[i][e] = Elt<T>::to_f32(*reinterpret_cast<const T*>(
          rows + (32 * i + 8 * c + e) * kPitch + (16 * wave + r) * sizeof(T)));
  put_tile(a, static_cast<int64_t>(m) * a.rtiles + tr, kt, tr * 16 + r < a.rows, v);
}

namespace {

template <typename T>
void run_quantize(const ArgTable& t, const F4QuantArgs& a, bool transpose, hipStream_t s) {
  if (sizeof(T) == 2 && transpose && a.rows % 8 == 0) {
    const int64_t strips = a.tiles / a.ktiles / a.rtiles * ((a.rtiles + 3) / 4);
    hipLaunchKernelGGL(k_f4_quantize_t, block_grid(strips * a.ktiles), dim3(kThreads), 0, s, t, a);
    return;
  }
  const dim3 grid = block_grid((a.tiles + kThreads / 64 - 1) / (kThreads / 64));
  if (transpose)
    hipLaunchKernelGGL((k_f4_quantize<T, true>), grid, dim3(kThreads), 0, s, t, a);
  else
    hipLaunchKernelGGL((k_f4_quantize<T, false>), grid, dim3(kThreads), 0, s, t, a);
}

}  // namespace

hipError_t launch_f4_quantize(const ArgTable& t, const F4QuantArgs& a, bool is_bf16,
                              bool transpose, hipStream_t s) {
  if (a.tiles <= 0) return hipSuccess;
  if (is_bf16)
    run_quantize<uint16_t>(t, a, transpose, s);
  else
    run_quantize<float>(t, a, transpose, s);
  return hipGetLastError();
}

}  // namespace muon
