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

}  // namespace

// A wave takes one tile: lane 16 c + r the columns 32 i + 8 c .. + 7, i = 0 .. 3,
// of row r.
template <typename T, bool TRANSPOSE>
__global__ __launch_bounds__(kThreads) void k_f4_quantize(ArgTable, F4QuantArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, c = lane >> 4;
  const int64_t tile = static_cast<int64_t>(block_number()) * (kThreads / 64) + wave;
  if (tile >= a.tiles) return;
  const int32_t kt = static_cast<int32_t>(tile % a.ktiles);
  const int64_t rest = tile / a.ktiles;
  const int32_t tr = static_cast<int32_t>(rest % a.rtiles), m = static_cast<int32_t>(rest / a.rtiles);
  typedef const void* ptr_t;
  const T* const w = static_cast<const T*>(load_const(reinterpret_cast<const ptr_t*>(table_base(a.table)) + m));
  const int32_t row = tr * 16 + r;
  u32x4_t codes = {0, 0, 0, 0};
  uint32_t scales = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int32_t k0 = kt * kF4Tile + 32 * i + 8 * c;
    float v[8];
    float top = 0.f;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = 0.f;
      if (row < a.rows && k0 + e < a.cols)
        v[e] = Elt<T>::to_f32(TRANSPOSE ? w[static_cast<int64_t>(k0 + e) * a.rows + row]
                                        : w[static_cast<int64_t>(row) * a.cols + k0 + e]);
      const float m1 = fabsf(v[e]);
      bad = bad || !(m1 < __builtin_inff());
      top = fmaxf(top, m1);
    }
    // over the four lanes that share the group
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const uint64_t any = __ballot(bad);
    bad = (any >> r & 0x0001000100010001ull) != 0;
    const int e = group_exp(bad ? 0.f : top);
    const float scale = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
#pragma unroll
    for (int x = 0; x < 8; ++x)
      v[x] = bad ? 0.f : fminf(fmaxf(v[x], -kF4Largest), kF4Largest);
    uint32_t q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], scale, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], scale, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], scale, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], scale, 3);
    codes[i] = q;
    scales |= static_cast<uint32_t>(bad ? 255 : row < a.rows ? e + 127 : 127) << (8 * i);
  }
  st16(a.q + (tile * 64 + lane) * 16, codes);
  if (c == 0) {
    // the scales of four tiles lie together, those past the last are 1
    const int32_t quads = (a.ktiles + 3) / 4;
    uint32_t* const to =
        reinterpret_cast<uint32_t*>(a.s) + ((rest * quads + kt / 4) * 16 + r) * 4;
    to[kt % 4] = scales;
    if (kt + 1 == a.ktiles)
      for (int k = kt % 4 + 1; k < 4; ++k) to[k] = 0x7f7f7f7fu;
  }
}

hipError_t launch_f4_quantize(const ArgTable& t, const F4QuantArgs& a, bool is_bf16,
                              bool transpose, hipStream_t s) {
  if (a.tiles <= 0) return hipSuccess;
  const dim3 grid = block_grid((a.tiles + kThreads / 64 - 1) / (kThreads / 64));
  if (is_bf16) {
    if (transpose)
      hipLaunchKernelGGL((k_f4_quantize<uint16_t, true>), grid, dim3(kThreads), 0, s, t, a);
    else
      hipLaunchKernelGGL((k_f4_quantize<uint16_t, false>), grid, dim3(kThreads), 0, s, t, a);
  } else {
    if (transpose)
      hipLaunchKernelGGL((k_f4_quantize<float, true>), grid, dim3(kThreads), 0, s, t, a);
    else
      hipLaunchKernelGGL((k_f4_quantize<float, false>), grid, dim3(kThreads), 0, s, t, a);
  }
  return hipGetLastError();
}

}  // namespace muon
