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

// Four outputs of a row from column r on.
template <typename To>
__device__ __forceinline__ void store4_to(To* y, int32_t left, bool whole, const f32x4_t& v) {
  if (whole) {
    if constexpr (sizeof(To) == 2) {
      u32x2_t w;
      w[0] = Elt<uint16_t>::pack2(v[0], v[1]);
      w[1] = Elt<uint16_t>::pack2(v[2], v[3]);
      *(GLOBAL_AS u32x2_t*)(y) = w;
    } else {
      st16(y, __builtin_bit_cast(u32x4_t, v));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) y[i] = Elt<To>::from_f32(v[i]);
  }
}

// What a wave reads of RT tile rows over four tiles (512 columns).
template <int RT>
struct Quad {
  u32x4_t w[4][RT];
  u32x4_t s[RT];
};

template <int RT>
__device__ __forceinline__ void load_quad(const F4ProdArgs& a, const char* const (&q)[RT],
                                          const char* const (&s)[RT], int32_t quad, Quad<RT>& to) {
#pragma unroll
  for (int i = 0; i < RT; ++i) to.s[i] = ld16(s[i] + static_cast<int64_t>(quad) * 256);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int32_t t = 4 * quad + j;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      to.w[j][i] = u32x4_t{0, 0, 0, 0};
      if (t < a.ktiles) to.w[j][i] = ld16(q[i] + static_cast<int64_t>(t) * 1024);
    }
  }
}

}  // namespace

// A wave sums RT tile rows times MT * 16 rows of x over its share of the columns.
template <typename To, int RT, int MT, bool VEC>
__global__ __launch_bounds__(64 * kF4Waves) void k_f4_matmul(F4ProdArgs a) {
  constexpr int kOnce = RT * MT < 4 ? RT * MT : 4;  // result tiles joined at a time
  __shared__ __attribute__((aligned(16))) f32x4_t part[kOnce][kF4Waves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int waves = blockDim.x >> 6;
  int32_t e = 0;
  int64_t p0 = 0, p1 = a.m;
  if (a.active != nullptr) {
    if (static_cast<int32_t>(blockIdx.y) >= a.active[0]) return;
    e = a.active[1 + blockIdx.y];
    if (e < 0 || e >= a.experts) return;
    p0 = max(a.offsets[e], 0);
    p1 = min(static_cast<int64_t>(a.offsets[e + 1]), a.m);
  }
  const int32_t quads = (a.ktiles + 3) / 4;
  const char *q[RT], *s[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    // strips past the last take that one's place: their results are not stored
    const int64_t strip = static_cast<int64_t>(e) * a.rtiles +
                          min(static_cast<int32_t>(blockIdx.x) * RT + i, a.rtiles - 1);
    q[i] = a.q + (strip * a.ktiles * 64 + lane) * 16;
    s[i] = a.s + (strip * quads * 16 + (lane & 15)) * 16;
  }
  const int32_t q0 = quads * wave / waves, q1 = quads * (wave + 1) / waves;
  const int32_t kc = 8 * (lane >> 4);
  for (; p0 < p1; p0 += 16 * MT) {
    const uint16_t* x[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      // lanes past the last row take that row's: their results are not stored
      int64_t row = min(p0 + 16 * j + (lane & 15), p1 - 1);
      if (a.slots != nullptr) {
        row = a.slots[row] / a.top_k;
        if (row < 0 || row >= a.x_rows) row = 0;
      }
      x[j] = static_cast<const uint16_t*>(a.x) + row * a.cols;
    }
    f32x4_t acc[RT][MT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int32_t quad = q0; quad < q1; ++quad) {
      Quad<RT> w;
      load_quad<RT>(a, q, s, quad, w);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          bf16x8_t b[MT];
#pragma unroll
          for (int j = 0; j < MT; ++j)
            b[j] = row8<VEC>(x[j], quad * 512 + t * kF4Tile + 32 * g + kc, a.cols);
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const bf16x8_t v = weights8(w.w[t][i][g], scale_of(w.s[i][t] >> (8 * g) & 255u));
#pragma unroll
            for (int j = 0; j < MT; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, b[j], acc[i][j], 0, 0, 0);
          }
        }
      }
    }
#pragma unroll
    for (int first = 0; first < RT * MT; first += kOnce) {
#pragma unroll
      for (int u = 0; u < kOnce; ++u) part[u][wave][lane] = acc[(first + u) / MT][(first + u) % MT];
      __syncthreads();
      for (int u = wave; u < kOnce; u += waves) {
        f32x4_t sum = part[u][0][lane];
        for (int w = 1; w < waves; ++w) sum += part[u][w][lane];
        const int32_t r = (blockIdx.x * RT + (first + u) / MT) * 16 + 4 * (lane >> 4);
        const int64_t p = p0 + 16 * ((first + u) % MT) + (lane & 15);
        if (p < p1 && r < a.rows)
          store4_to(static_cast<To*>(a.y) + p * a.rows + r, a.rows - r, a.rows % 4 == 0, sum);
      }
      __syncthreads();
    }
  }
}

namespace {

template <typename To, int RT, int MT>
void run(const F4ProdArgs& a, const dim3& grid, const dim3& block, hipStream_t s) {
  if (a.cols % 8 == 0)
    hipLaunchKernelGGL((k_f4_matmul<To, RT, MT, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((k_f4_matmul<To, RT, MT, false>), grid, block, 0, s, a);
}

template <typename To>
hipError_t run(const F4ProdArgs& a, hipStream_t s) {
  const int64_t most = a.active != nullptr ? (a.m < a.experts ? a.m : a.experts) : 1;
  const int32_t quads = (a.ktiles + 3) / 4;
  const int32_t per = (quads + kF4Waves - 1) / kF4Waves;
  const dim3 block(quads > 0 ? 64 * ((quads + per - 1) / per) : 64);
  const int64_t each = (a.m + most - 1) / most;
  const int rt = most * a.rtiles >= 2048 ? 4 : most * a.rtiles >= 1024 ? 2 : 1;
  const dim3 grid((a.rtiles + rt - 1) / rt, static_cast<uint32_t>(most));
  if (each > 12) {
    if (rt == 4)
      run<To, 4, 4>(a, grid, block, s);
    else if (rt == 2)
      run<To, 2, 4>(a, grid, block, s);
    else
      run<To, 1, 4>(a, grid, block, s);
  } else if (rt == 4) {
    run<To, 4, 1>(a, grid, block, s);
  } else if (rt == 2) {
    run<To, 2, 1>(a, grid, block, s);
  } else {
    run<To, 1, 1>(a, grid, block, s);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_f4_matmul(const F4ProdArgs& a, bool is_bf16, hipStream_t s) {
  if (a.m <= 0 || a.rows <= 0) return hipSuccess;
  return is_bf16 ? run<uint16_t>(a, s) : run<float>(a, s);
}

}  // namespace muon
