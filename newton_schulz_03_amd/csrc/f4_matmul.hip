// Rows times matrices of 4-bit weights with group scales (f4_operand.hip):
//
//   y[p][r] = sum_k x[p][k] W_e[r][k],   offsets[e] <= p < offsets[e + 1]
//
// bf16 rows, fp32 sums, rounded once.  A weight's value is a bf16 number, so that
// the products are exact in fp32: two weights and their scale are one conversion
// (v_cvt_scalef32_pk_bf16_fp4), and four 16x16x32 matrix instructions take a tile
// of 16 weight rows x 128 columns times up to 16 rows of x.
//
// Bound by the weights' bytes: 128 tokens x 8 of 384 experts, of which 265 have
// rows, 3.9 on average, take 299 to 318 us of 6144 x 2048 (fp32 results, 5.6 to 5.9
// TB/s, from machine to machine) and 294 to 299 of 2048 x 6144 (bf16).  Nothing but
// the loads of the weights reached 7.0 TB/s in this order and with those of the scales
// and one row of x 6.5.  What it took: one weight tile is 1024 bytes in a row, so that
// a wave's load is; a wave takes RT strips of 16 rows, since every one of them needs
// the same x (RT 1: 439 us against 315, the loads of x are the bound); a ring of tiles in
// registers that is refilled as it is used, without conditions, which cost registers
// for copies and left one wave a SIMD (a third longer); two waves a SIMD that do not
// spill (three that do: a quarter longer).
#include <algorithm>

#include "device_common.hpp"

namespace muon {

namespace {

constexpr int kF4Waves = 4;  // of a block, 8 where 8 share the columns
constexpr int kF4MaxSplit = 8;
// Most rows of an expert, on average, of the kernel without LDS, which reads the
// weights again for every 16 (one matrix 6144 x 6144: 16 rows 10.2 us, by the kernel
// of many rows 19; 32 rows 27 and 19; 256 tokens x 8 of 384 experts 464 and 558; 512 tokens,
// 10.7 rows on average and 107 at most, 656 and 617 of 2048 x 6144, 571 and 664 of 6144 x
// 2048).  The host knows the average alone: 1024 rows that all fall on 8 of 384
// experts, 2.7 on average, take 257 us, and would take 62 by the other kernel.
constexpr int64_t kF4FewRows = 16;
constexpr int64_t kF4Cus = 256;
// Waves that keep the memory busy.
constexpr int64_t kF4Busy = 2048;

// The bf16 pairs that a word of four bytes stands for.
__device__ __forceinline__ bf16x8_t weights8(uint32_t q, float scale) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 0);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 1);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 2);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 3);
  return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// 2^(byte - 127) of byte g of a word, by its exponent alone; the conversions make
// NaN of the exponent 255.
__device__ __forceinline__ float scale_of(uint32_t word, int g) {
  return __uint_as_float(g == 3 ? word >> 24 << 23 : (word >> (8 * g) & 255u) << 23);
}

// Eight values of a row from column k on.  Rows of odd length lie at any even
// address; the load is the same, but slower for many rows (64 experts of 2048
// weight rows, 1024 rows of x in all: 137 us at 6144 columns, 265 at 6145).
typedef u32x4_t u32x4_at2_t __attribute__((aligned(2)));
__device__ __forceinline__ bf16x8_t row8(const uint16_t* x, int32_t k) {
  return __builtin_bit_cast(bf16x8_t, u32x4_t(*(const GLOBAL_AS u32x4_at2_t*)(x + k)));
}
// The same, zero past the row's end.
__device__ __forceinline__ bf16x8_t row8(const uint16_t* x, int32_t k, int32_t cols) {
  if (k + 8 <= cols) return row8(x, k);
  uint16_t v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = k + e < cols ? x[k + e] : 0;
  bf16x8_t r;
  __builtin_memcpy(&r, v, 16);
  return r;
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

// What a wave of the kernel below holds: RT strips of 16 weight rows, and 16 rows of
// x, of which this lane has one.  A ring of four tiles of weights and scales, and of
// two of x, is in flight.
template <int RT>
struct Strips {
  const char *q[RT], *s[RT];  // uniform
  uint32_t qat, sat;          // this lane's bytes of a tile, of four tiles' scales
  const uint16_t* x;
  int32_t cols, kc;
  u32x4_t w[4][RT];
  u32x2_t sc[2][RT];          // of an even tile and the one after it
  bf16x8_t b[2][4];
  f32x4_t acc[RT];

  __device__ __forceinline__ void load_w(int u, int32_t t) {
#pragma unroll
    for (int i = 0; i < RT; ++i) w[u][i] = ld16_nt(q[i] + static_cast<int64_t>(t) * 1024 + qat);
  }
  __device__ __forceinline__ void load_s(int h, int32_t t) {  // t even, h = t / 2 % 2
#pragma unroll
    for (int i = 0; i < RT; ++i)
      sc[h][i] = *(const GLOBAL_AS u32x2_t*)(s[i] + static_cast<int64_t>(t) * 64 + (h ? 8 - 128 : 0) + sat);
  }
  __device__ __forceinline__ void load_x(int v, int32_t t) {
#pragma unroll
    for (int g = 0; g < 4; ++g) b[v][g] = row8(x, t * kF4Tile + 32 * g + kc);
  }
  __device__ __forceinline__ void multiply(int u) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
#pragma unroll
      for (int i = 0; i < RT; ++i)
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            weights8(w[u][i][g], scale_of(sc[u / 2][i][u % 2], g)), b[u % 2][g], acc[i], 0, 0, 0);
      // the scheduler would convert everything first, and spill
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  __device__ __forceinline__ void begin(int32_t t) {
    load_s(0, t);
    load_s(1, t + 2);
#pragma unroll
    for (int u = 0; u < 4; ++u) load_w(u, t + u);
  }
  // Four tiles from t on; MORE: the next four are asked for.
  template <bool MORE>
  __device__ __forceinline__ void quad(int32_t t) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (MORE || u < 3) load_x(1 - u % 2, t + u + 1);
      multiply(u);
      if (MORE) load_w(u, t + u + 4);
      if (MORE && u % 2 == 1) load_s(u / 2, t + u + 3);
    }
  }
  // One tile, which may lie partly past the columns.
  __device__ __forceinline__ void tile(int32_t t) {
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      w[0][i] = ld16_nt(q[i] + static_cast<int64_t>(t) * 1024 + qat);
      sc[0][i][0] = *(const GLOBAL_AS uint32_t*)(s[i] + static_cast<int64_t>(t / 4) * 256 + t % 4 * 4 + sat);
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) b[0][g] = row8(x, t * kF4Tile + 32 * g + kc, cols);
    multiply(0);
  }
};

}  // namespace

// A wave sums RT tile rows times 16 rows of x over its share of the columns: the
// block's waves are `ksplit` shares of the columns times groups of RT tile rows.
template <typename To, int RT>
__global__ __launch_bounds__(64 * kF4MaxSplit, 2) void k_f4_matmul(F4ProdArgs a) {
  __shared__ __attribute__((aligned(16))) f32x4_t part[RT][kF4MaxSplit][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ks = wave % a.ksplit, rs = wave / a.ksplit;
  int32_t e = 0;
  int64_t p0 = 0, p1 = a.m;
  if (a.active != nullptr) {
    e = load_const(a.active + 1 + blockIdx.y);  // with the next load: one wait for both
    if (static_cast<int32_t>(blockIdx.y) >= load_const(a.active)) return;
    if (e < 0 || e >= a.experts) return;
  }
  const int32_t quads = (a.ktiles + 3) / 4;
  const int32_t strip0 = (blockIdx.x * ((blockDim.x >> 6) / a.ksplit) + rs) * RT;
  Strips<RT> z;
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    // strips past the last take that one's place: their results are not stored
    const int64_t strip = static_cast<int64_t>(e) * a.rtiles + min(strip0 + i, a.rtiles - 1);
    z.q[i] = a.q + strip * a.ktiles * 1024;
    z.s[i] = a.s + strip * quads * 256;
  }
  z.qat = lane * 16;
  z.sat = (lane & 15) * 16;
  z.cols = a.cols;
  z.kc = 8 * (lane >> 4);
  // tiles t0 .. t1 - 1, whole quads of them up to tq
  const int32_t t0 = quads * ks / a.ksplit * 4, t1 = min(quads * (ks + 1) / a.ksplit * 4, a.ktiles);
  const int32_t tq = max(t0, min(quads * (ks + 1) / a.ksplit, a.cols / (4 * kF4Tile)) * 4);
  if (tq > t0) z.begin(t0);  // the weights are on their way before the rows are known
  if (a.active != nullptr) {
    p0 = max(load_const(a.offsets + e), 0);
    p1 = min(static_cast<int64_t>(load_const(a.offsets + e + 1)), a.m);
  }
  for (; p0 < p1; p0 += 16) {
    // lanes past the last row take that row's: their results are not stored
    int64_t row = min(p0 + (lane & 15), p1 - 1);
    if (a.slots != nullptr) {
      row = a.slots[row] / a.top_k;
      if (row < 0 || row >= a.x_rows) row = 0;
    }
    z.x = static_cast<const uint16_t*>(a.x) + row * a.cols;
#pragma unroll
    for (int i = 0; i < RT; ++i) z.acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    if (tq > t0) {
      z.load_x(0, t0);
      int32_t t = t0;
      for (; t + 4 < tq; t += 4) z.template quad<true>(t);
      z.template quad<false>(t);
    }
    for (int32_t t = tq; t < t1; ++t) z.tile(t);
    if (a.ksplit > 1) {
#pragma unroll
      for (int i = 0; i < RT; ++i) part[i][wave][lane] = z.acc[i];
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      if (a.ksplit > 1) {
        // each of the waves that share these rows stores some of them
        if (i % a.ksplit != ks) continue;
        z.acc[i] = part[i][rs * a.ksplit][lane];
        for (int k = 1; k < a.ksplit; ++k) z.acc[i] += part[i][rs * a.ksplit + k][lane];
      }
      const int32_t r = (strip0 + i) * 16 + 4 * (lane >> 4);
      const int64_t p = p0 + (lane & 15);
      if (p < p1 && r < a.rows)
        store4_to(static_cast<To*>(a.y) + p * a.rows + r, a.rows - r, a.rows % 4 == 0, z.acc[i]);
    }
    if (p0 + 16 < p1) {
      if (a.ksplit > 1) __syncthreads();
      if (tq > t0) z.begin(t0);
    }
  }
}

// The same for experts of many rows: 64 rows of x at a time go through LDS, one tile's
// columns after the other, and serve every wave of the block.  Four waves take RT
// strips each, KS groups of four a share of the columns each.
namespace {
constexpr int kManyRows = 64;
constexpr int kManyTile = kManyRows * kF4Tile * 2;  // bytes of x
}  // namespace

template <typename To, int RT, int KS>
__global__ __launch_bounds__(256 * KS, 2) void k_f4_many(F4ProdArgs a) {
  constexpr int MT = kManyRows / 16;
  // [group][buffer][row][16 bytes of 8 columns at chunk ^ row % 16], then the sums
  __shared__ __attribute__((aligned(16))) char xs[KS][2][kManyTile];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ks = wave / 4, rs = wave % 4;
  int32_t e = 0;
  int64_t p0 = 0, p1 = a.m;
  if (a.active != nullptr) {
    e = load_const(a.active + 1 + blockIdx.y);
    if (static_cast<int32_t>(blockIdx.y) >= load_const(a.active)) return;
    if (e < 0 || e >= a.experts) return;
    p0 = max(load_const(a.offsets + e), 0);
    p1 = min(static_cast<int64_t>(load_const(a.offsets + e + 1)), a.m);
  }
  const int32_t quads = (a.ktiles + 3) / 4;
  const int32_t strip0 = (blockIdx.x * 4 + rs) * RT;
  const char *q[RT], *s[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int64_t strip = static_cast<int64_t>(e) * a.rtiles + min(strip0 + i, a.rtiles - 1);
    q[i] = a.q + strip * a.ktiles * 1024;
    s[i] = a.s + strip * quads * 256;
  }
  const uint32_t qat = lane * 16, sat = (lane & 15) * 16;
  const int32_t t0 = a.ktiles * ks / KS, t1 = a.ktiles * (ks + 1) / KS;
  const int32_t steps = (a.ktiles + KS - 1) / KS;  // of the longest share
  // steps whose tiles are whole in every share, in fours
  const int32_t whole = min(a.ktiles / KS, a.cols / kF4Tile - a.ktiles * (KS - 1) / KS) / 4 * 4;
  const int at = threadIdx.x & 255, chunk = at & 15;
  for (p0 += static_cast<int64_t>(blockIdx.z) * kManyRows; p0 < p1;
       p0 += static_cast<int64_t>(gridDim.z) * kManyRows) {
    const uint16_t* x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      int64_t row = min(p0 + 16 * j + (at >> 4), p1 - 1);
      if (a.slots != nullptr) {
        row = a.slots[row] / a.top_k;
        if (row < 0 || row >= a.x_rows) row = 0;
      }
      x[j] = static_cast<const uint16_t*>(a.x) + row * a.cols + 8 * chunk;
    }
    u32x4_t w[4][RT], xr[2][4];
    uint32_t sc[4][RT];
    f32x4_t acc[RT][MT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    auto load_w = [&](int u, int32_t t) {
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        w[u][i] = ld16(q[i] + static_cast<int64_t>(t) * 1024 + qat);
        sc[u][i] = *(const GLOBAL_AS uint32_t*)(s[i] + static_cast<int64_t>(t / 4) * 256 + t % 4 * 4 + sat);
      }
    };
    auto load_x = [&](int v, int32_t t) {
#pragma unroll
      for (int j = 0; j < 4; ++j) xr[v][j] = __builtin_bit_cast(u32x4_t, row8(x[j], t * kF4Tile));
    };
    auto store_x = [&](char* buf, int v) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 16 * j + (at >> 4);
        *reinterpret_cast<u32x4_t*>(buf + r * 256 + ((chunk ^ (r & 15)) << 4)) = xr[v][j];
      }
    };
    // x of the next group of 32 columns is read while this one's is multiplied
    auto read_b = [&](const char* buf, int g, bf16x8_t (&b)[MT]) {
      const int r = lane & 15;
#pragma unroll
      for (int j = 0; j < MT; ++j)
        b[j] = *reinterpret_cast<const bf16x8_t*>(buf + (16 * j + r) * 256 +
                                                  (((4 * g + (lane >> 4)) ^ r) << 4));
    };
    auto multiply = [&](const char* buf, int u) {
      bf16x8_t b[2][MT];
      read_b(buf, 0, b[0]);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        if (g < 3) read_b(buf, g + 1, b[(g + 1) & 1]);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const bf16x8_t v = weights8(w[u][i][g], scale_of(sc[u][i], g));
#pragma unroll
          for (int j = 0; j < MT; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, b[g & 1][j], acc[i][j], 0, 0, 0);
        }
      }
    };
    if (whole > 0) {
      load_x(0, t0);
      load_x(1, t0 + 1);
#pragma unroll
      for (int u = 0; u < 4; ++u) load_w(u, t0 + u);
      const int32_t last = t0 + whole - 1;  // asked for again where there is no next one
      for (int32_t t = t0; t <= last; t += 4) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          store_x(xs[ks][u & 1], u & 1);
          load_x(u & 1, min(t + u + 2, last));
          // who read this buffer two steps ago has passed a barrier since
          __syncthreads();
          multiply(xs[ks][u & 1], u);
          load_w(u, min(t + u + 4, last));
        }
      }
    }
    for (int32_t n = whole; n < steps; ++n) {
      const int32_t t = t0 + n;
      __syncthreads();
      if (t < t1) {
        load_w(0, t);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          xr[0][j] = __builtin_bit_cast(
              u32x4_t, row8(x[j] - 8 * chunk, t * kF4Tile + 8 * chunk, a.cols));
        store_x(xs[ks][0], 0);
      }
      __syncthreads();
      if (t < t1) multiply(xs[ks][0], 0);
    }
    if constexpr (KS == 2) {
      // the second share's sums go through LDS, one strip at a time
      f32x4_t* const part = reinterpret_cast<f32x4_t*>(xs);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        __syncthreads();
        if (ks == 1)
#pragma unroll
          for (int j = 0; j < MT; ++j) part[(rs * MT + j) * 64 + lane] = acc[i][j];
        __syncthreads();
        if (ks == 0)
#pragma unroll
          for (int j = 0; j < MT; ++j) acc[i][j] += part[(rs * MT + j) * 64 + lane];
      }
    }
    if (ks == 0) {
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          const int32_t r = (strip0 + i) * 16 + 4 * (lane >> 4);
          const int64_t p = p0 + 16 * j + (lane & 15);
          if (p < p1 && r < a.rows)
            store4_to(static_cast<To*>(a.y) + p * a.rows + r, a.rows - r, a.rows % 4 == 0, acc[i][j]);
        }
    }
    __syncthreads();  // before the next rows' first buffer
  }
}

namespace {

template <typename To, int RT>
void run(const F4ProdArgs& a, int64_t experts, hipStream_t s) {
  const int waves = std::max(kF4Waves, a.ksplit), strips = waves / a.ksplit * RT;
  const dim3 grid((a.rtiles + strips - 1) / strips, static_cast<uint32_t>(experts));
  const dim3 block(64 * waves);
  hipLaunchKernelGGL((k_f4_matmul<To, RT>), grid, block, 0, s, a);
}

template <typename To, int RT, int KS>
void run_many(const F4ProdArgs& a, int64_t experts, int64_t passes, hipStream_t s) {
  const dim3 grid((a.rtiles + 4 * RT - 1) / (4 * RT), static_cast<uint32_t>(experts),
                  static_cast<uint32_t>(passes));
  hipLaunchKernelGGL((k_f4_many<To, RT, KS>), grid, dim3(256 * KS), 0, s, a);
}

template <typename To>
hipError_t run(F4ProdArgs a, hipStream_t s) {
  const int64_t most = a.active != nullptr ? (a.m < a.experts ? a.m : a.experts) : 1;
  const int64_t strips = most * a.rtiles;
  const int64_t each = (a.m + most - 1) / most;
  if (each > kF4FewRows) {
    const int64_t passes = std::min<int64_t>((each + kManyRows - 1) / kManyRows, 65535);
    // Two shares of the columns while those blocks, of which a CU holds one, are no
    // more than the CUs, or two strips a wave, half as many waves a strip (8192 x 8192,
    // 128 rows, 256 blocks of two shares: 28 us, two strips 39; 6144 x 6144, 192 rows, 288
    // blocks: 37.5 and 30.4, 256 rows, 384 blocks: 37.7 and 30.5; one strip and one share
    // lies between them).
    const int64_t blocks = most * ((a.rtiles + 3) / 4) * passes;
    if (blocks > kF4Cus)
      run_many<To, 2, 1>(a, most, passes, s);
    else
      run_many<To, 1, 2>(a, most, passes, s);
    return hipGetLastError();
  }
  const int32_t quads = (a.ktiles + 3) / 4;
  const int64_t most_split = std::min<int64_t>(kF4MaxSplit, quads);
  // As many strips a wave as leave enough waves: 8 experts of 2048 x 6144 with two
  // 11.3 us, with one 14.2, with four 13.2; 265 of 6144 x 2048 with four 315, with two 320 to
  // 334, with one 439.  Then as many waves to share the columns as make up kF4Busy (one
  // matrix 2048 x 6144: 6.0 us by eight, 6.4 by four; of 16 rows 9.3 and 8.9).
  const int rt = strips * most_split >= 8 * kF4Busy ? 4 : strips * most_split >= kF4Busy ? 2 : 1;
  a.ksplit = 1;
  while (a.ksplit < kF4MaxSplit && 2 * a.ksplit <= quads && strips / rt * a.ksplit < kF4Busy) a.ksplit *= 2;
  if (rt == 4)
    run<To, 4>(a, most, s);
  else if (rt == 2)
    run<To, 2>(a, most, s);
  else
    run<To, 1>(a, most, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_f4_matmul(const F4ProdArgs& a, bool is_bf16, hipStream_t s) {
  if (a.m <= 0 || a.rows <= 0) return hipSuccess;
  return is_bf16 ? run<uint16_t>(a, s) : run<float>(a, s);
}

}  // namespace muon
