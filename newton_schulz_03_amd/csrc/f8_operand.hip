// Block-scaled e4m3 operands of a ragged batch of matrices (F8QuantDesc in
// muon_internal.hpp): the matrix, its transpose, or both from one read.
//
// A block (1 x 128 along the contracted side, or 128 x 128) shares one scale
// 2^e: the smallest power of two, at least 2^-127, with the block's largest
// finite magnitude at most 448 * 2^e (448: e4m3's largest value), so that
// nothing saturates.  An element x is stored as the e4m3 rounding (to nearest
// even) of x * 2^-e in one conversion (v_cvt_scalef32_pk_fp8_*).  Infinities and
// NaNs become NaN and take no part in the scale.
//
// Bandwidth-bound: one block per 128 x 128 tile reads it once, 16 bytes a lane
// and every load issued first, and writes whole 128-byte rows of values; the
// transpose goes through 16 KiB of LDS as bytes.  Maxima are taken on the bit
// patterns, two bf16 values an instruction, across lanes by DPP, and values are
// converted two at a time with their scale: with the arithmetic done value by
// value in fp32 (17 instructions a value for both outputs, now 3) the
// instructions were the bound, 61 us against 44 for the tokens of 32 experts.
// Columns that are no multiple of 8 (bf16) or 4 (fp32) are read element by element:
// 16 matrices of 2048 x 6145, both outputs, bf16 270 us against 151 of 2048 x 6144, fp32
// 376 against 217.
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
__device__ __forceinline__ float scale_of(int e) {  // 2^e, e in [-127, 120]; 2^-127 is subnormal
  return __uint_as_float(e == -127 ? 0x400000u : static_cast<uint32_t>(e + 127) << 23);
}

typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
typedef short s16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// The value of lane (i + N) % 16 of this lane's row of 16.
template <int N>
__device__ __forceinline__ uint32_t row_ror(uint32_t v) {
  return static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x120 + N, 0xf, 0xf, true));
}

// The 8 x 8 sub-block a thread holds, as 32-bit words of kPer values along a row.
// A word's magnitudes are compared as integers, all kPer of them at once.
template <typename T> struct Sub;

template <> struct Sub<uint16_t> {
  static constexpr int kPer = 2, kWords = 4;
  static constexpr uint32_t kInf = 0x7f80u;
  uint32_t x[8][4];
  static __device__ __forceinline__ uint32_t mag(uint32_t w) { return w & 0x7fff7fffu; }
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a),
                                                                  __builtin_bit_cast(u16x2_t, b)));
  }
  // The larger half of a and of b, as the two halves of one word.
  static __device__ __forceinline__ uint32_t fold(uint32_t a, uint32_t b) {
    return max(__builtin_amdgcn_perm(b, a, 0x05040100u), __builtin_amdgcn_perm(b, a, 0x07060302u));
  }
  static __device__ __forceinline__ uint32_t half(uint32_t w, int h) {
    return h ? w >> 16 : w & 0xffffu;
  }
  static __device__ __forceinline__ uint32_t f32_bits(uint32_t m) { return m << 16; }
  // Non-finite values become NaN and count as zero.
  static __device__ __forceinline__ void clean(uint32_t& w) {
    if ((w & 0x7f80u) == 0x7f80u) w |= 0x7fffu;
    if ((w & 0x7f800000u) == 0x7f800000u) w |= 0x7fff0000u;
  }
  static __device__ __forceinline__ uint32_t finite_mag(uint32_t w) {
    uint32_t m = mag(w);
    if ((m & 0xffffu) >= 0x7f80u) m &= 0xffff0000u;
    if ((m >> 16) >= 0x7f80u) m &= 0xffffu;
    return m;
  }
  // Four values of row p, columns 4 q ..; four of column c, rows 4 q ..
  __device__ __forceinline__ uint32_t along_row(int p, int q, float scale) const {
    return pack(x[p][2 * q], x[p][2 * q + 1], scale);
  }
  __device__ __forceinline__ uint32_t along_col(int c, int q, float scale) const {
    const int w = c >> 1;
    const uint32_t sel = c & 1 ? 0x07060302u : 0x05040100u;
    return pack(__builtin_amdgcn_perm(x[4 * q + 1][w], x[4 * q][w], sel),
                __builtin_amdgcn_perm(x[4 * q + 3][w], x[4 * q + 2][w], sel), scale);
  }
  static __device__ __forceinline__ uint32_t pack(uint32_t lo, uint32_t hi, float scale) {
    s16x2_t r = {0, 0};
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, lo), scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, hi), scale, true);
    return __builtin_bit_cast(uint32_t, r);
  }
  __device__ __forceinline__ void load_row(int p, const uint16_t* g) {
    const u32x4_t v = ld16(g);
#pragma unroll
    for (int k = 0; k < 4; ++k) x[p][k] = v[k];
  }
  __device__ __forceinline__ void load_some(int p, const uint16_t* g, int n) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      x[p][k] = (2 * k < n ? g[2 * k] : 0u) | (2 * k + 1 < n ? static_cast<uint32_t>(g[2 * k + 1]) << 16 : 0u);
  }
};

template <> struct Sub<float> {
  static constexpr int kPer = 1, kWords = 8;
  static constexpr uint32_t kInf = 0x7f800000u;
  uint32_t x[8][8];
  static __device__ __forceinline__ uint32_t mag(uint32_t w) { return w & 0x7fffffffu; }
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) { return a > b ? a : b; }
  static __device__ __forceinline__ uint32_t half(uint32_t w, int) { return w; }
  static __device__ __forceinline__ uint32_t f32_bits(uint32_t m) { return m; }
  static __device__ __forceinline__ void clean(uint32_t& w) {
    if ((w & kInf) == kInf) w |= 0x7fffffffu;
  }
  static __device__ __forceinline__ uint32_t finite_mag(uint32_t w) {
    const uint32_t m = mag(w);
    return m < kInf ? m : 0u;
  }
  __device__ __forceinline__ uint32_t along_row(int p, int q, float scale) const {
    return pack(x[p][4 * q], x[p][4 * q + 1], x[p][4 * q + 2], x[p][4 * q + 3], scale);
  }
  __device__ __forceinline__ uint32_t along_col(int c, int q, float scale) const {
    return pack(x[4 * q][c], x[4 * q + 1][c], x[4 * q + 2][c], x[4 * q + 3][c], scale);
  }
  static __device__ __forceinline__ uint32_t pack(uint32_t a, uint32_t b, uint32_t c, uint32_t d,
                                                  float scale) {
    s16x2_t r = {0, 0};
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, __uint_as_float(a), __uint_as_float(b), scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, __uint_as_float(c), __uint_as_float(d), scale, true);
    return __builtin_bit_cast(uint32_t, r);
  }
  __device__ __forceinline__ void load_row(int p, const float* g) {
    const u32x4_t v = ld16(g), w = ld16(g + 4);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[p][k] = v[k];
      x[p][4 + k] = w[k];
    }
  }
  __device__ __forceinline__ void load_some(int p, const float* g, int n) {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[p][k] = k < n ? __float_as_uint(g[k]) : 0u;
  }
};

// Largest magnitudes of a thread's rows over the 16 lanes that share them
// (row[p], the same in all of them) and of its columns over its own 8 rows
// (col, in words).
template <typename T, bool ROWS, bool COLS, bool FINITE>
__device__ __forceinline__ void maxima(const Sub<T>& s, uint32_t* row, uint32_t* col) {
  using S = Sub<T>;
  auto m = [&](int p, int w) { return FINITE ? S::finite_mag(s.x[p][w]) : S::mag(s.x[p][w]); };
  if constexpr (COLS) {
#pragma unroll
    for (int w = 0; w < S::kWords; ++w) {
      col[w] = m(0, w);
#pragma unroll
      for (int p = 1; p < 8; ++p) col[w] = S::max(col[w], m(p, w));
    }
  }
  if constexpr (ROWS) {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      row[p] = m(p, 0);
#pragma unroll
      for (int w = 1; w < S::kWords; ++w) row[p] = S::max(row[p], m(p, w));
    }
#pragma unroll
    for (int p = 0; p < 8; p += S::kPer) {
      uint32_t v = row[p];
      if constexpr (S::kPer == 2) v = S::fold(row[p], row[p + 1]);
      v = S::max(v, row_ror<8>(v));
      v = S::max(v, row_ror<4>(v));
      v = S::max(v, row_ror<2>(v));
      v = S::max(v, row_ror<1>(v));
#pragma unroll
      for (int h = 0; h < S::kPer; ++h) row[p + h] = S::half(v, h);
    }
  }
}

}  // namespace

// Thread t holds the 8 x 8 sub-block of rows 8 (t / 16) .. + 7 and columns
// 8 (t % 16) .. + 7 of the tile: 16 lanes cover a row's 128 columns, and the
// 8 rows of a column are 8 bytes of the transpose.  Tiles without infinities
// and NaNs, which the block votes on, skip the selects that set them apart.
// NT: the values are stored with the nontemporal hint, for outputs that outgrow
// the caches.  16 matrices of 2048 x 6144 from memory, both outputs: bf16 144 us
// (5.6 TB/s) with the hint on the stores, 149 without, 150 on the loads alone;
// fp32 214, 221 and 244 us.
template <typename T, bool SQUARE, bool NT>
__global__ __launch_bounds__(kThreads) void k_f8_quantize(ArgTable, F8QuantCtx c) {
  using S = Sub<T>;
  __shared__ __attribute__((aligned(16))) uint8_t tr[kQ * 144];  // [column][row], pitch 144
  __shared__ uint32_t part[4][kQ / S::kPer];
  __shared__ __attribute__((aligned(16))) uint8_t sc[2][kQ];
  __shared__ int slot;
  const char* const table = table_base(c.table);
  const int32_t* const prefix = reinterpret_cast<const int32_t*>(table + c.prefix_off);
  const int j = __builtin_amdgcn_readfirstlane(locate_matrix(prefix, c.batch, blockIdx.x, &slot));
  const F8QuantDesc d = load_const(reinterpret_cast<const F8QuantDesc*>(table) + j);
  const int32_t t = blockIdx.x - load_const(prefix + j);
  const int32_t tpr = (d.cols + kQ - 1) / kQ;
  const int32_t r0 = t / tpr * kQ, c0 = t % tpr * kQ;
  const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;

  S s;
  const int32_t col = c0 + 8 * cg;
  const bool vec = d.cols % Elt<T>::kVec == 0 && col + 8 <= d.cols;
  const T* const x = static_cast<const T*>(d.x) + static_cast<int64_t>(r0 + 8 * rg) * d.cols + col;
  if (vec && r0 + kQ <= d.rows) {
#pragma unroll
    for (int p = 0; p < 8; ++p) s.load_row(p, x + static_cast<int64_t>(p) * d.cols);
  } else {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const int n = r0 + 8 * rg + p < d.rows ? min(8, d.cols - col) : 0;
      if (vec && n > 0)
        s.load_row(p, x + static_cast<int64_t>(p) * d.cols);
      else
        s.load_some(p, x + static_cast<int64_t>(p) * d.cols, n);
    }
  }

  // The maxima: of the 1 x 128 blocks along the rows and down the columns, or
  // (SQUARE) of the tile, which the columns' words lead to.
  uint32_t rm[8], cm[S::kWords];
  uint32_t top = 0;
  maxima<T, !SQUARE, true, false>(s, rm, cm);
#pragma unroll
  for (int w = 0; w < S::kWords; ++w) top = S::max(top, cm[w]);
  bool bad = S::half(top, 0) >= S::kInf;
  if constexpr (S::kPer == 2) bad = bad || S::half(top, 1) >= S::kInf;
  if (__syncthreads_or(bad)) {
    maxima<T, !SQUARE, true, true>(s, rm, cm);
    top = 0;
#pragma unroll
    for (int w = 0; w < S::kWords; ++w) top = S::max(top, cm[w]);
#pragma unroll
    for (int p = 0; p < 8; ++p)
#pragma unroll
      for (int w = 0; w < S::kWords; ++w) S::clean(s.x[p][w]);
  }

  int esq = -127;  // SQUARE: the tile's exponent
  if constexpr (SQUARE) {
    uint32_t m = S::max(top, row_ror<8>(top));
    m = S::max(m, row_ror<4>(m));
    m = S::max(m, row_ror<2>(m));
    m = S::max(m, row_ror<1>(m));
    m = S::max(m, __shfl_xor(m, 16, 64));
    m = S::max(m, __shfl_xor(m, 32, 64));
    if (lane == 0) part[wave][0] = m;
    __syncthreads();
    m = S::max(S::max(part[0][0], part[1][0]), S::max(part[2][0], part[3][0]));
    if constexpr (S::kPer == 2) m = max(m & 0xffffu, m >> 16);
    esq = scale_exp(S::f32_bits(m));
  }

  if (d.q != nullptr) {
    const int32_t kp = tpr * kQ;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const int e = SQUARE ? esq : scale_exp(S::f32_bits(rm[p]));
      const float scale = scale_of(e);
      const int32_t row = r0 + 8 * rg + p;
      if (cg == 0) sc[0][8 * rg + p] = row < d.rows ? static_cast<uint8_t>(e + 127) : 0;
      if (row < d.rows) {
        u32x2_t w;
        w[0] = s.along_row(p, 0, scale);
        w[1] = s.along_row(p, 1, scale);
        GLOBAL_AS u32x2_t* const to =
            (GLOBAL_AS u32x2_t*)(d.q + static_cast<int64_t>(row) * kp + col);
        if constexpr (NT)
          __builtin_nontemporal_store(w, to);
        else
          *to = w;
      }
    }
  }
  if (d.qt != nullptr) {
    if constexpr (!SQUARE) {
#pragma unroll
      for (int w = 0; w < S::kWords; ++w) {
        cm[w] = S::max(cm[w], __shfl_xor(cm[w], 16, 64));
        cm[w] = S::max(cm[w], __shfl_xor(cm[w], 32, 64));
        if (lane < 16) part[wave][S::kWords * cg + w] = cm[w];
      }
      __syncthreads();
#pragma unroll
      for (int w = 0; w < S::kWords; ++w) {
        const int k = S::kWords * cg + w;
        cm[w] = S::max(S::max(part[0][k], part[1][k]), S::max(part[2][k], part[3][k]));
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int cc = 8 * cg + e;
      const int ex = SQUARE ? esq : scale_exp(S::f32_bits(S::half(cm[e / S::kPer], e % S::kPer)));
      const float scale = scale_of(ex);
      if (rg == 0) sc[1][cc] = c0 + cc < d.cols ? static_cast<uint8_t>(ex + 127) : 0;
      u32x2_t w;
      w[0] = s.along_col(e, 0, scale);
      w[1] = s.along_col(e, 1, scale);
      // 16-byte chunk i of a column sits at i ^ (cg / 2): the 16 lanes of a row
      // group then spread over the banks
      *reinterpret_cast<u32x2_t*>(tr + cc * 144 + (((rg >> 1) ^ (cg >> 1)) << 4) + 8 * (rg & 1)) = w;
    }
  }
  __syncthreads();
  if (d.q != nullptr) {
    const int32_t rp = (d.rows + 15) / 16 * 16;
    if (threadIdx.x < kQ / 16 && r0 + 16 * static_cast<int>(threadIdx.x) < rp)
      st16(d.s + static_cast<int64_t>(c0 / kQ) * rp + r0 + 16 * threadIdx.x,
           *reinterpret_cast<const u32x4_t*>(sc[0] + 16 * threadIdx.x));
  }
  if (d.qt != nullptr) {
    const int32_t kp = (d.rows + kQ - 1) / kQ * kQ;
    const int32_t rp = (d.cols + 15) / 16 * 16;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int cc = (threadIdx.x >> 3) + 32 * u, i = threadIdx.x & 7;
      if (c0 + cc >= d.cols) continue;
      uint8_t* const to = d.qt + static_cast<int64_t>(c0 + cc) * kp + r0 + 16 * i;
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(tr + cc * 144 + ((i ^ (cc >> 4)) << 4));
      if constexpr (NT)
        st16_nt(to, v);
      else
        st16(to, v);
    }
    if (threadIdx.x < kQ / 16 && c0 + 16 * static_cast<int>(threadIdx.x) < rp)
      st16(d.st + static_cast<int64_t>(r0 / kQ) * rp + c0 + 16 * threadIdx.x,
           *reinterpret_cast<const u32x4_t*>(sc[1] + 16 * threadIdx.x));
  }
}

namespace {

// Input bytes from which the data comes from memory rather than from caches.
constexpr int64_t kNtBytes = 128ll << 20;

template <typename T, bool SQUARE>
hipError_t run_quantize(const ArgTable& t, const F8QuantCtx& c, int32_t nblocks, bool nt) {
  if (nt)
    hipLaunchKernelGGL((k_f8_quantize<T, SQUARE, true>), dim3(nblocks), dim3(kThreads), 0, c.stream,
                       t, c);
  else
    hipLaunchKernelGGL((k_f8_quantize<T, SQUARE, false>), dim3(nblocks), dim3(kThreads), 0,
                       c.stream, t, c);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_f8_quantize(const ArgTable& t, const F8QuantCtx& c, int32_t nblocks, bool is_bf16,
                              int32_t block_rows, int64_t bytes) {
  if (nblocks <= 0) return hipSuccess;
  const bool nt = bytes > kNtBytes;
  if (block_rows == kF8Block)
    return is_bf16 ? run_quantize<uint16_t, true>(t, c, nblocks, nt)
                   : run_quantize<float, true>(t, c, nblocks, nt);
  return is_bf16 ? run_quantize<uint16_t, false>(t, c, nblocks, nt)
                 : run_quantize<float, false>(t, c, nblocks, nt);
}

}  // namespace muon
