// C = A B^T (+ C) over block-scaled e4m3 operands (F8ProdDesc in
// muon_internal.hpp), ragged over a batch.
//
//   C[m][n] = sum_kb 2^(sa[kb][m]-127) 2^(sb[kb][n]-127) sum_{k in block kb} a[m][k] b[n][k]
//
// The scales are powers of two, so applying them rounds nothing; C is rounded
// once, at the store.  Two ways to the sum:
//  * bf16 C: the scaled matrix instruction (v_mfma_scale_f32_32x32x64_f8f6f4)
//    on the stored bytes.  It adds 8 consecutive products of a lane in a window
//    of about 14 binades below the largest before they reach the fp32
//    accumulator (measured: a product 2^-13 of its group's largest counts, one
//    of 2^-14 does not).  On Gaussian operands that is 1.5e-5 of the result at
//    any K, far below the 1.7e-3 of the bf16 rounding.
//  * fp32 C: that error would be 250 times the output's own rounding, so the
//    operands are converted on the way from LDS to bf16, scale included
//    (v_cvt_scalef32_pk_bf16_fp8: exact, but for values below bf16's smallest,
//    2^-133), and v_mfma_f32_32x32x16_bf16 sums them with fp32 precision, at
//    half the matrix rate.
//
// 256 x 256 tiles, four waves of 128 x 128, K in slices of 64 through an LDS
// ring of 4 stages filled by direct-to-LDS loads (gemm_pipeline.hpp's slice
// loop and swizzle).  The operands are row-major; a slice takes 64 bytes of
// each of the tile's 256 rows.  Rows past the operand's end repeat its last
// one: what they give is not stored.
//   The first matrix operand (P) is B, the second (Q) A: a lane's registers
// then run along a row of C.  LDS row 128 h + 32 i + r holds the tile's row
// 128 h + 4 r + i, so that lane r of fragment i works on row 4 r + i: the
// scales of a lane's four fragments are one aligned dword of the scale row
// (op_sel picks the byte), and a lane's registers hold 16 consecutive columns
// of C for each of its rows.
#include <utility>

#include "gemm_pipeline.hpp"

namespace muon {

namespace {

static_assert(kF8Tile == kTile, "the pipeline's tile");
constexpr int SCB = 256;                   // scale bytes per operand and stage
constexpr int STAGE8 = 2 * OPB + 2 * SCB;  // P data, Q data, P scales, Q scales
constexpr int LDS8 = NST * STAGE8;
constexpr int LOADS8 = 2 * LPO + 1;        // loads per wave and stage: P, then scales, then Q
static_assert(LDS8 + 1024 <= 160 * 1024, "LDS of a CU");

typedef int32_t i32x8_t __attribute__((ext_vector_type(8)));

// One dword per lane straight into LDS (lane i's 4 bytes at lds_addr + 4 i),
// counted by hand like lds_dma16.
__device__ __forceinline__ void lds_dma4(uint32_t lds_addr, int32_t voff, i32x4_t rsrc) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :
               : "s"(lds_addr), "v"(voff), "s"(rsrc)
               : "memory", "m0");
}

__device__ __forceinline__ i32x4_t make_rsrc(const uint8_t* base, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  i32x4_t r;
  r[0] = __builtin_amdgcn_readfirstlane(static_cast<int32_t>(b & 0xffffffffu));
  r[1] = __builtin_amdgcn_readfirstlane(static_cast<int32_t>((b >> 32) & 0xffffu));
  r[2] = __builtin_amdgcn_readfirstlane(static_cast<int32_t>(bytes));
  r[3] = 0x00020000;
  return r;
}

// Tile row held by LDS row s (0 .. 255).
__device__ __forceinline__ int tile_row(int s) {
  return (s & 128) + 4 * (s & 31) + ((s >> 5) & 3);
}

// One operand's rows of the tile, 64 bytes of each per slice.
struct RowStream {
  const uint8_t* base;  // the tile's first row (uniform)
  uint32_t bytes;       // of the tile's rows that exist
  int32_t voff[LPO];    // per-lane offsets, one per load instruction
  int32_t lds;          // LDS offset of this wave's first 1 KiB block, within the operand

  __device__ __forceinline__ void init(const uint8_t* rows0, int32_t valid, int32_t kp, int wave,
                                       int lane) {
    base = rows0;
    bytes = static_cast<uint32_t>(valid) * static_cast<uint32_t>(kp);
#pragma unroll
    for (int u = 0; u < LPO; ++u) {
      const int s = 16 * (LPO * wave + u) + (lane >> 2);
      const int row = tile_row(s);
      voff[u] = (row < valid ? row : valid - 1) * kp + (((lane & 3) ^ kkey(s)) << 4);
    }
    lds = LPO * wave * 1024;
  }
  __device__ __forceinline__ i32x4_t rsrc(int ks) const {
    return make_rsrc(base + 64 * ks, bytes - 64u * ks);
  }
  __device__ __forceinline__ void issue_one(const i32x4_t& r, uint32_t stage_op, int u) const {
    lds_dma16(__builtin_amdgcn_readfirstlane(stage_op + lds + u * 1024), voff[u], r);
  }
  __device__ __forceinline__ void issue(int ks, uint32_t stage_op) const {
    const i32x4_t r = rsrc(ks);
#pragma unroll
    for (int u = 0; u < LPO; ++u) issue_one(r, stage_op, u);
  }
};

// The tile's scale bytes of one operand: waves 0 and 2 load P's, 1 and 3 Q's
// (each pair the same bytes to the same place, so that every wave has the same
// number of loads in flight).
struct ScaleRows {
  const uint8_t* base;  // scale row 0 at the tile's first row (uniform)
  int32_t rp;           // bytes of a scale row
  int32_t voff;         // this lane's four rows, or the last four that exist
  int32_t lds;

  __device__ __forceinline__ void init(const uint8_t* s, int32_t row0, int32_t rows, int wave,
                                       int lane) {
    base = s + row0;
    rp = (rows + 15) & ~15;
    const int32_t last = rp - 4 - row0;
    voff = 4 * lane < last ? 4 * lane : last;
    lds = 2 * OPB + (wave & 1) * SCB;
  }
  __device__ __forceinline__ void issue(int ks, uint32_t stage) const {
    const i32x4_t r = make_rsrc(base + static_cast<int64_t>(ks >> 1) * rp, 256);
    lds_dma4(__builtin_amdgcn_readfirstlane(stage + lds), voff, r);
  }
};

struct Frags8 {
  i32x8_t p[4];    // dwords 0-3: chunk h of the 64-byte row, 4-7: chunk 2 + h
  i32x8_t q[4];
  int32_t sp, sq;  // byte i: the scale of fragment i's row
};

// The scale of byte i as a float (2^-127 is subnormal).
__device__ __forceinline__ float scale_value(int32_t bytes, int i) {
  const uint32_t e = (static_cast<uint32_t>(bytes) >> (8 * i)) & 255u;
  const uint32_t b = e << 23;
  return __uint_as_float(b > 0x400000u ? b : 0x400000u);
}

// A fragment as bf16: v[s] holds the lane's K values 8 s .. 8 s + 7 for matrix
// step s of the slice.
struct Wide {
  bf16x8_t v[4];
};
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
// Converts dword d (four values) of a raw fragment.
__device__ __forceinline__ void widen(Wide& w, int d, int32_t raw, float scale) {
  const bf16x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw, scale, false);
  const bf16x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw, scale, true);
  const int s = d >> 1, o = 4 * (d & 1);
  w.v[s][o] = lo[0];
  w.v[s][o + 1] = lo[1];
  w.v[s][o + 2] = hi[0];
  w.v[s][o + 3] = hi[1];
}

__device__ __forceinline__ void set_half(i32x8_t& f, int h, const u32x4_t& v) {
#pragma unroll
  for (int k = 0; k < 4; ++k) f[4 * h + k] = static_cast<int32_t>(v[k]);
}

// Sixteen consecutive columns of one row of C.
template <typename T>
__device__ __forceinline__ void store16(T* c, float* v, int32_t left, bool vec, bool add) {
  constexpr int V = Elt<T>::kVec;
  if (left >= 16 && vec) {
    if (add) {
      float o[16];
#pragma unroll
      for (int h = 0; h < 16 / V; ++h) vec_to_f32<T>(ld16(c + h * V), o + h * V);
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] += o[e];
    }
#pragma unroll
    for (int h = 0; h < 16 / V; ++h) st16(c + h * V, f32_to_vec<T>(v + h * V));
    return;
  }
#pragma unroll
  for (int e = 0; e < 16; ++e)
    if (e < left) c[e] = Elt<T>::from_f32(add ? v[e] + Elt<T>::to_f32(c[e]) : v[e]);
}

}  // namespace

template <typename T>
__global__ __launch_bounds__(kThreads, 1) void k_f8_prod(F8ProdCtx c) {
  __shared__ __attribute__((aligned(1024))) char smem[LDS8];
  __shared__ int slot;
  const int32_t b = xcd_remap(blockIdx.x, gridDim.x);
  const int j = __builtin_amdgcn_readfirstlane(locate_matrix(c.prefix, c.batch, b, &slot));
  const F8ProdDesc d = load_const(c.desc + j);
  const int32_t t = b - load_const(c.prefix + j);
  const int32_t tm = (d.m + kTile - 1) / kTile;
  const int32_t m0 = t % tm * kTile, n0 = t / tm * kTile;  // down a column of tiles: B stays

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int lr = lane & 31, lh = lane >> 5;

  f32x16_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][k][e] = 0.f;

  const int nk = d.kp / 64;
  if (nk > 0) {
    RowStream sp, sq;
    sp.init(d.b + static_cast<int64_t>(n0) * d.kp, min(kTile, d.n - n0), d.kp, wave, lane);
    sq.init(d.a + static_cast<int64_t>(m0) * d.kp, min(kTile, d.m - m0), d.kp, wave, lane);
    ScaleRows ss;
    if (wave & 1)
      ss.init(d.sa, m0, d.m, wave, lane);
    else
      ss.init(d.sb, n0, d.n, wave, lane);

    int32_t qoff[2], poff[2];
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const int sw = ((2 * sub + lh) ^ kkey(lr)) << 4;
      qoff[sub] = OPB + (wn * 128 + lr) * KROW + sw;
      poff[sub] = (wm * 128 + lr) * KROW + sw;
    }
    const int32_t psc = 2 * OPB + 4 * (32 * wm + lr);
    const int32_t qsc = 2 * OPB + SCB + 4 * (32 * wn + lr);

    // Fragment reads in the order the MFMAs consume them: the scales, P[0],
    // Q[0..3], then P[1..3]; two 16-byte reads per fragment.
    constexpr int NREAD8 = 18;
    auto read_op = [&](Frags8& f, const char* stage, int i) {
      if (i == 0) {
        f.sp = *reinterpret_cast<const int32_t*>(stage + psc);
      } else if (i == 1) {
        f.sq = *reinterpret_cast<const int32_t*>(stage + qsc);
      } else if (i < 4) {
        set_half(f.p[0], i - 2, lds16(stage + poff[i - 2]));
      } else if (i < 12) {
        const int ni = (i - 4) >> 1, h = (i - 4) & 1;
        set_half(f.q[ni], h, lds16(stage + qoff[h] + ni * 32 * KROW));
      } else {
        const int mi = 1 + ((i - 12) >> 1), h = (i - 12) & 1;
        set_half(f.p[mi], h, lds16(stage + poff[h] + mi * 32 * KROW));
      }
    };

    const uint32_t ring = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((LDS_AS char*)smem));
    // Prologue: slices 0..NST-2 requested (P, scales, Q each), slice 0 awaited.
    // Slice indices past the end are clamped to the last slice: those loads
    // refill a stage nobody reads again and keep the count in flight constant.
#pragma unroll
    for (int s = 0; s < NST - 1; ++s) {
      const int ks = s < nk ? s : nk - 1;
      sp.issue(ks, ring + s * STAGE8);
      ss.issue(ks, ring + s * STAGE8);
      sq.issue(ks, ring + s * STAGE8 + OPB);
    }
    wait_vm<(NST - 2) * LOADS8>();
    __syncthreads();

    if constexpr (sizeof(T) == 2) {
      Frags8 f0, f1;
  #pragma unroll
      for (int i = 0; i < NREAD8; ++i) read_op(f0, smem, i);

      // Slice kt on fragments fa (stage kt), reading stage kt+1 into fb.
      auto slice = [&](int kt, Frags8& fa, Frags8& fb) {
        const int ks = kt + NST - 1 < nk ? kt + NST - 1 : nk - 1;
        const uint32_t fill = ring + ((kt + NST - 1) & (NST - 1)) * STAGE8;
        const i32x4_t rp = sp.rsrc(ks);
        static_for(
            [&](auto I) {
              constexpr int i = decltype(I)::value;
              if constexpr ((i & 1) == 0) sp.issue_one(rp, fill, i >> 1);
              if constexpr (i == 7) ss.issue(ks, fill);
              acc[i >> 2][i & 3] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                  fa.p[i >> 2], fa.q[i & 3], acc[i >> 2][i & 3], 0, 0, i >> 2, fa.sp, i & 3, fa.sq);
              __builtin_amdgcn_sched_barrier(0);
            },
            std::make_integer_sequence<int, 8>{});
        // slice kt+1 has landed once only slice kt+2 and the P and scale loads of
        // kt+NST-1 remain
        wait_vm<(NST - 3) * LOADS8 + LPO + 1>();
        wait_lgkm0();  // this wave's reads of stage kt+NST-1's previous slice are done
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
        const i32x4_t rq = sq.rsrc(ks);
        const char* next = smem + ((kt + 1) & (NST - 1)) * STAGE8;
        static_for(
            [&](auto I) {
              constexpr int i = 8 + decltype(I)::value;
              constexpr int j = decltype(I)::value;
              if constexpr ((j & 1) == 0) sq.issue_one(rq, fill + OPB, j >> 1);
              // 18 reads over 8 MFMAs: three in the first two, two in the rest
              constexpr int r0 = j < 2 ? 3 * j : 6 + 2 * (j - 2);
              constexpr int r1 = j < 2 ? 3 * j + 3 : 6 + 2 * (j - 1);
  #pragma unroll
              for (int r = r0; r < r1; ++r) read_op(fb, next, r);
              acc[i >> 2][i & 3] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                  fa.p[i >> 2], fa.q[i & 3], acc[i >> 2][i & 3], 0, 0, i >> 2, fa.sp, i & 3, fa.sq);
              __builtin_amdgcn_sched_barrier(0);
            },
            std::make_integer_sequence<int, 8>{});
      };
      // nk is even: the operands' K is padded to whole blocks of 128
      for (int kt = 0; kt < nk; kt += 2) {
        slice(kt, f0, f1);
        slice(kt + 1, f1, f0);
      }
    } else {
      // Fragments of slice kt are converted one step ahead of the MFMAs that take
      // them, between MFMAs.  On entry to a slice: Q[0..2] and P[0] converted,
      // Q[3] raw.
      Wide qb[4], pb[2];
      i32x8_t rq[4], rp;
      int32_t ssp, ssq, nsp = 0, nsq = 0;
      auto load_q = [&](const char* stage, int ni, int h) {
        set_half(rq[ni], h, lds16(stage + qoff[h] + ni * 32 * KROW));
      };
      auto load_p = [&](const char* stage, int mi, int h) {
        set_half(rp, h, lds16(stage + poff[h] + mi * 32 * KROW));
      };
      auto widen_q = [&](int ni, int d, int32_t sc) { widen(qb[ni], d, rq[ni][d], scale_value(sc, ni)); };
      auto widen_p = [&](int mi, int d, int32_t sc) { widen(pb[mi & 1], d, rp[d], scale_value(sc, mi)); };
      ssp = *reinterpret_cast<const int32_t*>(smem + psc);
      ssq = *reinterpret_cast<const int32_t*>(smem + qsc);
#pragma unroll
      for (int ni = 0; ni < 4; ++ni)
#pragma unroll
        for (int h = 0; h < 2; ++h) load_q(smem, ni, h);
#pragma unroll
      for (int h = 0; h < 2; ++h) load_p(smem, 0, h);
#pragma unroll
      for (int d = 0; d < 8; ++d) {
#pragma unroll
        for (int ni = 0; ni < 3; ++ni) widen_q(ni, d, ssq);
        widen_p(0, d, ssp);
      }
      for (int kt = 0; kt < nk; ++kt) {
        const int ks = kt + NST - 1 < nk ? kt + NST - 1 : nk - 1;
        const uint32_t fill = ring + ((kt + NST - 1) & (NST - 1)) * STAGE8;
        const char* cur = smem + (kt & (NST - 1)) * STAGE8;
        const char* next = smem + ((kt + 1) & (NST - 1)) * STAGE8;
        const i32x4_t rsp = sp.rsrc(ks), rsq = sq.rsrc(ks);
        static_for<64>([&](auto I) {
          constexpr int i = decltype(I)::value;
          constexpr int mi = i >> 4, ni = (i >> 2) & 3, s = i & 3, j = i & 15;
          if constexpr (i == 48) {
            // slice kt+1 has landed once only slice kt+2 and kt+NST-1 remain; this
            // wave has read all it needs of stage kt
            wait_vm<(NST - 2) * LOADS8>();
            wait_lgkm0();
            __syncthreads();
            __builtin_amdgcn_sched_barrier(0);
          }
          if constexpr (mi < 3) {
            // the next P fragment: read, then converted half a quarter later
            if constexpr (j < 2) load_p(cur, mi + 1, j);
            if constexpr (j >= 8) widen_p(mi + 1, j - 8, ssp);
            // Q[3], before its first use
            if constexpr (mi == 0 && j < 8) widen_q(3, j, ssq);
          } else {
            // slice kt+1: scales, Q[0..3], P[0]
            if constexpr (j == 0) {
              nsp = *reinterpret_cast<const int32_t*>(next + psc);
              nsq = *reinterpret_cast<const int32_t*>(next + qsc);
            }
            if constexpr (j < 4) {
              load_q(next, j, 0);
              load_q(next, j, 1);
            }
            if constexpr (j >= 4 && j < 6) load_p(next, 0, j - 4);
            if constexpr (j >= 4) {  // Q[ni - 1] has had its last MFMA
              widen_q(ni - 1, 2 * s, nsq);
              widen_q(ni - 1, 2 * s + 1, nsq);
            }
            if constexpr (j >= 8) widen_p(0, j - 8, nsp);
          }
          if constexpr (mi == 1 && (j & 3) == 0) sp.issue_one(rsp, fill, j >> 2);
          if constexpr (mi == 1 && j == 14) ss.issue(ks, fill);
          if constexpr (mi == 2 && (j & 3) == 0) sq.issue_one(rsq, fill + OPB, j >> 2);
          acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(pb[mi & 1].v[s], qb[ni].v[s],
                                                                acc[mi][ni], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        });
        ssp = nsp;
        ssq = nsq;
      }
    }
    wait_vm<0>();  // no load may still target LDS when the block ends
  }

  // acc[mi][ni][4 g + e] of this lane: row 128 wn + 4 lr + ni, column
  // 128 wm + 4 (8 g + 4 lh + e) + mi of the tile.
  T* const cc = static_cast<T*>(d.c);
  const bool vec = d.n % Elt<T>::kVec == 0;
#pragma unroll
  for (int ni = 0; ni < 4; ++ni) {
    const int32_t row = m0 + 128 * wn + 4 * lr + ni;
    if (row >= d.m) continue;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int32_t col = n0 + 128 * wm + 32 * g + 16 * lh;
      float v[16];
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int mi = 0; mi < 4; ++mi) v[4 * e + mi] = acc[mi][ni][4 * g + e];
      if (col < d.n)
        store16(cc + static_cast<int64_t>(row) * d.n + col, v, d.n - col, vec, c.accumulate != 0);
    }
  }
}

hipError_t launch_f8_prod(const F8ProdCtx& c, int32_t ntiles, bool is_bf16) {
  if (ntiles <= 0) return hipSuccess;
  if (is_bf16)
    hipLaunchKernelGGL(k_f8_prod<uint16_t>, dim3(ntiles), dim3(kThreads), 0, c.stream, c);
  else
    hipLaunchKernelGGL(k_f8_prod<float>, dim3(ntiles), dim3(kThreads), 0, c.stream, c);
  return hipGetLastError();
}

}  // namespace muon
