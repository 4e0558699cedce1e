// C = A B^T (+ C) over block-scaled e4m3 operands (F8ProdDesc in
// muon_internal.hpp), ragged over a batch.
//
//   C[m][n] = sum_kb 2^(sa[kb][m]-127) 2^(sb[kb][n]-127) sum_{k in block kb} a[m][k] b[n][k]
//
// The scales are powers of two, so applying them rounds nothing; C is rounded
// once, at the store.  Two ways to the sum:
//  * bf16 C: the scaled matrix instruction (v_mfma_scale_f32_32x32x64_f8f6f4)
//    on the stored bytes.  It adds 8 consecutive products on a common grid
//    before they reach the fp32 accumulator (measured, for products 8 i .. 8 i + 7:
//    one of 2^-13 of the 8's largest counts, one of 2^-14 does not; between groups
//    the sum is fp32's).  That is below 2^-10 of the sum of the magnitudes, and on
//    Gaussian operands 1.5e-5 of the result at any K, far below the 1.7e-3 of the
//    bf16 rounding.
//  * fp32 C: that error would be 250 times the output's own rounding, so the
//    operands are converted on the way from LDS to bf16, scale included
//    (v_cvt_scalef32_pk_bf16_fp8: exact, but for values below bf16's smallest,
//    2^-133, and from 2^128 on, which become infinite), and
//    v_mfma_f32_32x32x16_bf16 sums them with fp32 precision, at half the matrix
//    rate.
//
// 256 x 256 tiles, four waves of 128 x 128, K in blocks of 128 through two LDS
// buffers filled by direct-to-LDS loads, each block in two slices of 64.  The
// operands are row-major, and a load instruction takes the whole 128-byte lines
// of 8 rows: with 64-byte pieces of 16 rows and four buffers of 64 the L2 served
// twice the requests and the loop ran 15% slower (16 products 1024 x 2048 x
// 6144: 217 us against 184 with whole lines).  Rows past the operand's end
// repeat its last one: what they give is not stored.
//   The first matrix operand (P) is B, the second (Q) A: a lane's registers
// then run along a row of C.  LDS row 128 h + 32 i + r holds the tile's row
// 128 h + 4 r + i (RowStream), so that lane r of fragment i works on row 4 r + i: the
// scales of a lane's four fragments are one aligned dword of the scale row
// (op_sel picks the byte), and a lane's registers hold 16 consecutive columns
// of C for each of its rows.
#include <utility>

#include "gemm_pipeline.hpp"

namespace muon {

namespace {

static_assert(kF8Tile == kTile, "the pipeline's tile");
constexpr int LROW = kF8Block;             // bytes of an LDS row: one K block of one row
constexpr int OPB8 = kTile * LROW;         // 32 KiB per operand and buffer
constexpr int SCB = 256;                   // scale bytes per operand and buffer
constexpr int BUF8 = 2 * OPB8 + 2 * SCB;   // P data, Q data, P scales, Q scales
constexpr int LDS8 = 2 * BUF8;
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

// One operand's 64 N rows of the tile (N = 4; 2 or 1 for A in a half or quarter
// tile), 128
// bytes of each per block.  LDS row 32 (N h + i) + r holds tile row
// 32 N h + N r + i, its 16-byte chunk c at c ^ ((r / 2) % 8): the rows of a
// fragment read then fall on distinct banks.
template <int N>
struct RowStream {
  static constexpr int kLoads = 2 * N;  // per wave and block
  const uint8_t* base;  // the tile's first row (uniform)
  uint32_t bytes;       // of the tile's rows that exist
  int32_t voff[kLoads];  // per-lane offsets, one per load instruction
  int32_t lds;          // LDS offset of this wave's first 1 KiB block, within the operand

  __device__ __forceinline__ void init(const uint8_t* rows0, int32_t valid, int32_t kp, int wave,
                                       int lane) {
    base = rows0;
    bytes = static_cast<uint32_t>(valid) * static_cast<uint32_t>(kp);
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int s = 8 * (kLoads * wave + u) + (lane >> 3);
      const int row = s / (32 * N) * (32 * N) + N * (s & 31) + (s >> 5) % N;
      voff[u] = (row < valid ? row : valid - 1) * kp + (((lane & 7) ^ ((s >> 1) & 7)) << 4);
    }
    lds = kLoads * wave * 1024;
  }
  __device__ __forceinline__ i32x4_t rsrc(int kb) const {
    return make_rsrc(base + static_cast<int64_t>(kb) * kF8Block, bytes - static_cast<uint32_t>(kF8Block) * kb);
  }
  __device__ __forceinline__ void issue_one(const i32x4_t& r, uint32_t at, int u) const {
    lds_dma16(__builtin_amdgcn_readfirstlane(at + lds + u * 1024), voff[u], r);
  }
  __device__ __forceinline__ void issue(int kb, uint32_t at) const {
    const i32x4_t r = rsrc(kb);
#pragma unroll
    for (int u = 0; u < kLoads; ++u) issue_one(r, at, u);
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
    lds = 2 * OPB8 + (wave & 1) * SCB;
  }
  __device__ __forceinline__ void issue(int kb, uint32_t at) const {
    const i32x4_t r = make_rsrc(base + static_cast<int64_t>(kb) * rp, 256);
    lds_dma4(__builtin_amdgcn_readfirstlane(at + lds), voff, r);
  }
};

template <int NQ>
struct Frags8 {
  i32x8_t p[4];    // dwords 0-3: chunk h of the slice's 64 bytes, 4-7: chunk 2 + h
  i32x8_t q[NQ];
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

// Stores the wave's 32 NQ x 128 part of the tile, whose first element is row
// m0, column n0 of C.  acc[mi][ni][4 g + e] of lane (lr, lh) is row NQ lr + ni,
// column 4 (8 g + 4 lh + e) + mi.  The 32 rows of one ni go through 16 KiB of
// LDS of the wave's own in fp32, four columns (the four mi) a 16-byte chunk,
// chunk c of row r at c ^ r; they come out as whole rows, so that every store
// covers full 128-byte lines (written from the accumulators, 16 bytes a row,
// the store ran at 2.5 TB/s).  ADD: the old C of one ni is requested while the
// one before it is stored.  NT: C passes the caches by (F8ProdCtx::nt).  Rows of C
// whose length is no multiple of a lane's 16 bytes go element by element: 16
// products 1024 x 2047 x 6144, bf16: 196 us against 167 of 2048 columns, added to an
// old C 262 against 185.
template <typename T, bool ADD, int NQ, bool NT>
__device__ __forceinline__ void store_part(const f32x16_t (&acc)[4][NQ], char* lds, T* c, int32_t m0,
                                           int32_t n0, int32_t m, int32_t n, int lane) {
  constexpr int V = Elt<T>::kVec;            // columns per lane: 16 bytes
  constexpr int LPR = 128 / V;               // lanes per row
  constexpr int RPI = 64 / LPR;              // rows per instruction
  constexpr int NI = 32 / RPI;               // instructions per ni
  const int lr = lane & 31, lh = lane >> 5;
  const int rr0 = lane / LPR, ch = lane % LPR * (V / 4);
  const int32_t col = n0 + lane % LPR * V;
  const bool vec = n % V == 0;               // then a lane's columns all exist, or none
  const bool fast = vec && col < n;
  T* const corner = c + static_cast<int64_t>(m0) * n + col;
  u32x4_t old[2][ADD ? NI : 1];
  auto request = [&](int ni, u32x4_t* to) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int32_t r = NQ * (RPI * i + rr0) + ni;
      if (fast && m0 + r < m) {
        const T* const at = corner + static_cast<int64_t>(r) * n;
        to[i] = NT ? ld16_nt(at) : ld16(at);
      }
    }
  };
  if constexpr (ADD) request(0, old[0]);
#pragma unroll
  for (int ni = 0; ni < NQ; ++ni) {
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f32x4_t x;
#pragma unroll
        for (int mi = 0; mi < 4; ++mi) x[mi] = acc[mi][ni][4 * g + e];
        *reinterpret_cast<f32x4_t*>(lds + lr * 512 + (((8 * g + 4 * lh + e) ^ lr) << 4)) = x;
      }
    __builtin_amdgcn_wave_barrier();
    if constexpr (ADD)
      if (ni + 1 < NQ) request(ni + 1, old[(ni + 1) & 1]);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int rr = RPI * i + rr0;
      float v[V];
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        const f32x4_t x = *reinterpret_cast<const f32x4_t*>(lds + rr * 512 + (((ch + q) ^ rr) << 4));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * q + e] = x[e];
      }
      const int32_t r = NQ * rr + ni;
      if (m0 + r >= m || col >= n) continue;
      T* const to = corner + static_cast<int64_t>(r) * n;
      if (fast) {
        if constexpr (ADD) {
          float o[V];
          vec_to_f32<T>(old[ni & 1][i], o);
#pragma unroll
          for (int e = 0; e < V; ++e) v[e] += o[e];
        }
        if constexpr (NT)
          st16_nt(to, f32_to_vec<T>(v));
        else
          st16(to, f32_to_vec<T>(v));
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (col + e < n) to[e] = Elt<T>::from_f32(ADD ? v[e] + Elt<T>::to_f32(to[e]) : v[e]);
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// One tile: 256 columns of C from n0, 64 NQ rows from m0.
template <typename T, bool ADD, int NQ>
__device__ __forceinline__ void prod_tile(const F8ProdDesc& d, int32_t m0, int32_t n0, char* smem,
                                          bool nt) {
  constexpr int kRows = 64 * NQ;
  constexpr int kPLoads = RowStream<4>::kLoads, kQLoads = RowStream<NQ>::kLoads;
  constexpr int kLoads = kPLoads + kQLoads + 1;  // per wave and block
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int lr = lane & 31, lh = lane >> 5;

  f32x16_t acc[4][NQ];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int k = 0; k < NQ; ++k)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][k][e] = 0.f;

  const int nb = d.kp / kF8Block;
  if (nb > 0) {
    RowStream<4> sp;
    RowStream<NQ> sq;
    sp.init(d.b + static_cast<int64_t>(n0) * d.kp, min(kTile, d.n - n0), d.kp, wave, lane);
    sq.init(d.a + static_cast<int64_t>(m0) * d.kp, min(kRows, d.m - m0), d.kp, wave, lane);
    ScaleRows ss;
    if (wave & 1)
      ss.init(d.sa, m0, d.m, wave, lane);
    else
      ss.init(d.sb, n0, d.n, wave, lane);

    // Offsets of this lane's two chunks of a fragment row in slice 0 and 1 of a
    // block: chunks h and 2 + h, and 4 more.
    int32_t poff[2][2], qoff[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int x = ((2 * h + lh) ^ ((lr >> 1) & 7)) << 4;
      poff[0][h] = (wm * 128 + lr) * LROW + x;
      poff[1][h] = poff[0][h] ^ 64;
      qoff[0][h] = OPB8 + (wn * 32 * NQ + lr) * LROW + x;
      qoff[1][h] = qoff[0][h] ^ 64;
    }
    const int32_t psc = 2 * OPB8 + 4 * (32 * wm + lr);
    const int32_t qsc = 2 * OPB8 + SCB + NQ * (32 * wn + lr);
    auto p_scales = [&](const char* buf) { return *reinterpret_cast<const int32_t*>(buf + psc); };
    auto q_scales = [&](const char* buf) -> int32_t {
      if constexpr (NQ == 4)
        return *reinterpret_cast<const int32_t*>(buf + qsc);
      else if constexpr (NQ == 2)
        return *reinterpret_cast<const uint16_t*>(buf + qsc);
      else
        return *reinterpret_cast<const uint8_t*>(buf + qsc);
    };

    const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((LDS_AS char*)smem));
    // Requests number 0 .. kLoads - 1 of a block: P's, the scales, Q's.  Block
    // indices past the end are clamped to the last block: those loads refill a
    // buffer nobody reads again and keep the count in flight constant.
    auto request = [&](int kb, uint32_t at, const i32x4_t& rp, const i32x4_t& rq, auto U) {
      constexpr int u = decltype(U)::value;
      if constexpr (u < kPLoads)
        sp.issue_one(rp, at, u);
      else if constexpr (u == kPLoads)
        ss.issue(kb, at);
      else
        sq.issue_one(rq, at + OPB8, u - kPLoads - 1);
    };
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int kb = b < nb ? b : nb - 1;
      sp.issue(kb, lds0 + b * BUF8);
      ss.issue(kb, lds0 + b * BUF8);
      sq.issue(kb, lds0 + b * BUF8 + OPB8);
    }
    wait_vm<kLoads>();  // block 0
    __syncthreads();

    if constexpr (sizeof(T) == 2) {
      // Fragment reads in the order the MFMAs consume them: the scales, P[0],
      // the Qs, then P[1..3]; two 16-byte reads per fragment.
      constexpr int kReads = 2 + 2 * (4 + NQ), kMfma = 4 * NQ, kHalf = kMfma / 2;
      auto read_op = [&](Frags8<NQ>& f, const char* buf, int sub, int i) {
        if (i == 0) {
          f.sp = p_scales(buf);
        } else if (i == 1) {
          f.sq = q_scales(buf);
        } else if (i < 4) {
          set_half(f.p[0], i - 2, lds16(buf + poff[sub][i - 2]));
        } else if (i < 4 + 2 * NQ) {
          const int ni = (i - 4) >> 1, h = (i - 4) & 1;
          set_half(f.q[ni], h, lds16(buf + qoff[sub][h] + ni * 32 * LROW));
        } else {
          const int mi = 1 + ((i - 4 - 2 * NQ) >> 1), h = (i - 4) & 1;
          set_half(f.p[mi], h, lds16(buf + poff[sub][h] + mi * 32 * LROW));
        }
      };
      Frags8<NQ> f0, f1;
#pragma unroll
      for (int i = 0; i < kReads; ++i) read_op(f0, smem, 0, i);

      // Block b: slice 0 on f0, slice 1 on f1.  Slice 1's fragments are read in
      // the first half of slice 0; every wave has then left the buffer, and block
      // b + 2 is requested into it from the second half of slice 0 (P) to the
      // first half of slice 1 (scales, Q).  Slice 1 reads block b + 1's first
      // fragments.
      constexpr int kEarly = kPLoads;  // requests issued in slice 0
      for (int b = 0; b < nb; ++b) {
        const char* const cur = smem + (b & 1) * BUF8;
        const char* const next = smem + ((b + 1) & 1) * BUF8;
        const uint32_t fill = lds0 + (b & 1) * BUF8;
        const int kb = b + 2 < nb ? b + 2 : nb - 1;
        const i32x4_t rp = sp.rsrc(kb), rq = sq.rsrc(kb);
        static_for<kMfma>([&](auto I) {
          constexpr int i = decltype(I)::value, mi = i / NQ, ni = i % NQ;
          if constexpr (i < kHalf) {
#pragma unroll
            for (int r = i * kReads / kHalf; r < (i + 1) * kReads / kHalf; ++r) read_op(f1, cur, 1, r);
          }
          if constexpr (i == kHalf) {
            wait_lgkm0();  // this wave's reads of the buffer are done
            __syncthreads();
            __builtin_amdgcn_sched_barrier(0);
          }
          if constexpr (i >= kHalf) {
            static_for<kEarly / kHalf>([&](auto U) {
              request(kb, fill, rp, rq,
                      std::integral_constant<int, (i - kHalf) * (kEarly / kHalf) + decltype(U)::value>{});
            });
          }
          acc[mi][ni] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              f0.p[mi], f0.q[ni], acc[mi][ni], 0, 0, mi, f0.sp, ni, f0.sq);
          __builtin_amdgcn_sched_barrier(0);
        });
        wait_vm<kEarly>();  // block b + 1 has landed
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
        static_for<kMfma>([&](auto I) {
          constexpr int i = decltype(I)::value, mi = i / NQ, ni = i % NQ;
#pragma unroll
          for (int r = i * kReads / kMfma; r < (i + 1) * kReads / kMfma; ++r) read_op(f0, next, 0, r);
          if constexpr (i == 0) request(kb, fill, rp, rq, std::integral_constant<int, kPLoads>{});
          if constexpr (i < kHalf) {
            static_for<kQLoads / kHalf>([&](auto U) {
              request(kb, fill, rp, rq,
                      std::integral_constant<int, kPLoads + 1 + i * (kQLoads / kHalf) + decltype(U)::value>{});
            });
          }
          acc[mi][ni] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              f1.p[mi], f1.q[ni], acc[mi][ni], 0, 0, mi, f1.sp, ni, f1.sq);
          __builtin_amdgcn_sched_barrier(0);
        });
      }
    } else {
      // Fragments of a slice are converted one step ahead of the MFMAs that take
      // them, between MFMAs.  On entry to a slice: P[0] and the Qs but the last
      // converted, the last Q raw.  A quarter of a slice is one P fragment; the
      // last quarter turns to the next slice.  The last quarter of a block's slice
      // 1 leaves its buffer; block b + 2 is requested into it from there to the
      // third quarter of the next slice.
      constexpr int kQuarter = 4 * NQ, kPer = 4 / NQ;  // dwords converted per MFMA
      constexpr int kLast = NQ - 1;
      Wide qb[NQ], pb[2];
      i32x8_t rq[NQ], rp;
      int32_t ssp, ssq, nsp = 0, nsq = 0;
      auto load_q = [&](const char* buf, int sub, int ni, int h) {
        set_half(rq[ni], h, lds16(buf + qoff[sub][h] + ni * 32 * LROW));
      };
      auto load_p = [&](const char* buf, int sub, int mi, int h) {
        set_half(rp, h, lds16(buf + poff[sub][h] + mi * 32 * LROW));
      };
      auto widen_q = [&](int ni, int d, int32_t sc) { widen(qb[ni], d, rq[ni][d], scale_value(sc, ni)); };
      auto widen_p = [&](int mi, int d, int32_t sc) { widen(pb[mi & 1], d, rp[d], scale_value(sc, mi)); };
      ssp = p_scales(smem);
      ssq = q_scales(smem);
#pragma unroll
      for (int ni = 0; ni < NQ; ++ni)
#pragma unroll
        for (int h = 0; h < 2; ++h) load_q(smem, 0, ni, h);
#pragma unroll
      for (int h = 0; h < 2; ++h) load_p(smem, 0, 0, h);
#pragma unroll
      for (int d = 0; d < 8; ++d) {
#pragma unroll
        for (int ni = 0; ni < kLast; ++ni) widen_q(ni, d, ssq);
        widen_p(0, d, ssp);
      }
      // One slice: `sub` of the block in `cur`; the last quarter reads the other
      // slice of the block in `next`.  Requests are for block kb, into `fill`.
      auto slice = [&](auto SUB, const char* cur, const char* next, int kb, uint32_t fill,
                       const i32x4_t& drp, const i32x4_t& drq) {
        constexpr int sub = decltype(SUB)::value, nsub = sub ^ 1;
        static_for<4 * kQuarter>([&](auto I) {
          constexpr int i = decltype(I)::value;
          constexpr int mi = i / kQuarter, ni = (i >> 2) % NQ, s = i & 3, j = i % kQuarter;
          if constexpr (sub == 1 && i == 3 * kQuarter) {
            wait_vm<0>();  // block b + 1 has landed: nothing else is in flight
            wait_lgkm0();  // this wave has left the buffer
            __syncthreads();
            __builtin_amdgcn_sched_barrier(0);
          }
          if constexpr (mi < 3) {
            // the next P fragment: read, then converted half a quarter later
            if constexpr (j < 2) load_p(cur, sub, mi + 1, j);
            if constexpr (j >= kQuarter / 2)
#pragma unroll
              for (int k = 0; k < kPer; ++k) widen_p(mi + 1, (j - kQuarter / 2) * kPer + k, ssp);
            // the last Q, before its first use
            if constexpr (mi == 0 && j < kQuarter / 2)
#pragma unroll
              for (int k = 0; k < kPer; ++k) widen_q(kLast, j * kPer + k, ssq);
          } else {
            // the next slice: scales, the Qs, P[0]
            if constexpr (j == 0) {
              nsp = p_scales(next);
              nsq = q_scales(next);
            }
            if constexpr (j < NQ) {
              load_q(next, nsub, j, 0);
              load_q(next, nsub, j, 1);
            }
            if constexpr (j >= NQ && j < NQ + 2) load_p(next, nsub, 0, j - NQ);
            if constexpr (ni > 0) {  // Q[ni - 1] has had its last MFMA
              widen_q(ni - 1, 2 * s, nsq);
              widen_q(ni - 1, 2 * s + 1, nsq);
            }
            if constexpr (j >= kQuarter / 2)
#pragma unroll
              for (int k = 0; k < kPer; ++k) widen_p(0, (j - kQuarter / 2) * kPer + k, nsp);
          }
          // four requests of a block in slice 1, the others in slice 0
          if constexpr (sub == 1 && mi == 3 && j % NQ == NQ - 1)
            request(kb, fill, drp, drq, std::integral_constant<int, j / NQ>{});
          if constexpr (sub == 0 && mi < 3) {
            constexpr int kRest = kLoads - 4, kSpan = 3 * kQuarter;
            constexpr int a = i * kRest / kSpan, z = (i + 1) * kRest / kSpan;
            if constexpr (z > a) request(kb, fill, drp, drq, std::integral_constant<int, 4 + a>{});
          }
          acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(pb[mi & 1].v[s], qb[ni].v[s],
                                                                acc[mi][ni], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        });
        ssp = nsp;
        ssq = nsq;
      };
      // Slice 0 of block b goes on with the requests for block b + 1 that slice 1
      // of block b - 1 began.  (Block 0's repeats part of those for block 1, the
      // same bytes to the same place.)
      for (int b = 0; b < nb; ++b) {
        const char* const cur = smem + (b & 1) * BUF8;
        const char* const next = smem + ((b + 1) & 1) * BUF8;
        const int kb1 = b + 1 < nb ? b + 1 : nb - 1, kb2 = b + 2 < nb ? b + 2 : nb - 1;
        const i32x4_t p1 = sp.rsrc(kb1), q1 = sq.rsrc(kb1);
        slice(std::integral_constant<int, 0>{}, cur, cur, kb1, lds0 + ((b + 1) & 1) * BUF8, p1, q1);
        const i32x4_t p2 = sp.rsrc(kb2), q2 = sq.rsrc(kb2);
        slice(std::integral_constant<int, 1>{}, cur, next, kb2, lds0 + (b & 1) * BUF8, p2, q2);
      }
    }
    wait_vm<0>();  // no load may still target LDS: the buffers are reused for the store
  }
  __syncthreads();
  if (nt)
    store_part<T, ADD, NQ, true>(acc, smem + wave * 16384, static_cast<T*>(d.c), m0 + 32 * NQ * wn,
                                 n0 + 128 * wm, d.m, d.n, lane);
  else
    store_part<T, ADD, NQ, false>(acc, smem + wave * 16384, static_cast<T*>(d.c), m0 + 32 * NQ * wn,
                                  n0 + 128 * wm, d.m, d.n, lane);
}

}  // namespace

namespace {

// Block `blk` of the n that the prefixes number: its product (*j) and its tile
// there.  Each XCD takes one contiguous range of the launch (neighbouring tiles
// share operands), or, with `spread`, one contiguous eighth of every product:
// block g then belongs to the product that holds g, and the product's blocks of
// one XCD (equal g % 8) become neighbours.
__device__ __forceinline__ int32_t place_block(const F8ProdCtx& c, const int32_t* prefix,
                                               int32_t blk, int32_t n, int* slot, int* j) {
  const int32_t b = c.spread ? blk : xcd_remap(blk, n);
  *j = __builtin_amdgcn_readfirstlane(locate_matrix(prefix, c.batch, b, slot));
  const int32_t p0 = load_const(prefix + *j);
  if (!c.spread) return b - p0;
  const int32_t p1 = load_const(prefix + *j + 1), x = blk % kXcd;
  // blocks below p on XCDs below x, and on XCD x
  auto before = [&](int32_t p) { return p / kXcd * x + min(p % kXcd, x); };
  auto mine = [&](int32_t p) { return (p + kXcd - 1 - x) / kXcd; };
  return before(p1) - before(p0) + blk / kXcd - mine(p0);
}

}  // namespace

// The launch's tiles: full ones of 256 x 256 first, then half ones of 128 x 256
// and quarter ones of 64 x 256 (F8ProdDesc: the product's rows of each; the
// quarter ones take the rest), which end ragged products and fill the launch's
// last round.  All of them add every element up the same way.
template <typename T, bool ADD>
__global__ __launch_bounds__(kThreads, 1) void k_f8_prod(ArgTable, F8ProdCtx c, int32_t nfull,
                                                         int32_t nhalf) {
  __shared__ __attribute__((aligned(1024))) char smem[LDS8];
  __shared__ int slot;
  const char* const table = table_base(c.table);
  int32_t blk = blockIdx.x, n = nfull, kind = 0;
  if (blk >= nfull) {
    blk -= nfull;
    n = nhalf;
    kind = 1;
    if (blk >= nhalf) {
      blk -= nhalf;
      n = static_cast<int32_t>(gridDim.x) - nfull - nhalf;
      kind = 2;
    }
  }
  const int32_t* const prefix =
      reinterpret_cast<const int32_t*>(table + c.prefix_off) + kind * (c.batch + 1);
  int j;
  const int32_t t = place_block(c, prefix, blk, n, &slot, &j);
  const F8ProdDesc d = load_const(reinterpret_cast<const F8ProdDesc*>(table) + j);
  const int32_t full = d.full, half = d.half;
  // down a column of tiles: B stays
  if (kind == 0) {
    prod_tile<T, ADD, 4>(d, t % full * kTile, t / full * kTile, smem, c.nt != 0);
  } else if (kind == 1) {
    prod_tile<T, ADD, 2>(d, full * kTile + t % half * (kTile / 2), t / half * kTile, smem,
                         c.nt != 0);
  } else {
    const int32_t row0 = full * kTile + half * (kTile / 2);
    const int32_t rows = (d.m - row0 + kTile / 4 - 1) / (kTile / 4);
    prod_tile<T, ADD, 1>(d, row0 + t % rows * (kTile / 4), t / rows * kTile, smem, c.nt != 0);
  }
}

// ---------------------------------------------------------------------------
// Few rows, or a batch of few tiles: blocks of 16 MT rows of A by 16 NT rows of
// B, the K blocks of 128 dealt to the four waves (kb = wave, wave + 4, ...) and
// the four partial tiles joined through LDS in a fixed order.  Each wave streams
// its own K blocks through LDS of its own, kStages deep, with no barrier until
// the join: direct-to-LDS loads of whole 128-byte rows.  (Loaded straight into
// registers, where neighbouring lanes sit in different rows, a load took 64
// cycles of the address unit instead of 16, and that bounded the kernel.)
//   v_mfma_f32_16x16x.. with B as its first operand: lane (r, g) holds the
// 16-byte chunks g and 4 + g of row r's 128 bytes (both operands alike, so the
// order of K within them does not matter).  Row r of B's fragment t is row
// NT r + t of the tile, so that a lane's NT scales are neighbours and its
// results 4 NT consecutive columns of C.  Chunk c of LDS row s sits at
// c ^ ((s / 2) % 8): the 16 rows of a fragment read fall on distinct banks.
// ---------------------------------------------------------------------------
namespace {

__device__ __forceinline__ i32x8_t joined(const u32x4_t& lo, const u32x4_t& hi) {
  typedef uint32_t u32x8_t __attribute__((ext_vector_type(8)));
  const u32x8_t v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(i32x8_t, v);
}

// Waits until at most N of this wave's loads are in flight; the compiler moves
// no memory access across it.
template <int N>
__device__ __forceinline__ void await_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// The rows of one operand, 128 bytes of each per K block: N fragments of 16.
template <int N>
struct SmallStream {
  const uint8_t* base;    // the tile's first row (uniform)
  const uint8_t* scales;  // scale row 0 at the tile's first row (uniform)
  uint32_t bytes;         // of the tile's rows that exist
  int32_t rp;             // bytes of a scale row
  int32_t voff[2 * N];
  int32_t soff;

  // STRIDE: tile row of LDS row 16 t + r is N r + t (B) or 16 t + r (A).
  template <bool STRIDE>
  __device__ __forceinline__ void init(const uint8_t* q, const uint8_t* s, int32_t row0,
                                       int32_t rows, int32_t kp, int lane) {
    const int32_t valid = min(16 * N, rows - row0);
    base = q + static_cast<int64_t>(row0) * kp;
    bytes = static_cast<uint32_t>(valid) * static_cast<uint32_t>(kp);
    scales = s + row0;
    rp = (rows + 15) & ~15;
#pragma unroll
    for (int u = 0; u < 2 * N; ++u) {
      const int l = 8 * u + (lane >> 3);  // LDS row
      const int row = STRIDE ? N * (l & 15) + (l >> 4) : l;
      voff[u] = min(row, valid - 1) * kp + (((lane & 7) ^ ((l >> 1) & 7)) << 4);
    }
    soff = min(4 * lane, rp - 4 - row0);
  }
  __device__ __forceinline__ void issue(int kb, uint32_t lds, uint32_t lds_scales) const {
    const i32x4_t r = make_rsrc(base + static_cast<int64_t>(kb) * kF8Block,
                                bytes - static_cast<uint32_t>(kb) * kF8Block);
#pragma unroll
    for (int u = 0; u < 2 * N; ++u) lds_dma16(lds + 1024 * u, voff[u], r);
    lds_dma4(lds_scales, soff, make_rsrc(scales + static_cast<int64_t>(kb) * rp, 256));
  }
};

template <int N>
__device__ __forceinline__ int32_t lds_scales(const char* p) {
  if constexpr (N == 4)
    return *reinterpret_cast<const int32_t*>(p);
  else if constexpr (N == 2)
    return *reinterpret_cast<const uint16_t*>(p);
  else
    return *reinterpret_cast<const uint8_t*>(p);
}

template <int MT, int NT>
struct SmallShape {
  static constexpr int kA = 2048 * NT, kSB = kA + 2048 * MT, kSA = kSB + 256;  // within a stage
  static constexpr int kStageBytes = kSA + 256;
  static constexpr int kStages = 4 * 3 * kStageBytes <= 152 * 1024 ? 3 : 2;
  static constexpr int kWaveBytes = kStages * kStageBytes;
  static constexpr int kPitch = 16 * NT + 4;  // floats per row of a partial tile
  static constexpr int kLoads = 2 * NT + 2 * MT + 2;  // per stage
  static_assert(16 * MT * kPitch * 4 <= kWaveBytes, "a partial tile fits the wave's ring");
};

}  // namespace

template <typename T, int MT, int NT>
__global__ __launch_bounds__(kThreads) void k_f8_small(ArgTable, F8ProdCtx c) {
  using S = SmallShape<MT, NT>;
  constexpr int BM = 16 * MT, BN = 16 * NT, PITCH = S::kPitch;
  __shared__ __attribute__((aligned(1024))) char smem[4 * S::kWaveBytes];
  __shared__ int slot;
  const char* const table = table_base(c.table);
  const int32_t* const prefix = reinterpret_cast<const int32_t*>(table + c.prefix_off);
  int j;
  const int32_t t = place_block(c, prefix, blockIdx.x, gridDim.x, &slot, &j);
  const F8ProdDesc d = load_const(reinterpret_cast<const F8ProdDesc*>(table) + j);
  const int32_t tm = (d.m + BM - 1) / BM;
  const int32_t m0 = t % tm * BM, n0 = t / tm * BN;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  char* const mine = smem + wave * S::kWaveBytes;

  f32x4_t acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int k = 0; k < NT; ++k) acc[i][k] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  const int nkb = d.kp / kF8Block;
  const int steps = (nkb - wave + 3) / 4;  // of this wave; 0 or less: none
  if (steps > 0) {
    SmallStream<NT> sb;
    SmallStream<MT> sa;
    sb.template init<true>(d.b, d.sb, n0, d.n, d.kp, lane);
    sa.template init<false>(d.a, d.sa, m0, d.m, d.kp, lane);
    const uint32_t ring = __builtin_amdgcn_readfirstlane(
        static_cast<uint32_t>(reinterpret_cast<uintptr_t>((LDS_AS char*)mine)));
    // Past the end the last block is loaded again: nobody reads it, and the
    // count in flight stays constant.
    auto issue = [&](int s, int stage) {
      const int kb = wave + 4 * min(s, steps - 1);
      const uint32_t at = ring + stage * S::kStageBytes;
      sb.issue(kb, at, at + S::kSB);
      sa.issue(kb, at + S::kA, at + S::kSA);
    };
#pragma unroll
    for (int s = 0; s < S::kStages - 1; ++s) issue(s, s);
    const int ch0 = (g ^ ((r >> 1) & 7)) << 4, ch1 = ((4 + g) ^ ((r >> 1) & 7)) << 4;
    int stage = 0;
    for (int s = 0; s < steps; ++s) {
      // refill the stage read in the last step
      issue(s + S::kStages - 1, stage == 0 ? S::kStages - 1 : stage - 1);
      await_loads<(S::kStages - 1) * S::kLoads>();
      const char* const at = mine + stage * S::kStageBytes;
      u32x4_t b[NT][2], a[MT][2];
      int32_t xa[MT];
      const int32_t xb = lds_scales<NT>(at + S::kSB + NT * r);
#pragma unroll
      for (int i = 0; i < MT; ++i) xa[i] = lds_scales<1>(at + S::kSA + 16 * i + r);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        a[i][0] = lds16(at + S::kA + (16 * i + r) * 128 + ch0);
        a[i][1] = lds16(at + S::kA + (16 * i + r) * 128 + ch1);
      }
#pragma unroll
      for (int k = 0; k < NT; ++k) {
        b[k][0] = lds16(at + (16 * k + r) * 128 + ch0);
        b[k][1] = lds16(at + (16 * k + r) * 128 + ch1);
      }
      if constexpr (sizeof(T) == 2) {
        static_for<NT>([&](auto K) {
          constexpr int k = decltype(K)::value;
          const i32x8_t fb = joined(b[k][0], b[k][1]);
          static_for<MT>([&](auto I) {
            constexpr int i = decltype(I)::value;
            acc[i][k] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                fb, joined(a[i][0], a[i][1]), acc[i][k], 0, 0, k, xb, 0, xa[i]);
          });
        });
      } else {
        Wide wa[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int q = 0; q < 8; ++q)
            widen(wa[i], q, static_cast<int32_t>(a[i][q >> 2][q & 3]), scale_value(xa[i], 0));
#pragma unroll
        for (int k = 0; k < NT; ++k) {
          Wide wb;
#pragma unroll
          for (int q = 0; q < 8; ++q)
            widen(wb, q, static_cast<int32_t>(b[k][q >> 2][q & 3]), scale_value(xb, k));
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < MT; ++i)
              acc[i][k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb.v[q], wa[i].v[q], acc[i][k], 0, 0, 0);
        }
      }
      wait_lgkm0();  // the reads are done before the stage is refilled
      stage = stage + 1 == S::kStages ? 0 : stage + 1;
    }
    await_loads<0>();  // no load may still target LDS: the ring is reused for the join
  }

  // acc[i][k][e] of lane (r, g): row 16 i + r, column NT (4 g + e) + k
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float* to = reinterpret_cast<float*>(mine) + (16 * i + r) * PITCH + NT * (4 * g + e);
#pragma unroll
      for (int k = 0; k < NT; ++k) to[k] = acc[i][k][e];
    }
  __syncthreads();
  constexpr int LPR = BN / 4;  // threads per row, four columns each
  const int32_t col = n0 + 4 * static_cast<int>(threadIdx.x % LPR);
  const bool vec = d.n % 4 == 0;
  T* const cc = static_cast<T*>(d.c);
  for (int rr = threadIdx.x / LPR; rr < BM; rr += kThreads / LPR) {
    const int32_t row = m0 + rr;
    if (row >= d.m || col >= d.n) break;
    const float* from = reinterpret_cast<const float*>(smem) + rr * PITCH + 4 * (threadIdx.x % LPR);
    constexpr int W = S::kWaveBytes / 4;
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = ((from[e] + from[W + e]) + from[2 * W + e]) + from[3 * W + e];
    T* to = cc + static_cast<int64_t>(row) * d.n + col;
    if (vec) {
      if (c.accumulate) {
        float o[4];
        load4<T>(to, o);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += o[e];
      }
      store4<T>(to, v);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + e < d.n)
          to[e] = Elt<T>::from_f32(c.accumulate ? v[e] + Elt<T>::to_f32(to[e]) : v[e]);
    }
  }
}

namespace {

template <typename T>
hipError_t run_small(const ArgTable& t, const F8ProdCtx& c, int32_t nblocks, int32_t mt,
                     int32_t nt) {
  const dim3 grid(nblocks), block(kThreads);
  if (nt == 4) {
    if (mt == 1)
      hipLaunchKernelGGL((k_f8_small<T, 1, 4>), grid, block, 0, c.stream, t, c);
    else if (mt == 2)
      hipLaunchKernelGGL((k_f8_small<T, 2, 4>), grid, block, 0, c.stream, t, c);
    else
      hipLaunchKernelGGL((k_f8_small<T, 4, 4>), grid, block, 0, c.stream, t, c);
  } else if (nt == 2) {
    if (mt == 1)
      hipLaunchKernelGGL((k_f8_small<T, 1, 2>), grid, block, 0, c.stream, t, c);
    else if (mt == 2)
      hipLaunchKernelGGL((k_f8_small<T, 2, 2>), grid, block, 0, c.stream, t, c);
    else
      hipLaunchKernelGGL((k_f8_small<T, 4, 2>), grid, block, 0, c.stream, t, c);
  } else {
    if (mt == 1)
      hipLaunchKernelGGL((k_f8_small<T, 1, 1>), grid, block, 0, c.stream, t, c);
    else if (mt == 2)
      hipLaunchKernelGGL((k_f8_small<T, 2, 1>), grid, block, 0, c.stream, t, c);
    else
      hipLaunchKernelGGL((k_f8_small<T, 4, 1>), grid, block, 0, c.stream, t, c);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_f8_small(const ArgTable& t, const F8ProdCtx& c, int32_t nblocks, bool is_bf16,
                           int32_t mt, int32_t nt) {
  if (nblocks <= 0) return hipSuccess;
  return is_bf16 ? run_small<uint16_t>(t, c, nblocks, mt, nt)
                 : run_small<float>(t, c, nblocks, mt, nt);
}

namespace {

template <typename T>
hipError_t run_prod(const ArgTable& t, const F8ProdCtx& c, int32_t nfull, int32_t nhalf,
                    int32_t nquarter) {
  const dim3 grid(nfull + nhalf + nquarter);
  if (c.accumulate)
    hipLaunchKernelGGL((k_f8_prod<T, true>), grid, dim3(kThreads), 0, c.stream, t, c, nfull, nhalf);
  else
    hipLaunchKernelGGL((k_f8_prod<T, false>), grid, dim3(kThreads), 0, c.stream, t, c, nfull, nhalf);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_f8_prod(const ArgTable& t, const F8ProdCtx& c, int32_t nfull, int32_t nhalf,
                          int32_t nquarter, bool is_bf16) {
  if (nfull + nhalf + nquarter <= 0) return hipSuccess;
  return is_bf16 ? run_prod<uint16_t>(t, c, nfull, nhalf, nquarter)
                 : run_prod<float>(t, c, nfull, nhalf, nquarter);
}

}  // namespace muon
