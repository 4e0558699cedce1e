// Tokens to the experts and back.  Slot s = t K + k of token t is its k-th
// expert's id; ids outside 0 .. E - 1 are dropped.
//
//   offsets[e] = number of kept slots with a smaller id
//   rows[s]    = offsets[e_s] + number of slots s' < s with the same id (-1: dropped)
//   slots[p]   = the slot with rows[s] = p (-1 behind the last)
//   dispatch:  xs[rows[s]] = x[t]
//   combine:   out[t] = sum_k w[s] y[rows[s]], in fp32, k ascending, rounded once
//   backward:  dy[rows[s]] = w[s] dout[t],  dw[s] = sum_c dout[t][c] y[rows[s]][c]
//
// Nothing depends on the order in which blocks or waves run: equal calls give
// equal bits.
//
// Dispatch, combine and its gradient are bound by the rows' bytes: a token's row is
// read once, the rows of up to kBatch of its slots are asked for (or stored)
// together.  4096 tokens x 8 x 6144 bf16: 79, 82 and 160 us (5.7, 5.5 and 5.3 TB/s; a slot
// after the other, 92, 98 and 184).  Rows whose length is no multiple of 16 bytes are
// read and written 16 bytes at a time all the same, at element-aligned addresses
// (16384 x 4 x 1001 bf16: 30, 32 and 58 us; by elements 34, 60 and 121).
//
// The sort: a few slots in a kernel that compares all of them, up to kSortPiece in one
// block, more in two launches, counts and rows (524288 slots of 8 bytes, 384 experts:
// 3.2 + 13.2 us; one block for all of them took 880).  Pieces of 2048 slots there: 22
// us for the rows, since every block adds up the counts of twice as many.
#include <algorithm>
#include <type_traits>

#include "device_common.hpp"

namespace muon {

namespace {

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
// Words of 16-bit counts, two experts each.
constexpr int kPairs = kMoeMaxExperts / 2;
constexpr int kSumBatch = 16;  // loads of a thread in flight while it adds up the blocks' counts

template <typename I>
__device__ __forceinline__ int expert_of(const I* ids, int64_t s, int64_t n, int experts) {
  if (s >= n) return -1;
  const int64_t v = static_cast<int64_t>(ids[s]);
  return v >= 0 && v < experts ? static_cast<int>(v) : -1;
}

// The lanes of the wave that hold the same id as this one (of `bits` bits; those
// without one have id -1 and match each other).
__device__ __forceinline__ uint64_t same_id(int id, int bits) {
  uint64_t m = __ballot(id >= 0);
  if (id < 0) m = ~m;
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot((id >> b) & 1);
    m &= (id >> b) & 1 ? set : ~set;
  }
  return m;
}

// Sum of v over the threads before this one; *total: over all of them.
__device__ __forceinline__ int block_before(int v, int* scratch /* kSortWaves */, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int inc = v;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(inc, off, 64);
    if (lane >= off) inc += o;
  }
  __syncthreads();  // scratch may still be read from the last call
  if (lane == 63) scratch[wave] = inc;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    const int t = scratch[w];
    before += w < wave ? t : 0;
    all += t;
  }
  *total = all;
  return before + inc - v;
}

}  // namespace

namespace {

// This thread's slots of a piece, from s0 on: each wave holds 64 * STEPS slots in a
// row, 64 at a time.
template <typename I, int STEPS>
__device__ __forceinline__ void load_ids(const MoeSortArgs& a, int64_t s0, int (&e)[STEPS]) {
  const I* const ids = static_cast<const I*>(a.ids);
#pragma unroll
  for (int u = 0; u < STEPS; ++u) e[u] = expert_of(ids, s0 + u * 64, a.n, a.experts);
}

// Adds one to expert e's 16 bits.
__device__ __forceinline__ void count_one(uint32_t* counts, int e) {
  if (e >= 0) atomicAdd(&counts[e >> 1], 1u << (16 * (e & 1)));
}

}  // namespace

// How many slots of each expert a block of the sort will find, two 16-bit counts a
// word.  Only for lists of more than one block.
template <typename I, int STEPS>
__global__ __launch_bounds__(kSortThreads) void k_moe_count(MoeSortArgs a) {
  constexpr int kPiece = STEPS * kSortThreads;
  __shared__ uint32_t counts[kPairs];
  const int me = threadIdx.x, pairs = (a.experts + 1) / 2;
  if (me < pairs) counts[me] = 0;
  __syncthreads();
  const int64_t from = static_cast<int64_t>(blockIdx.x) * a.span;
  for (int64_t at = from; at < from + a.span && at < a.n; at += kPiece) {
    int e[STEPS];
    load_ids<I>(a, at + (me >> 6) * (64 * STEPS) + (me & 63), e);
#pragma unroll
    for (int u = 0; u < STEPS; ++u) count_one(counts, e[u]);
  }
  __syncthreads();
  if (me < pairs) a.counts[blockIdx.x * pairs + me] = counts[me];
}

// The rows of the slots.  A block takes `span` slots in pieces of 1024 * STEPS.  The
// waves' counts of each expert in a piece become where their rows begin, and each
// wave walks its slots 64 at a time: a slot's row is its expert's next one plus
// the lanes before it with that id.  Where the block's rows begin follows from all
// blocks' counts, which every block adds up for itself (128 blocks, 384 experts:
// 98 KB from the L2).
template <typename I, int STEPS>
__global__ __launch_bounds__(kSortThreads) void k_moe_sort(MoeSortArgs a) {
  constexpr int kPiece = STEPS * kSortThreads;
  __shared__ int32_t base[kMoeMaxExperts];     // the first row of the piece for each expert
  __shared__ int32_t totals[kMoeMaxExperts];   // slots of each expert in all blocks
  __shared__ uint32_t next[kSortWaves * kPairs];  // each wave's next row after that
  __shared__ int scratch[kSortWaves];
  static_assert(kMoeMaxExperts <= kSortThreads && kPiece < (1 << 16));
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int me = threadIdx.x;  // the expert that a thread counts for
  const int pairs = (a.experts + 1) / 2;
  const int bits = 32 - __builtin_clz((a.experts - 1) | 1);
  const int64_t from = static_cast<int64_t>(blockIdx.x) * a.span;
  const int64_t to = min(a.n, from + a.span);
  const bool single = gridDim.x == 1 && to - from <= kPiece;
  uint32_t* const row = next + wave * pairs;
  volatile uint16_t* const mine = reinterpret_cast<volatile uint16_t*>(row);

  int e[STEPS];
  load_ids<I>(a, from + wave * (64 * STEPS) + lane, e);
  for (int i = me; i < kSortWaves * pairs; i += kSortThreads) next[i] = 0;
  base[me] = 0;
  totals[me] = 0;
  __syncthreads();
  if (!single) {
    // threads share a pair of experts: `groups` of them, each for every groups-th block
    const int groups = kSortThreads / pairs, g = me / pairs, p = me - g * pairs;
    if (g < groups) {
      int before[2] = {0, 0}, all[2] = {0, 0};
      const int blocks = static_cast<int>(gridDim.x), here = static_cast<int>(blockIdx.x);
      for (int b0 = g; b0 < blocks; b0 += kSumBatch * groups) {
        uint32_t c[kSumBatch];  // all requested before the first is added
#pragma unroll
        for (int u = 0; u < kSumBatch; ++u) {
          const int b = b0 + u * groups;
          c[u] = b < blocks ? a.counts[b * pairs + p] : 0u;
        }
#pragma unroll
        for (int u = 0; u < kSumBatch; ++u) {
          const int lo = c[u] & 0xffffu, hi = c[u] >> 16;
          const bool earlier = b0 + u * groups < here;
          all[0] += lo;
          all[1] += hi;
          before[0] += earlier ? lo : 0;
          before[1] += earlier ? hi : 0;
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        atomicAdd(&totals[2 * p + h], all[h]);
        atomicAdd(&base[2 * p + h], before[h]);
      }
    }
  }
  int64_t piece = from;
  do {
#pragma unroll
    for (int u = 0; u < STEPS; ++u) count_one(row, e[u]);
    __syncthreads();
    if (me < pairs) {
      uint32_t sum = 0;
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        const uint32_t t = next[w * pairs + me];
        next[w * pairs + me] = sum;
        sum += t;
      }
      if (single) {
        totals[2 * me] = sum & 0xffffu;
        totals[2 * me + 1] = sum >> 16;
      }
    }
    __syncthreads();
    if (piece == from) {
      const int count = totals[me];
      int kept, some;
      const int first = block_before(count, scratch, &kept);
      const int at = block_before(count > 0 ? 1 : 0, scratch, &some);
      base[me] += first;
      if (blockIdx.x == 0 && me < a.experts) {
        a.offsets[me] = first;
        if (count > 0) a.active[1 + at] = me;
        if (me >= some) a.active[1 + me] = -1;
        if (me == 0) {
          a.offsets[a.experts] = kept;
          a.active[0] = some;
        }
      }
      for (int64_t p = max(static_cast<int64_t>(kept), from) + me; p < to; p += kSortThreads)
        a.slots[p] = -1;
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
      const int64_t s = piece + wave * (64 * STEPS) + u * 64 + lane;
      const uint64_t same = same_id(e[u], bits);
      const int rank = __popcll(same & ((1ull << lane) - 1));
      int to_row = -1, begun = 0;
      if (e[u] >= 0) {
        begun = mine[e[u]];
        to_row = base[e[u]] + begun + rank;
      }
      __builtin_amdgcn_wave_barrier();  // every lane has read before the first writes
      if (e[u] >= 0 && rank == 0) mine[e[u]] = static_cast<uint16_t>(begun + __popcll(same));
      __builtin_amdgcn_wave_barrier();
      if (s < to) {
        a.rows[s] = to_row;
        if (to_row >= 0) a.slots[to_row] = static_cast<int32_t>(s);
      }
    }
    piece += kPiece;
    if (piece >= to) break;
    load_ids<I>(a, piece + wave * (64 * STEPS) + lane, e);
    __syncthreads();
    // the last wave's next rows are past all of the piece's
    const uint32_t last = next[(kSortWaves - 1) * pairs + (me >> 1)];
    if (me < a.experts) base[me] += (me & 1 ? last >> 16 : last) & 0xffffu;
    __syncthreads();
    for (int i = me; i < kSortWaves * pairs; i += kSortThreads) next[i] = 0;
    __syncthreads();
  } while (true);
}

namespace {

// A piece of V bytes of a row: 16, whose address is a multiple of A, or one element.
typedef u32x4_t u32x4_at4_t __attribute__((aligned(4)));
typedef u32x4_t u32x4_at2_t __attribute__((aligned(2)));
template <int V, int A> struct Piece { typedef u32x4_t type; };
template <> struct Piece<16, 4> { typedef u32x4_at4_t type; };
template <> struct Piece<16, 2> { typedef u32x4_at2_t type; };
template <int A> struct Piece<4, A> { typedef uint32_t type; };
template <int A> struct Piece<2, A> { typedef uint16_t type; };

template <int V, int A, bool NT>
__device__ __forceinline__ typename Piece<V, 16>::type ld(const void* p) {
  const GLOBAL_AS typename Piece<V, A>::type* q = (const GLOBAL_AS typename Piece<V, A>::type*)(p);
  return NT ? __builtin_nontemporal_load(q) : *q;
}
template <int V, int A, bool NT>
__device__ __forceinline__ void st(void* p, const typename Piece<V, 16>::type& v) {
  GLOBAL_AS typename Piece<V, A>::type* q = (GLOBAL_AS typename Piece<V, A>::type*)(p);
  if constexpr (NT)
    __builtin_nontemporal_store(v, q);
  else
    *q = v;
}

// The values of a piece, V / sizeof(T) of them.
template <typename T, int V>
__device__ __forceinline__ void unpack(const typename Piece<V, 16>::type& p, float* v) {
  if constexpr (V == 16)
    vec_to_f32<T>(p, v);
  else
    v[0] = Elt<T>::to_f32(__builtin_bit_cast(T, p));
}
template <typename T, int V>
__device__ __forceinline__ typename Piece<V, 16>::type pack(const float* v) {
  if constexpr (V == 16)
    return f32_to_vec<T>(v);
  else
    return __builtin_bit_cast(typename Piece<V, 16>::type, Elt<T>::from_f32(v[0]));
}

constexpr int kBatch = 8;  // slots whose rows are asked for together

// The sorted rows of slots k .. k + kBatch - 1 of a token, -1 for those that are
// dropped or past the last slot.
struct Batch {
  int32_t row[kBatch];
  __device__ __forceinline__ Batch(const int32_t* rows, int k, int top_k, int64_t sorted_rows) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      row[j] = load_const(rows + min(k + j, top_k - 1));
      if (k + j >= top_k || row[j] >= sorted_rows) row[j] = -1;
    }
  }
};

// The lanes that share a token's row: the block (W = 4 waves), a wave (1) or 16 (0).
template <int W>
constexpr int kLanes = W == 0 ? 16 : 64 * W;
// This lane's token, or -1.
template <int W>
__device__ __forceinline__ int64_t token_of(const MoeRowArgs& a) {
  int part = threadIdx.x / kLanes<W>;
  if (W > 0) part = __builtin_amdgcn_readfirstlane(part);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / kLanes<W>) + part;
  return t < a.tokens_n ? t : -1;
}
template <int W>
__device__ __forceinline__ int lane_of() {
  return threadIdx.x % kLanes<W>;
}

// Calls body(offset, V) for this lane's pieces of a row: 16 bytes each, at addresses
// that are multiples of A, then (A < 16) the last elements, one a lane.
template <int A, int W, typename F>
__device__ __forceinline__ void for_pieces(int64_t row_bytes, F body) {
  for (int64_t i = lane_of<W>() * 16; i + 16 <= row_bytes; i += kLanes<W> * 16)
    body(i, std::integral_constant<int, 16>());
  if constexpr (A < 16) {
    const int64_t i = row_bytes / 16 * 16 + lane_of<W>() * A;
    if (i < row_bytes) body(i, std::integral_constant<int, A>());
  }
}

}  // namespace

// Each piece of the token's row is read once and stored top_k times.
template <int A, int W, bool NT>
__global__ __launch_bounds__(kThreads) void k_moe_dispatch(MoeRowArgs a) {
  const int64_t t = token_of<W>(a);
  if (t < 0) return;
  const char* const x = static_cast<const char*>(a.tokens) + t * a.row_bytes;
  const int32_t* const rows = a.rows + t * a.top_k;
  for_pieces<A, W>(a.row_bytes, [&](int64_t i, auto v) {
    constexpr int V = v();
    const auto p = ld<V, A, false>(x + i);
    for (int k = 0; k < a.top_k; k += kBatch) {
      const Batch b(rows, k, a.top_k, a.sorted_rows);
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (b.row[j] >= 0) st<V, A, NT>(static_cast<char*>(a.out) + b.row[j] * a.row_bytes + i, p);
    }
  });
}

template <typename T, int A, int W, bool NT>
__global__ __launch_bounds__(kThreads) void k_moe_combine(MoeRowArgs a) {
  const int64_t t = token_of<W>(a);
  if (t < 0) return;
  const int32_t* const rows = a.rows + t * a.top_k;
  for_pieces<A, W>(a.row_bytes, [&](int64_t i, auto size) {
    constexpr int V = size();
    constexpr int kN = V / sizeof(T);
    float acc[kN] = {};
    for (int k = 0; k < a.top_k; k += kBatch) {
      const Batch b(rows, k, a.top_k, a.sorted_rows);
      typename Piece<V, 16>::type v[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (b.row[j] >= 0)
          v[j] = ld<V, A, NT>(static_cast<const char*>(a.sorted) + b.row[j] * a.row_bytes + i);
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (b.row[j] < 0) continue;
        float y[kN];
        unpack<T, V>(v[j], y);
        const float f = a.weights != nullptr ? load_const(a.weights + t * a.top_k + k + j) : 1.f;
#pragma unroll
        for (int c = 0; c < kN; ++c) acc[c] = __builtin_fmaf(f, y[c], acc[c]);
      }
    }
    st<V, A, false>(static_cast<char*>(a.out) + t * a.row_bytes + i, pack<T, V>(acc));
  });
}

// The products of a token's row with its experts' rows are summed by lanes, then
// over the token's lanes of the wave, then (W = 4) over the waves.
template <typename T, int A, int W, bool NT>
__global__ __launch_bounds__(kThreads) void k_moe_backward(MoeRowArgs a) {
  __shared__ float part[kMoeMaxTopK][kThreads / 64];
  const int64_t t = token_of<W>(a);
  if (t < 0) return;  // all lanes of a token; with W = 4 none
  const int32_t* const rows = a.rows + t * a.top_k;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int k = 0; k < a.top_k; k += kBatch) {
    const Batch b(rows, k, a.top_k, a.sorted_rows);
    float dot[kBatch] = {}, f[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      f[j] = b.row[j] >= 0 ? load_const(a.weights + t * a.top_k + k + j) : 0.f;
    for_pieces<A, W>(a.row_bytes, [&](int64_t i, auto size) {
      constexpr int V = size();
      constexpr int kN = V / sizeof(T);
      const auto dv = ld<V, A, false>(static_cast<const char*>(a.tokens) + t * a.row_bytes + i);
      typename Piece<V, 16>::type v[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (b.row[j] >= 0)
          v[j] = ld<V, A, NT>(static_cast<const char*>(a.sorted) + b.row[j] * a.row_bytes + i);
      float d[kN];
      unpack<T, V>(dv, d);
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (b.row[j] < 0) continue;
        float y[kN], o[kN];
        unpack<T, V>(v[j], y);
#pragma unroll
        for (int c = 0; c < kN; ++c) {
          dot[j] = __builtin_fmaf(d[c], y[c], dot[j]);
          o[c] = f[j] * d[c];
        }
        st<V, A, NT>(static_cast<char*>(a.out) + b.row[j] * a.row_bytes + i, pack<T, V>(o));
      }
    });
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (k + j >= a.top_k) break;
      float sum = dot[j];
#pragma unroll
      for (int off = W == 0 ? 8 : 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
      if ((W == 0 ? lane & 15 : lane) == 0) {
        if constexpr (W < 4)
          a.dweights[t * a.top_k + k + j] = sum;
        else
          part[k + j][wave] = sum;
      }
    }
  }
  if constexpr (W == 4) {
    __syncthreads();
    const int k = threadIdx.x;
    if (k < a.top_k)
      a.dweights[t * a.top_k + k] = (part[k][0] + part[k][1]) + (part[k][2] + part[k][3]);
  }
}

// The plan of up to kSortFew slots, by comparing all of them with each other and
// with every expert: two barriers and no counts to clear and add up (8 slots of
// 384 experts 2.2 us; the kernel above 4.2).
constexpr int kFewThreads = 512;
template <typename I>
__global__ __launch_bounds__(kFewThreads) void k_moe_sort_few(MoeSortArgs a) {
  __shared__ __attribute__((aligned(16))) int id[kSortFew], once[kSortFew];
  const int me = threadIdx.x, n = static_cast<int>(a.n);
  const int fours = (n + 3) / 4;
  const int mine = expert_of(static_cast<const I*>(a.ids), me, n, a.experts);
  if (me < 4 * fours) id[me] = mine >= 0 ? mine : INT32_MAX;
  __syncthreads();
  const int4* const id4 = reinterpret_cast<const int4*>(id);
  const int4* const once4 = reinterpret_cast<const int4*>(once);
  if (me < 4 * fours) {
    int before = 0, kept = 0;
    bool first = mine >= 0;
    for (int j = 0; j < fours; ++j) {
      const int4 v = id4[j];
      const int w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const bool earlier = w[c] == mine && 4 * j + c < me;
        before += w[c] < mine || earlier ? 1 : 0;
        first = first && !earlier;
        kept += w[c] != INT32_MAX ? 1 : 0;
      }
    }
    once[me] = first ? mine : INT32_MAX;
    if (me < n) {
      a.rows[me] = mine >= 0 ? before : -1;
      if (mine >= 0) a.slots[before] = me;
      if (me >= kept) a.slots[me] = -1;
    }
  }
  __syncthreads();
  for (int e = me; e <= a.experts; e += kFewThreads) {
    int before = 0, at = 0, some = 0;
    bool has = false;
    for (int j = 0; j < fours; ++j) {
      const int4 v = id4[j], o = once4[j];
      const int w[4] = {v.x, v.y, v.z, v.w}, f[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        before += w[c] < e ? 1 : 0;
        at += f[c] < e ? 1 : 0;
        has = has || f[c] == e;
        some += f[c] != INT32_MAX ? 1 : 0;
      }
    }
    a.offsets[e] = before;
    if (e == a.experts) {
      a.active[0] = some;
    } else {
      if (has) a.active[1 + at] = e;
      if (e >= some) a.active[1 + e] = -1;
    }
  }
}

namespace {

// The most blocks of a sort: each adds up the counts of all.
constexpr int64_t kSortBlocks = 320;
// Pieces of 1024 slots up to kSortShort of them, so that more blocks share the
// work, but of 4096 where those need one launch instead of two, and beyond (384
// experts: 1024 slots 5.1 us in pieces of 1024, 7.1 of 4096; 4096 slots 8.8 and 8.1;
// 32768 slots 9.5 and 12.4; 131072 slots 12.7 either way).
constexpr int64_t kSortShort = 65536;

int64_t sort_piece(int64_t n) {
  return n <= kSortThreads || (n > kSortPiece && n <= kSortShort) ? kSortThreads : kSortPiece;
}
int64_t sort_span(int64_t n) {
  const int64_t pieces = (n + sort_piece(n) - 1) / sort_piece(n);
  return (pieces + kSortBlocks - 1) / kSortBlocks * sort_piece(n);
}
int64_t sort_blocks(int64_t n) { return n > 0 ? (n + sort_span(n) - 1) / sort_span(n) : 1; }
static_assert((kMoeMaxSlots / kSortPiece + kSortBlocks) / kSortBlocks * kSortPiece < (1 << 16),
              "16-bit counts of a block");

template <typename I, int STEPS>
hipError_t run_blocks(const MoeSortArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(sort_blocks(a.n)));
  if (grid.x > 1) {
    hipLaunchKernelGGL((k_moe_count<I, STEPS>), grid, dim3(kSortThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((k_moe_sort<I, STEPS>), grid, dim3(kSortThreads), 0, s, a);
  return hipGetLastError();
}

template <typename I>
hipError_t run_sort(const MoeSortArgs& a, hipStream_t s) {
  // 384 experts: 8 slots 2.2 us, by pieces 4.2; 32 slots 4.1 and 4.2; 64 slots 6.6 and 4.3;
  // 16 slots of 512 experts 3.4 and 4.4, 10 of 1024 3.4 and 4.8
  if (a.n * ((a.experts + kFewThreads) / kFewThreads) <= kSortFew) {
    hipLaunchKernelGGL(k_moe_sort_few<I>, dim3(1), dim3(kFewThreads), 0, s, a);
    return hipGetLastError();
  }
  return sort_piece(a.n) == kSortThreads
             ? run_blocks<I, 1>(a, s)
             : run_blocks<I, static_cast<int>(kSortPiece / kSortThreads)>(a, s);
}

}  // namespace

// The most blocks of any list of up to n slots: those of n slots themselves can be
// fewer, where pieces or spans get longer (65536 slots take 64 blocks, 65537 take
// 17), and one workspace is to serve shorter lists too.
size_t moe_sort_workspace(int64_t n, int32_t experts) {
  if (n <= kSortPiece) return 0;  // one block
  const int64_t shorter = (std::min(n, kSortShort) + kSortThreads - 1) / kSortThreads;
  const int64_t longer = std::min((n + kSortPiece - 1) / kSortPiece, kSortBlocks);
  return static_cast<size_t>(std::max(shorter, longer)) * ((experts + 1) / 2) * 4;
}

hipError_t launch_moe_sort(MoeSortArgs a, int32_t id_bytes, hipStream_t s) {
  a.span = a.n > 0 ? sort_span(a.n) : kSortThreads;
  return id_bytes == 8 ? run_sort<int64_t>(a, s) : run_sort<int32_t>(a, s);
}

namespace {

// Bytes of sorted rows from which they pass the caches by.  A call by itself is
// faster that way from 16 MB on (tokens x 8 x 6144 bf16, dispatch, combine and
// gradient: 128 MB 27, 29 and 58 us, without the hint 34, 31 and 62; 384 MB 79, 82 and
// 162, without 92, 93 and 175), but a call that follows then finds no rows in the
// caches (dispatch and a copy of its rows: 64 MB 41.6 us, without the hint 39.0; 128 MB
// 80.5 and 78.6; 256 MB 163 and 176; combine after a copy into its rows: 128 MB 73 and 77; 256 MB
// 153 and 155).
constexpr int64_t kNtRowBytes = 256ll << 20;
// Rows that are no whole pieces of 16 bytes share lines with their neighbours, which
// the hint then moves twice: only rows of this many bytes take it (300 MB of rows,
// four a token, dispatch, combine and gradient: 200 bytes 269, 172 and 389 us, without the
// hint 161, 141 and 243; 1000 bytes 114, 97 and 182, without 102, 96 and 175; 2004 bytes 107, 87 and
// 177, without 105, 89 and 181; 4004 bytes 105, 87 and 173, without 108, 90 and 187).
constexpr int64_t kNtOddRowBytes = 2000;
// Rows of fewer bytes than this are one wave's, of more the block's; with few
// tokens, whose waves do not fill the chip, already shorter ones are the block's
// (combine, 1000 tokens x 2 x 1001 fp32: 5.2 us by blocks, 6.6 by waves; 16384 x 4 x 1024 bf16
// 25.4 and 25.0, x 2048 63 and 80).
constexpr int64_t kBlockRowBytes = 4096, kBlockRowBytesFew = 1024, kFewTokens = 4096;
// Rows of up to this many bytes are 16 lanes' (65536 tokens x 8 bf16, dispatch, combine
// and gradient: 64 columns 13, 18 and 27 us, by waves 24, 38 and 60; 128 columns 24, 27 and
// 51, by waves 25, 39 and 76; 160 columns 32, 44 and 83, by waves 31, 41 and 87; 200 columns 47, 54
// and 137, by waves 40, 47 and 119).  With one or two choices a token the waves would
// win later only: 256 columns 12, 14 and 20 us by 16 lanes, 20, 23 and 39 by waves, which
// have one row to ask for.
constexpr int64_t kShortRowBytes = 256;

// Calls `launch` with a token's waves and the hint as constants; A: the rows'
// alignment.
template <int A, typename F>
hipError_t with_shape(const MoeRowArgs& a, F launch) {
  const bool wide = a.row_bytes >= (a.tokens_n < kFewTokens ? kBlockRowBytesFew : kBlockRowBytes);
  const bool narrow = a.row_bytes <= kShortRowBytes;
  using std::integral_constant;
  typedef integral_constant<int, 0> Part;
  typedef integral_constant<int, 1> One;
  typedef integral_constant<int, 4> Four;
  const int64_t per = wide ? 1 : kThreads / (narrow ? kLanes<0> : kLanes<1>);
  const dim3 grid(static_cast<uint32_t>((a.tokens_n + per - 1) / per));
  const bool nt = a.tokens_n * a.top_k * a.row_bytes > kNtRowBytes &&
                  (A == 16 || a.row_bytes >= kNtOddRowBytes);
  const auto with_hint = [&](auto w) {
    if constexpr (A == 16 || w() != 0)  // kNtOddRowBytes is past 16 lanes' rows
      if (nt) return launch(w, std::true_type(), grid);
    launch(w, std::false_type(), grid);
  };
  if (wide)
    with_hint(Four());
  else if (narrow)
    with_hint(Part());
  else
    with_hint(One());
  return hipGetLastError();
}

// Calls `launch` with the alignment of the rows as a constant: 16, or an element's.
template <typename T, typename F>
hipError_t with_rows(const MoeRowArgs& a, F launch) {
  if (a.row_bytes % 16 == 0) return launch(std::integral_constant<int, 16>());
  return launch(std::integral_constant<int, sizeof(T)>());
}

template <typename T>
hipError_t run_dispatch(const MoeRowArgs& a, hipStream_t s) {
  return with_rows<T>(a, [&](auto align) {
    return with_shape<align()>(a, [&](auto w, auto nt, dim3 grid) {
      hipLaunchKernelGGL((k_moe_dispatch<align(), w(), nt()>), grid, dim3(kThreads), 0, s, a);
    });
  });
}

template <typename T>
hipError_t run_combine(const MoeRowArgs& a, hipStream_t s) {
  return with_rows<T>(a, [&](auto align) {
    return with_shape<align()>(a, [&](auto w, auto nt, dim3 grid) {
      hipLaunchKernelGGL((k_moe_combine<T, align(), w(), nt()>), grid, dim3(kThreads), 0, s, a);
    });
  });
}

template <typename T>
hipError_t run_backward(const MoeRowArgs& a, hipStream_t s) {
  return with_rows<T>(a, [&](auto align) {
    return with_shape<align()>(a, [&](auto w, auto nt, dim3 grid) {
      hipLaunchKernelGGL((k_moe_backward<T, align(), w(), nt()>), grid, dim3(kThreads), 0, s, a);
    });
  });
}

}  // namespace

hipError_t launch_moe_dispatch(const MoeRowArgs& a, bool is_bf16, hipStream_t s) {
  return is_bf16 ? run_dispatch<uint16_t>(a, s) : run_dispatch<float>(a, s);
}
hipError_t launch_moe_combine(const MoeRowArgs& a, bool is_bf16, hipStream_t s) {
  return is_bf16 ? run_combine<uint16_t>(a, s) : run_combine<float>(a, s);
}
hipError_t launch_moe_backward(const MoeRowArgs& a, bool is_bf16, hipStream_t s) {
  return is_bf16 ? run_backward<uint16_t>(a, s) : run_backward<float>(a, s);
}

}  // namespace muon
