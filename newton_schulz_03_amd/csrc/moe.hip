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
#include "device_common.hpp"

namespace muon {

namespace {

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;

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

// The rows of the slots.  A block takes its slots in pieces of kSortPiece, each
// wave kSortPiece / 16 of them in a row: the waves' counts of each expert become
// where their rows begin, and each wave then walks its slots 64 at a time, a
// slot's row being its expert's next one plus the lanes before it with that id.
template <typename I>
__global__ __launch_bounds__(kSortThreads) void k_moe_sort(MoeSortArgs a) {
  constexpr int kSteps = kSortPiece / kSortThreads;
  constexpr int kPairs = kMoeMaxExperts / 2;
  __shared__ int32_t base[kMoeMaxExperts];  // the first row of the piece for each expert
  __shared__ uint32_t next[kSortWaves][kPairs];  // each wave's next row after that, 16 bits each
  __shared__ int scratch[kSortWaves];
  static_assert(kMoeMaxExperts <= kSortThreads && kSortPiece < (1 << 16));
  const I* const ids = static_cast<const I*>(a.ids);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int me = threadIdx.x;  // the expert that a thread counts for
  const int pairs = (a.experts + 1) / 2;
  int bits = 0;
  while ((1 << bits) < a.experts) ++bits;

  if (me < a.experts) base[me] = 0;
  __syncthreads();
  for (int64_t s = threadIdx.x; s < a.n; s += kSortThreads) {
    const int e = expert_of(ids, s, a.n, a.experts);
    if (e >= 0) atomicAdd(&base[e], 1);
  }
  __syncthreads();
  const int count = me < a.experts ? base[me] : 0;
  int kept, some;
  const int first = block_before(count, scratch, &kept);
  const int at = block_before(count > 0 ? 1 : 0, scratch, &some);
  if (me < a.experts) {
    base[me] = first;
    a.offsets[me] = first;
    if (count > 0) a.active[1 + at] = me;
    if (me >= some) a.active[1 + me] = -1;
  }
  if (me == 0) {
    a.offsets[a.experts] = kept;
    a.active[0] = some;
  }
  for (int64_t p = kept + threadIdx.x; p < a.n; p += kSortThreads) a.slots[p] = -1;

  volatile uint16_t* const mine = reinterpret_cast<volatile uint16_t*>(next[wave]);
  for (int64_t from = 0; from < a.n; from += kSortPiece) {
    for (int i = me; i < kSortWaves * pairs; i += kSortThreads) next[i / pairs][i % pairs] = 0;
    __syncthreads();
    const int64_t s0 = from + wave * (64 * kSteps) + lane;
    for (int u = 0; u < kSteps; ++u) {
      const int e = expert_of(ids, s0 + u * 64, a.n, a.experts);
      if (e >= 0) atomicAdd(&next[wave][e / 2], 1u << (16 * (e & 1)));
    }
    __syncthreads();
    for (int i = me; i < pairs; i += kSortThreads) {
      uint32_t sum = 0;
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        const uint32_t t = next[w][i];
        next[w][i] = sum;
        sum += t;
      }
    }
    __syncthreads();
    for (int u = 0; u < kSteps; ++u) {
      const int64_t s = s0 + u * 64;
      const int e = expert_of(ids, s, a.n, a.experts);
      const uint64_t same = same_id(e, bits);
      const int rank = __popcll(same & ((1ull << lane) - 1));
      int row = -1, begun = 0;
      if (e >= 0) {
        begun = mine[e];
        row = base[e] + begun + rank;
      }
      __builtin_amdgcn_wave_barrier();  // every lane has read before the first writes
      if (e >= 0 && rank == 0) mine[e] = static_cast<uint16_t>(begun + __popcll(same));
      __builtin_amdgcn_wave_barrier();
      if (s < a.n) {
        a.rows[s] = row;
        if (row >= 0) a.slots[row] = static_cast<int32_t>(s);
      }
    }
    __syncthreads();
    // the last wave's next rows are past all of the piece's
    if (me < a.experts)
      base[me] += reinterpret_cast<volatile uint16_t*>(next[kSortWaves - 1])[me];
    __syncthreads();
  }
}

namespace {

// A row in pieces of V bytes, the widest that its length allows.
template <int V> struct Piece;
template <> struct Piece<16> { typedef u32x4_t type; };
template <> struct Piece<8> { typedef u32x2_t type; };
template <> struct Piece<4> { typedef uint32_t type; };
template <> struct Piece<2> { typedef uint16_t type; };

template <int V>
__device__ __forceinline__ typename Piece<V>::type ld(const void* p) {
  return *(const GLOBAL_AS typename Piece<V>::type*)(p);
}
template <int V>
__device__ __forceinline__ void st(void* p, const typename Piece<V>::type& v) {
  *(GLOBAL_AS typename Piece<V>::type*)(p) = v;
}

// The values of a piece, V / sizeof(T) of them.
template <typename T, int V>
__device__ __forceinline__ void unpack(const typename Piece<V>::type& p, float* v) {
  T x[V / sizeof(T)];
  __builtin_memcpy(x, &p, V);
#pragma unroll
  for (int i = 0; i < static_cast<int>(V / sizeof(T)); ++i) v[i] = Elt<T>::to_f32(x[i]);
}
template <typename T, int V>
__device__ __forceinline__ typename Piece<V>::type pack(const float* v) {
  T x[V / sizeof(T)];
#pragma unroll
  for (int i = 0; i < static_cast<int>(V / sizeof(T)); ++i) x[i] = Elt<T>::from_f32(v[i]);
  typename Piece<V>::type p;
  __builtin_memcpy(&p, x, V);
  return p;
}

__device__ __forceinline__ bool has_row(int row, int64_t rows) {
  return row >= 0 && row < rows;
}

}  // namespace

// A block takes one token.
template <int V>
__global__ __launch_bounds__(kThreads) void k_moe_dispatch(MoeRowArgs a) {
  const int64_t t = blockIdx.x;
  const char* const x = static_cast<const char*>(a.tokens) + t * a.row_bytes;
  const int32_t* const rows = a.rows + t * a.top_k;
  for (int64_t i = static_cast<int64_t>(threadIdx.x) * V; i < a.row_bytes; i += kThreads * V) {
    const typename Piece<V>::type v = ld<V>(x + i);
    for (int k = 0; k < a.top_k; ++k)
      if (has_row(rows[k], a.sorted_rows))
        st<V>(static_cast<char*>(a.out) + rows[k] * a.row_bytes + i, v);
  }
}

template <typename T, int V>
__global__ __launch_bounds__(kThreads) void k_moe_combine(MoeRowArgs a) {
  constexpr int kN = V / sizeof(T);
  const int64_t t = blockIdx.x;
  const int32_t* const rows = a.rows + t * a.top_k;
  const float* const w = a.weights + t * a.top_k;
  for (int64_t i = static_cast<int64_t>(threadIdx.x) * V; i < a.row_bytes; i += kThreads * V) {
    float acc[kN] = {};
    for (int k = 0; k < a.top_k; ++k) {
      if (!has_row(rows[k], a.sorted_rows)) continue;
      float y[kN];
      unpack<T, V>(ld<V>(static_cast<const char*>(a.sorted) + rows[k] * a.row_bytes + i), y);
      const float f = a.weights != nullptr ? w[k] : 1.f;
#pragma unroll
      for (int c = 0; c < kN; ++c) acc[c] = __builtin_fmaf(f, y[c], acc[c]);
    }
    st<V>(static_cast<char*>(a.out) + t * a.row_bytes + i, pack<T, V>(acc));
  }
}

template <typename T, int V>
__global__ __launch_bounds__(kThreads) void k_moe_backward(MoeRowArgs a) {
  constexpr int kN = V / sizeof(T);
  __shared__ float scratch[kThreads / 64];
  const int64_t t = blockIdx.x;
  const int32_t* const rows = a.rows + t * a.top_k;
  for (int k = 0; k < a.top_k; ++k) {
    float dot = 0.f;
    if (has_row(rows[k], a.sorted_rows)) {
      const float f = a.weights[t * a.top_k + k];
      const int64_t at = rows[k] * a.row_bytes;
      for (int64_t i = static_cast<int64_t>(threadIdx.x) * V; i < a.row_bytes; i += kThreads * V) {
        float d[kN], y[kN];
        unpack<T, V>(ld<V>(static_cast<const char*>(a.tokens) + t * a.row_bytes + i), d);
        unpack<T, V>(ld<V>(static_cast<const char*>(a.sorted) + at + i), y);
#pragma unroll
        for (int c = 0; c < kN; ++c) {
          dot = __builtin_fmaf(d[c], y[c], dot);
          d[c] *= f;
        }
        st<V>(static_cast<char*>(a.out) + at + i, pack<T, V>(d));
      }
    }
    dot = block_sum(dot, scratch);
    if (threadIdx.x == 0) a.dweights[t * a.top_k + k] = dot;
  }
}

namespace {

int piece_bytes(int64_t row_bytes) {
  return row_bytes % 16 == 0 ? 16 : row_bytes % 8 == 0 ? 8 : row_bytes % 4 == 0 ? 4 : 2;
}

}  // namespace

hipError_t launch_moe_sort(const MoeSortArgs& a, int32_t id_bytes, hipStream_t s) {
  if (id_bytes == 8)
    hipLaunchKernelGGL(k_moe_sort<int64_t>, dim3(1), dim3(kSortThreads), 0, s, a);
  else
    hipLaunchKernelGGL(k_moe_sort<int32_t>, dim3(1), dim3(kSortThreads), 0, s, a);
  return hipGetLastError();
}

#define MOE_LAUNCH(kernel) \
  hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(a.tokens_n)), dim3(kThreads), 0, s, a)

hipError_t launch_moe_dispatch(const MoeRowArgs& a, hipStream_t s) {
  switch (piece_bytes(a.row_bytes)) {
    case 16: MOE_LAUNCH(k_moe_dispatch<16>); break;
    case 8: MOE_LAUNCH(k_moe_dispatch<8>); break;
    case 4: MOE_LAUNCH(k_moe_dispatch<4>); break;
    default: MOE_LAUNCH(k_moe_dispatch<2>);
  }
  return hipGetLastError();
}

hipError_t launch_moe_combine(const MoeRowArgs& a, bool is_bf16, hipStream_t s) {
  const int v = piece_bytes(a.row_bytes);
  if (is_bf16) {
    switch (v) {
      case 16: MOE_LAUNCH((k_moe_combine<uint16_t, 16>)); break;
      case 8: MOE_LAUNCH((k_moe_combine<uint16_t, 8>)); break;
      case 4: MOE_LAUNCH((k_moe_combine<uint16_t, 4>)); break;
      default: MOE_LAUNCH((k_moe_combine<uint16_t, 2>));
    }
  } else {
    switch (v) {
      case 16: MOE_LAUNCH((k_moe_combine<float, 16>)); break;
      case 8: MOE_LAUNCH((k_moe_combine<float, 8>)); break;
      default: MOE_LAUNCH((k_moe_combine<float, 4>));
    }
  }
  return hipGetLastError();
}

hipError_t launch_moe_backward(const MoeRowArgs& a, bool is_bf16, hipStream_t s) {
  const int v = piece_bytes(a.row_bytes);
  if (is_bf16) {
    switch (v) {
      case 16: MOE_LAUNCH((k_moe_backward<uint16_t, 16>)); break;
      case 8: MOE_LAUNCH((k_moe_backward<uint16_t, 8>)); break;
      case 4: MOE_LAUNCH((k_moe_backward<uint16_t, 4>)); break;
      default: MOE_LAUNCH((k_moe_backward<uint16_t, 2>));
    }
  } else {
    switch (v) {
      case 16: MOE_LAUNCH((k_moe_backward<float, 16>)); break;
      case 8: MOE_LAUNCH((k_moe_backward<float, 8>)); break;
      default: MOE_LAUNCH((k_moe_backward<float, 4>));
    }
  }
  return hipGetLastError();
}

}  // namespace muon
