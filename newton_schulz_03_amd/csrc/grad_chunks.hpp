// What the kernels over a ragged batch of flat tensors share (gradient norm and
// scale, dropout): four elements at a time, and the tensor that a chunk belongs to.
#pragma once

#include "device_common.hpp"

namespace muon {

// Four elements: 16 bytes of fp32, 8 of bf16.
template <typename T, bool NT>
__device__ __forceinline__ void load4(const T* p, float* v) {
  if constexpr (sizeof(T) == 2) {
    const GLOBAL_AS u32x2_t* q = (const GLOBAL_AS u32x2_t*)(p);
    const u32x2_t w = NT ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    vec_to_f32<T>(NT ? ld16_nt(p) : ld16(p), v);
  }
}
template <typename T, bool NT>
__device__ __forceinline__ void store4(T* p, const float* v) {
  if constexpr (sizeof(T) == 2) {
    u32x2_t w;
    w[0] = Elt<uint16_t>::pack2(v[0], v[1]);
    w[1] = Elt<uint16_t>::pack2(v[2], v[3]);
    GLOBAL_AS u32x2_t* q = (GLOBAL_AS u32x2_t*)(p);
    if constexpr (NT)
      __builtin_nontemporal_store(w, q);
    else
      *q = w;
  } else if constexpr (NT) {
    st16_nt(p, f32_to_vec<T>(v));
  } else {
    st16(p, f32_to_vec<T>(v));
  }
}

// One chunk (kGradSpan elements) of a tensor, or what is left of it.
struct Chunk {
  const void* g;
  void* out;
  int64_t base;  // first element
  int32_t tensor;
  int64_t n;     // elements, 1 .. kGradSpan
  bool in_bf16, out_bf16;
};

// Chunk c's tensor by binary search in the call's table.
__device__ __forceinline__ Chunk find_chunk(const GradCtx& ctx, int32_t c) {
  const char* const table = table_base(ctx.table);
  const GradDesc* const desc = reinterpret_cast<const GradDesc*>(table);
  int lo = 0, hi = ctx.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (load_const(&desc[mid].chunk) <= c)
      lo = mid;
    else
      hi = mid;
  }
  const GradDesc d = load_const(desc + lo);
  Chunk k;
  k.g = d.g;
  k.tensor = lo;
  k.out = const_cast<void*>(d.g);
  if (ctx.out_off > 0) {
    typedef void* ptr_t;
    k.out = load_const(reinterpret_cast<const ptr_t*>(table + ctx.out_off) + lo);
  }
  k.base = static_cast<int64_t>(c - d.chunk) * kGradSpan;
  const bool last = c + 1 == load_const(&desc[lo + 1].chunk);
  k.n = last ? kGradSpan - (d.tail & (kGradSpan - 1)) : kGradSpan;
  k.in_bf16 = (d.tail & kGradInBf16) != 0;
  k.out_bf16 = (d.tail & kGradOutBf16) != 0;
  return k;
}

}  // namespace muon
