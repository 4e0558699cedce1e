// Host side of the calls over a ragged batch of flat tensors (gradient norm, scale
// and clip; dropout): their checks, chunks and descriptor tables.
#pragma once

#include <vector>

#include "abi_common.hpp"
#include "muon_internal.hpp"
#include "muon_mi355x.h"

namespace muon {

// The scale pass numbers four blocks per chunk.
constexpr int64_t kMaxChunks = INT32_MAX / 4;

struct GradPlan {
  std::vector<GradDesc> desc;  // batch + 1
  std::vector<void*> outs;     // of a call that does not work in place
  size_t partials_off = 0, total_bytes = 0;
  int32_t chunks = 0;
  int64_t in_bytes = 0, out_bytes = 0;
};

inline int32_t make_grad_plan(int32_t batch, const int64_t* numel, GradPlan& pl) {
  if (batch < 0) return fail(MUON_ERR_INVALID_ARG, "batch = %d is negative", batch);
  if (batch > 0 && numel == nullptr) return fail(MUON_ERR_INVALID_ARG, "numel array is null");
  pl.desc.assign(static_cast<size_t>(batch) + 1, GradDesc{});
  int64_t total = 0;
  for (int32_t i = 0; i < batch; ++i) {
    if (numel[i] < 0)
      return fail(MUON_ERR_INVALID_ARG, "tensor %d: numel %lld is negative", i,
                  static_cast<long long>(numel[i]));
    if (numel[i] / kGradSpan > kMaxChunks - total - 1)
      return fail(MUON_ERR_UNSUPPORTED, "batch needs more than 2^31 blocks");
    const int64_t n = (numel[i] + kGradSpan - 1) / kGradSpan;
    pl.desc[i].chunk = static_cast<int32_t>(total);
    pl.desc[i].tail = static_cast<uint32_t>(n * kGradSpan - numel[i]);
    total += n;
  }
  pl.desc[batch].chunk = static_cast<int32_t>(total);
  pl.chunks = static_cast<int32_t>(total);
  pl.partials_off = align_up(sizeof(GradDesc) * (static_cast<size_t>(batch) + 1), kAlign) +
                    align_up(sizeof(void*) * static_cast<size_t>(batch), kAlign);
  pl.total_bytes = pl.partials_off + align_up(8 * static_cast<size_t>(kNormBlocks), kAlign);
  return MUON_OK;
}

inline int32_t known_dtype(int32_t dtype, int32_t i) {
  if (dtype != MUON_BF16 && dtype != MUON_FP32)
    return fail(MUON_ERR_INVALID_ARG, "tensor %d: unknown dtype %d", i, dtype);
  return MUON_OK;
}

// out == nullptr: the norm, which writes nothing.
inline int32_t bind_grads(int32_t batch, const int64_t* numel, const void* const* g, const int32_t* dtype,
                   void* const* out, const int32_t* out_dtype, GradPlan& pl) {
  if (batch == 0) return MUON_OK;
  if (g == nullptr || dtype == nullptr) return fail(MUON_ERR_INVALID_ARG, "g/dtype array is null");
  if (out != nullptr && out_dtype == nullptr)
    return fail(MUON_ERR_INVALID_ARG, "out_dtype array is null");
  bool in_place = true;
  for (int32_t i = 0; i < batch; ++i) {
    GradDesc& d = pl.desc[i];
    int32_t st = known_dtype(dtype[i], i);
    if (st != MUON_OK) return st;
    const bool in_bf16 = dtype[i] == MUON_BF16;
    bool out_bf16 = in_bf16;
    const void* to = g[i];
    if (out != nullptr) {
      if ((st = known_dtype(out_dtype[i], i)) != MUON_OK) return st;
      out_bf16 = out_dtype[i] == MUON_BF16;
      to = out[i];
    }
    d.g = g[i];
    d.tail |= (in_bf16 ? kGradInBf16 : 0u) | (out_bf16 ? kGradOutBf16 : 0u);
    if (numel[i] == 0) continue;
    pl.in_bytes += numel[i] * (in_bf16 ? 2 : 4);
    pl.out_bytes += numel[i] * (out_bf16 ? 2 : 4);
    if (g[i] == nullptr || to == nullptr)
      return fail(MUON_ERR_INVALID_ARG, "tensor %d: null device pointer", i);
    if (!aligned16(g[i]) || !aligned16(to))
      return fail(MUON_ERR_INVALID_ARG, "tensor %d: device pointer not 16-byte aligned", i);
    if (to == g[i] && out_bf16 != in_bf16)
      return fail(MUON_ERR_INVALID_ARG, "tensor %d: in place needs one dtype", i);
    in_place = in_place && to == g[i];
  }
  if (!in_place) pl.outs.assign(out, out + batch);
  return MUON_OK;
}

inline int32_t grad_table(const GradPlan& pl, char* ws, hipStream_t s, ArgTable& t, GradCtx& c) {
  const size_t desc_bytes = sizeof(GradDesc) * pl.desc.size();
  c.batch = static_cast<int32_t>(pl.desc.size()) - 1;
  c.out_off = pl.outs.empty() ? 0 : static_cast<int32_t>(align_up(desc_bytes, kAlign));
  c.stream = s;
  return place_table(pl.desc.data(), desc_bytes, pl.outs.data(), sizeof(void*) * pl.outs.size(), ws,
                     s, t, &c.table);
}

}  // namespace muon
