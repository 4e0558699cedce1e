// C ABI of the operators of an expert layer: tokens sorted by expert and back, and
// the products of few rows with 4-bit weights.  Kernel launches only, so that a
// call can be captured into a graph.
#include <vector>

#include "abi_common.hpp"
#include "muon_internal.hpp"
#include "muon_mi355x.h"

namespace muon {
namespace {

static_assert(MUON_MOE_MAX_EXPERTS == kMoeMaxExperts && MUON_MOE_MAX_TOP_K == kMoeMaxTopK &&
              MUON_MOE_MAX_SLOTS == kMoeMaxSlots && MUON_F4_GROUP == kF4Group);
constexpr int64_t kMaxTiles = 1ll << 28;  // of an operand of 4-bit weights

int64_t cdiv(int64_t x, int64_t a) { return (x + a - 1) / a; }

int32_t check_slots(int64_t tokens, int32_t top_k) {
  if (tokens < 0)
    return fail(MUON_ERR_INVALID_ARG, "tokens = %lld is negative", static_cast<long long>(tokens));
  if (top_k < 1) return fail(MUON_ERR_INVALID_ARG, "top_k = %d: must be >= 1", top_k);
  if (top_k > kMoeMaxTopK)
    return fail(MUON_ERR_UNSUPPORTED, "top_k = %d; the maximum is %d", top_k, kMoeMaxTopK);
  if (tokens > kMoeMaxSlots / top_k)
    return fail(MUON_ERR_UNSUPPORTED, "%lld tokens x %d slots; the maximum is %d slots",
                static_cast<long long>(tokens), top_k, MUON_MOE_MAX_SLOTS);
  return MUON_OK;
}

int32_t check_experts(int32_t experts, const char* what) {
  if (experts < 1) return fail(MUON_ERR_INVALID_ARG, "%s = %d: must be >= 1", what, experts);
  if (experts > kMoeMaxExperts)
    return fail(MUON_ERR_UNSUPPORTED, "%s = %d; the maximum is %d", what, experts, kMoeMaxExperts);
  return MUON_OK;
}

int32_t check_size(int64_t v, int64_t most, const char* what) {
  if (v < 0)
    return fail(MUON_ERR_INVALID_ARG, "%s = %lld is negative", what, static_cast<long long>(v));
  if (v > most)
    return fail(MUON_ERR_UNSUPPORTED, "%s = %lld; the maximum is %lld", what,
                static_cast<long long>(v), static_cast<long long>(most));
  return MUON_OK;
}

// An array of `n` elements; not read, and may be null, when n is 0.
int32_t check_array(const void* p, int64_t n, uintptr_t align, const char* what) {
  if (n == 0) return MUON_OK;
  if (p == nullptr) return fail(MUON_ERR_INVALID_ARG, "%s pointer is null", what);
  if ((reinterpret_cast<uintptr_t>(p) & (align - 1)) != 0)
    return fail(MUON_ERR_INVALID_ARG, "%s pointer not %d-byte aligned", what,
                static_cast<int>(align));
  return MUON_OK;
}

int32_t check_dtype(int32_t dtype) {
  if (dtype != MUON_BF16 && dtype != MUON_FP32)
    return fail(MUON_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  return MUON_OK;
}

int32_t launched(TimedLaunch& tl, hipError_t e, const char* what) {
  if (e != hipSuccess) return hip_fail(e, what);
  tl.done();
  return MUON_OK;
}

// What dispatch, combine and its gradient check alike.
int32_t row_args(int64_t tokens, int32_t top_k, int64_t cols, int64_t sorted_rows,
                 const int32_t* rows, int32_t dtype, MoeRowArgs& a) {
  int32_t st = check_slots(tokens, top_k);
  if (st != MUON_OK) return st;
  if ((st = check_size(cols, MUON_F8_MAX_DIM, "cols")) != MUON_OK) return st;
  if ((st = check_size(sorted_rows, kMoeMaxSlots, "number of sorted rows")) != MUON_OK) return st;
  if ((st = check_dtype(dtype)) != MUON_OK) return st;
  if ((st = check_array(rows, tokens, 4, "rows")) != MUON_OK) return st;
  a = MoeRowArgs{};
  a.rows = rows;
  a.tokens_n = tokens;
  a.sorted_rows = sorted_rows;
  a.row_bytes = cols * (dtype == MUON_BF16 ? 2 : 4);
  a.top_k = top_k;
  return MUON_OK;
}

// An output may share no byte with what the call reads.
int32_t apart(const void* out, int64_t out_bytes, const void* in, int64_t in_bytes,
              const char* what) {
  const uintptr_t o = reinterpret_cast<uintptr_t>(out), i = reinterpret_cast<uintptr_t>(in);
  const bool some = out_bytes > 0 && in_bytes > 0;
  if (out != nullptr &&
      (o == i || (some && o < i + static_cast<uintptr_t>(in_bytes) &&
                  i < o + static_cast<uintptr_t>(out_bytes))))
    return fail(MUON_ERR_INVALID_ARG, "%s must be another buffer", what);
  return MUON_OK;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" size_t muon_moe_workspace_bytes(int64_t tokens, int32_t top_k, int32_t experts) {
  clear_detail();
  if (check_slots(tokens, top_k) != MUON_OK || check_experts(experts, "experts") != MUON_OK)
    return SIZE_MAX;
  return moe_sort_workspace(tokens * top_k, experts);
}

extern "C" int32_t muon_moe_sort(int64_t tokens, int32_t top_k, int32_t experts, const void* ids,
                                 int32_t id_bytes, int32_t* offsets, int32_t* active,
                                 int32_t* rows, int32_t* slots, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  try {
    clear_detail();
    int32_t st = check_slots(tokens, top_k);
    if (st != MUON_OK) return st;
    if ((st = check_experts(experts, "experts")) != MUON_OK) return st;
    if (id_bytes != 4 && id_bytes != 8)
      return fail(MUON_ERR_INVALID_ARG, "id_bytes = %d: must be 4 or 8", id_bytes);
    if ((st = check_array(ids, tokens, id_bytes, "ids")) != MUON_OK) return st;
    if ((st = check_array(offsets, 1, 4, "offsets")) != MUON_OK) return st;
    if ((st = check_array(active, 1, 4, "active")) != MUON_OK) return st;
    if ((st = check_array(rows, tokens, 4, "rows")) != MUON_OK) return st;
    if ((st = check_array(slots, tokens, 4, "slots")) != MUON_OK) return st;
    MoeSortArgs a{};
    a.ids = ids;
    a.offsets = offsets;
    a.active = active;
    a.rows = rows;
    a.slots = slots;
    a.counts = static_cast<uint32_t*>(workspace);
    a.n = tokens * top_k;
    a.experts = experts;
    const size_t need = moe_sort_workspace(a.n, experts);
    if (need > 0 && (st = check_workspace(workspace, workspace_bytes, need)) != MUON_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    TimedLaunch tl(MUON_K_MOE_SORT, s);
    return launched(tl, launch_moe_sort(a, id_bytes, s), "launch token sort");
  } catch (...) {
    return fail(MUON_ERR_HIP, "unexpected host exception");
  }
}

extern "C" int32_t muon_moe_dispatch(int64_t tokens, int32_t top_k, int64_t cols, const void* x,
                                     const int32_t* rows, int64_t out_rows, void* out,
                                     int32_t dtype, void* stream) {
  try {
    clear_detail();
    MoeRowArgs a;
    int32_t st = row_args(tokens, top_k, cols, out_rows, rows, dtype, a);
    if (st != MUON_OK) return st;
    if ((st = check_array(x, tokens * cols, 16, "x")) != MUON_OK) return st;
    if ((st = check_array(out, out_rows * cols, 16, "out")) != MUON_OK) return st;
    if ((st = apart(out, out_rows * a.row_bytes, x, tokens * a.row_bytes, "out")) != MUON_OK) return st;
    if (tokens == 0 || cols == 0 || out_rows == 0) return MUON_OK;
    a.tokens = x;
    a.out = out;
    hipStream_t s = static_cast<hipStream_t>(stream);
    TimedLaunch tl(MUON_K_MOE_DISPATCH, s);
    return launched(tl, launch_moe_dispatch(a, dtype == MUON_BF16, s), "launch dispatch");
  } catch (...) {
    return fail(MUON_ERR_HIP, "unexpected host exception");
  }
}

extern "C" int32_t muon_moe_combine(int64_t tokens, int32_t top_k, int64_t cols, int64_t y_rows,
                                    const void* y, const int32_t* rows, const float* weights,
                                    void* out, int32_t dtype, void* stream) {
  try {
    clear_detail();
    MoeRowArgs a;
    int32_t st = row_args(tokens, top_k, cols, y_rows, rows, dtype, a);
    if (st != MUON_OK) return st;
    if ((st = check_array(y, y_rows * cols, 16, "y")) != MUON_OK) return st;
    if ((st = check_array(weights, weights != nullptr ? 1 : 0, 4, "weights")) != MUON_OK) return st;
    if ((st = check_array(out, tokens * cols, 16, "out")) != MUON_OK) return st;
    if ((st = apart(out, tokens * a.row_bytes, y, y_rows * a.row_bytes, "out")) != MUON_OK) return st;
    if (tokens == 0 || cols == 0) return MUON_OK;
    a.sorted = y;
    a.weights = weights;
    a.out = out;
    hipStream_t s = static_cast<hipStream_t>(stream);
    TimedLaunch tl(MUON_K_MOE_COMBINE, s);
    return launched(tl, launch_moe_combine(a, dtype == MUON_BF16, s), "launch combine");
  } catch (...) {
    return fail(MUON_ERR_HIP, "unexpected host exception");
  }
}

extern "C" int32_t muon_moe_combine_backward(int64_t tokens, int32_t top_k, int64_t cols,
                                             const void* dout, int64_t y_rows, const void* y,
                                             const int32_t* rows, const float* weights, void* dy,
                                             float* dweights, int32_t dtype, void* stream) {
  try {
    clear_detail();
    MoeRowArgs a;
    int32_t st = row_args(tokens, top_k, cols, y_rows, rows, dtype, a);
    if (st != MUON_OK) return st;
    if ((st = check_array(dout, tokens * cols, 16, "dout")) != MUON_OK) return st;
    if ((st = check_array(y, y_rows * cols, 16, "y")) != MUON_OK) return st;
    if ((st = check_array(weights, tokens, 4, "weights")) != MUON_OK) return st;
    if ((st = check_array(dy, y_rows * cols, 16, "dy")) != MUON_OK) return st;
    if ((st = check_array(dweights, tokens, 4, "dweights")) != MUON_OK) return st;
    const int64_t y_bytes = y_rows * a.row_bytes, w_bytes = tokens * top_k * 4;
    if ((st = apart(dy, y_bytes, y, y_bytes, "dy")) != MUON_OK) return st;
    if ((st = apart(dy, y_bytes, dout, tokens * a.row_bytes, "dy")) != MUON_OK) return st;
    if ((st = apart(dweights, w_bytes, weights, w_bytes, "dweights")) != MUON_OK) return st;
    if (tokens == 0) return MUON_OK;
    a.tokens = dout;
    a.sorted = y;
    a.weights = weights;
    a.out = dy;
    a.dweights = dweights;
    hipStream_t s = static_cast<hipStream_t>(stream);
    TimedLaunch tl(MUON_K_MOE_BACKWARD, s);
    return launched(tl, launch_moe_backward(a, dtype == MUON_BF16, s), "launch combine's gradient");
  } catch (...) {
    return fail(MUON_ERR_HIP, "unexpected host exception");
  }
}

extern "C" size_t muon_f4_workspace_bytes(int32_t count) {
  clear_detail();
  if (check_experts(count, "count") != MUON_OK) return SIZE_MAX;
  return align_up(sizeof(void*) * static_cast<size_t>(count), kAlign);
}

extern "C" int32_t muon_f4_quantize(int32_t count, int64_t rows, int64_t cols,
                                    const void* const* w, int32_t dtype, int32_t transpose,
                                    void* q, void* s, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  try {
    clear_detail();
    int32_t st = check_experts(count, "count");
    if (st != MUON_OK) return st;
    if ((st = check_size(rows, MUON_F8_MAX_DIM, "rows")) != MUON_OK) return st;
    if ((st = check_size(cols, MUON_F8_MAX_DIM, "cols")) != MUON_OK) return st;
    if ((st = check_dtype(dtype)) != MUON_OK) return st;
    if (transpose != 0 && transpose != 1)
      return fail(MUON_ERR_INVALID_ARG, "transpose must be 0 or 1");
    F4QuantArgs a{};
    a.rows = static_cast<int32_t>(rows);
    a.cols = static_cast<int32_t>(cols);
    a.rtiles = static_cast<int32_t>(cdiv(rows, 16));
    a.ktiles = static_cast<int32_t>(cdiv(cols, kF4Tile));
    a.tiles = static_cast<int64_t>(count) * a.rtiles * a.ktiles;
    if (a.tiles >= kMaxTiles) return fail(MUON_ERR_UNSUPPORTED, "2^28 tiles or more");
    if (a.tiles > 0) {
      if (w == nullptr) return fail(MUON_ERR_INVALID_ARG, "w array is null");
      for (int32_t i = 0; i < count; ++i)
        if ((st = check_array(w[i], 1, 16, "w")) != MUON_OK) return st;
    }
    if ((st = check_array(q, a.tiles, 16, "q")) != MUON_OK) return st;
    if ((st = check_array(s, a.tiles, 16, "s")) != MUON_OK) return st;
    const size_t need = muon_f4_workspace_bytes(count);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != MUON_OK) return st;
    if (a.tiles == 0) return MUON_OK;
    a.q = static_cast<char*>(q);
    a.s = static_cast<char*>(s);
    hipStream_t stm = static_cast<hipStream_t>(stream);
    ArgTable t;
    if ((st = place_table(w, sizeof(void*) * static_cast<size_t>(count), nullptr, 0,
                          static_cast<char*>(workspace), stm, t, &a.table)) != MUON_OK)
      return st;
    TimedLaunch tl(MUON_K_F4_QUANTIZE, stm);
    return launched(tl, launch_f4_quantize(t, a, dtype == MUON_BF16, transpose != 0, stm),
                    "launch 4-bit quantization");
  } catch (...) {
    return fail(MUON_ERR_HIP, "unexpected host exception");
  }
}

extern "C" int32_t muon_f4_matmul(int32_t count, int64_t rows, int64_t cols, const void* q,
                                  const void* s, int64_t m, const void* x, int64_t x_rows,
                                  const int32_t* offsets, const int32_t* active,
                                  const int32_t* slots, int32_t top_k, void* y, int32_t dtype,
                                  void* stream) {
  try {
    clear_detail();
    int32_t st = check_experts(count, "count");
    if (st != MUON_OK) return st;
    if ((st = check_size(rows, MUON_F8_MAX_DIM, "rows")) != MUON_OK) return st;
    if ((st = check_size(cols, MUON_F8_MAX_DIM, "cols")) != MUON_OK) return st;
    if ((st = check_size(m, kMoeMaxSlots, "m")) != MUON_OK) return st;
    if ((st = check_size(x_rows, kMoeMaxSlots, "x_rows")) != MUON_OK) return st;
    if ((st = check_dtype(dtype)) != MUON_OK) return st;
    if ((offsets == nullptr) != (active == nullptr))
      return fail(MUON_ERR_INVALID_ARG, "offsets and active go together");
    if (offsets == nullptr && (count != 1 || slots != nullptr))
      return fail(MUON_ERR_INVALID_ARG, "without offsets there is one matrix, and no slots");
    if (slots == nullptr && x_rows < m)
      return fail(MUON_ERR_INVALID_ARG, "x has fewer rows than y");
    if (slots != nullptr && (top_k < 1 || top_k > kMoeMaxTopK))
      return fail(MUON_ERR_INVALID_ARG, "top_k = %d: must lie in [1, %d]", top_k, kMoeMaxTopK);
    if (slots != nullptr && x_rows == 0 && m > 0)
      return fail(MUON_ERR_INVALID_ARG, "x has no rows");
    if ((st = check_array(offsets, offsets != nullptr ? 1 : 0, 4, "offsets")) != MUON_OK) return st;
    if ((st = check_array(active, active != nullptr ? 1 : 0, 4, "active")) != MUON_OK) return st;
    if ((st = check_array(slots, slots != nullptr ? 1 : 0, 4, "slots")) != MUON_OK) return st;
    F4ProdArgs a{};
    a.rows = static_cast<int32_t>(rows);
    a.cols = static_cast<int32_t>(cols);
    a.rtiles = static_cast<int32_t>(cdiv(rows, 16));
    a.ktiles = static_cast<int32_t>(cdiv(cols, kF4Tile));
    const int64_t tiles = static_cast<int64_t>(count) * a.rtiles * a.ktiles;
    if (tiles >= kMaxTiles) return fail(MUON_ERR_UNSUPPORTED, "2^28 tiles or more");
    if (m == 0 || rows == 0) return MUON_OK;
    if ((st = check_array(q, tiles, 16, "q")) != MUON_OK) return st;
    if ((st = check_array(s, tiles, 16, "s")) != MUON_OK) return st;
    if ((st = check_array(x, tiles, 16, "x")) != MUON_OK) return st;
    if ((st = check_array(y, 1, 16, "y")) != MUON_OK) return st;
    const int64_t y_bytes = m * rows * (dtype == MUON_BF16 ? 2 : 4);
    if ((st = apart(y, y_bytes, x, x_rows * cols * 2, "y")) != MUON_OK) return st;
    a.q = static_cast<const char*>(q);
    a.s = static_cast<const char*>(s);
    a.x = x;
    a.offsets = offsets;
    a.active = active;
    a.slots = slots;
    a.y = y;
    a.m = m;
    a.x_rows = x_rows;
    a.experts = count;
    a.top_k = top_k;
    hipStream_t stm = static_cast<hipStream_t>(stream);
    TimedLaunch tl(MUON_K_F4_PROD, stm);
    return launched(tl, launch_f4_matmul(a, dtype == MUON_BF16, stm), "launch 4-bit product");
  } catch (...) {
    return fail(MUON_ERR_HIP, "unexpected host exception");
  }
}
