// C ABI of dropout.  Kernel launches only, so that a call can be captured into a
// graph.
#include <cmath>

#include "abi_common.hpp"
#include "grad_plan.hpp"
#include "muon_internal.hpp"
#include "muon_mi355x.h"

using namespace muon;

extern "C" int32_t muon_dropout_batched(int32_t batch, const int64_t* numel, const void* const* x,
                                        const int32_t* dtype, void* const* out,
                                        const int32_t* out_dtype, const muon_dropout_params* p,
                                        const uint64_t* rng, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  try {
    clear_detail();
    GradPlan pl;
    int32_t st = make_grad_plan(batch, numel, pl);
    if (st != MUON_OK) return st;
    if (p == nullptr) return fail(MUON_ERR_INVALID_ARG, "params pointer is null");
    if (!(p->p >= 0.0 && p->p <= 1.0)) return fail(MUON_ERR_INVALID_ARG, "p must lie in [0, 1]");
    if ((reinterpret_cast<uintptr_t>(rng) & 7u) != 0)
      return fail(MUON_ERR_INVALID_ARG, "rng pointer not 8-byte aligned");
    for (int32_t i = 0; i < batch; ++i)
      if (numel[i] >= kDropMaxNumel)
        return fail(MUON_ERR_UNSUPPORTED, "tensor %d: %lld elements; the limit is 2^35", i,
                    static_cast<long long>(numel[i]));
    if (batch == 0) return MUON_OK;
    if (out == nullptr) return fail(MUON_ERR_INVALID_ARG, "out array is null");
    if ((st = bind_grads(batch, numel, x, dtype, out, out_dtype, pl)) != MUON_OK) return st;
    if ((st = check_workspace(workspace, workspace_bytes, pl.total_bytes)) != MUON_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    ArgTable t;
    GradCtx c{};
    if ((st = grad_table(pl, static_cast<char*>(workspace), s, t, c)) != MUON_OK) return st;
    DropArgs a{};
    a.rng = rng;
    a.seed = p->seed;
    a.offset = p->offset;
    a.threshold = static_cast<uint32_t>(std::nearbyint(p->p * 65536.0));
    a.scale = a.threshold < 65536u ? static_cast<float>(65536.0 / (65536.0 - a.threshold)) : 0.f;
    TimedLaunch tl(MUON_K_DROPOUT, s);
    const hipError_t e = launch_dropout(t, c, pl.chunks, a, pl.in_bytes + pl.out_bytes);
    if (e != hipSuccess) return hip_fail(e, "launch dropout");
    tl.done();
    return MUON_OK;
  } catch (...) {
    return fail(MUON_ERR_HIP, "unexpected host exception");
  }
}
