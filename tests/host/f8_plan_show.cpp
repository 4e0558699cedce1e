// Host-only: which kernels and tiles a block-scaled e4m3 product takes.
//
// Built with `hipcc --offload-host-only` against the ABI source itself, with stub
// kernel launchers (no kernel is compiled or run).  Arguments: dtype (0 bf16, 1
// fp32), accumulate, then m n k of each product.  Prints one line: full half quarter
// (tiles), spread (of the tiles), nt, blocks mt nt spread (of the few-rows kernel).
#include "ops_abi.hip"

#include <cstdio>
#include <cstdlib>

namespace muon {
int32_t fail(int32_t status, const char*, ...) { return status; }
int32_t hip_fail(hipError_t, const char*) { return MUON_ERR_HIP; }
void clear_detail() {}
int32_t check_workspace(const void*, size_t, size_t) { return MUON_OK; }
int32_t place_table(const void*, size_t, const void*, size_t, char*, hipStream_t, ArgTable&,
                    const void** mem) {
  *mem = nullptr;
  return MUON_OK;
}
TimedLaunch::TimedLaunch(int k, hipStream_t s, bool) : kernel(k), stream(s) {}
void TimedLaunch::done() {}
hipError_t launch_grad_norm(const ArgTable&, const GradCtx&, const GradNormArgs&, int32_t, int64_t) {
  return hipSuccess;
}
hipError_t launch_grad_scale(const ArgTable&, const GradCtx&, int32_t, const float*,
                             const GradNormArgs*, int32_t, int64_t) {
  return hipSuccess;
}
bool grad_few_blocks(int32_t) { return false; }
hipError_t launch_f8_quantize(const ArgTable&, const F8QuantCtx&, int32_t, bool, int32_t, int64_t) {
  return hipSuccess;
}
hipError_t launch_f8_prod(const ArgTable&, const F8ProdCtx& c, int32_t nfull, int32_t nhalf,
                          int32_t nquarter, bool) {
  std::printf("%d %d %d %d %d ", nfull, nhalf, nquarter, c.spread, c.nt);
  return hipSuccess;
}
hipError_t launch_f8_small(const ArgTable&, const F8ProdCtx& c, int32_t nblocks, bool, int32_t mt,
                           int32_t nt) {
  std::printf("%d %d %d %d\n", nblocks, mt, nt, c.spread);
  return hipSuccess;
}
}  // namespace muon

int main(int argc, char** argv) {
  if (argc < 3 || argc % 3 != 0) return 2;
  const int32_t batch = argc / 3 - 1;
  std::vector<int64_t> m(batch), n(batch), k(batch);
  for (int32_t i = 0; i < batch; ++i) {
    m[i] = std::atoll(argv[3 + 3 * i]);
    n[i] = std::atoll(argv[4 + 3 * i]);
    k[i] = std::atoll(argv[5 + 3 * i]);
  }
  const std::vector<void*> p(batch, reinterpret_cast<void*>(4096));
  return muon_f8_matmul_batched(batch, m.data(), n.data(), k.data(), p.data(), p.data(), p.data(),
                                p.data(), p.data(), std::atoi(argv[1]), std::atoi(argv[2]),
                                reinterpret_cast<void*>(4096), SIZE_MAX, nullptr);
}
