// Host-only check of what captured calls enqueue.
//
// Built with `hipcc --offload-host-only` against the ABI source itself, with stub
// kernel launchers and stub runtime calls (no kernel is compiled or run).  The step,
// with and without a factor, and the orthogonalization copy their descriptor table
// from a pinned slot; on a stream that is being captured they copy nothing and
// record no event, and kernels carry the table, with the same bytes.  A step with
// the momentum in host memory is refused there.
// Prints "OK" and exits 0, or names the first failure and exits 1.
#include "muon_abi.hip"

#include <cstdio>
#include <cstdlib>

namespace {

int copies = 0, written = 0, events = 0;
hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;

int failures = 0;
void expect(bool ok, const char* what, const char* where) {
  if (!ok && failures++ == 0) std::printf("FAIL %s: %s\n", where, what);
}

}  // namespace

// the runtime calls of a staged copy
extern "C" {
hipError_t hipGetDevice(int* d) {
  *d = 0;
  return hipSuccess;
}
hipError_t hipHostMalloc(void** p, size_t n, unsigned int) {
  *p = std::malloc(n);
  return hipSuccess;
}
hipError_t hipHostFree(void* p) {
  std::free(p);
  return hipSuccess;
}
hipError_t hipEventCreateWithFlags(hipEvent_t* e, unsigned) {
  *e = reinterpret_cast<hipEvent_t>(16);
  return hipSuccess;
}
hipError_t hipEventRecord(hipEvent_t, hipStream_t) {
  ++events;
  return hipSuccess;
}
hipError_t hipEventQuery(hipEvent_t) { return hipSuccess; }
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipMemcpyAsync(void* to, const void* from, size_t n, hipMemcpyKind, hipStream_t) {
  ++copies;
  std::memcpy(to, from, n);
  return hipSuccess;
}
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus* s) {
  *s = capture;
  return hipSuccess;
}
hipError_t hipPointerGetAttributes(hipPointerAttribute_t* a, const void*) {
  a->type = hipMemoryTypeHost;
  return hipSuccess;
}
}

namespace muon {
hipError_t launch_prepare(const LaunchCtx&, int32_t, bool, const ElemParams&) { return hipSuccess; }
hipError_t launch_finalize(const LaunchCtx&, const ElemParams&) { return hipSuccess; }
hipError_t launch_finish(const LaunchCtx&, int32_t, bool, const ElemParams&) { return hipSuccess; }
hipError_t launch_gram(const LaunchCtx&, const XcdSplit&, bool, int32_t, float, bool) {
  return hipSuccess;
}
hipError_t launch_poly(const LaunchCtx&, const XcdSplit&, bool, float, float) {
  return hipSuccess;
}
hipError_t launch_prod(const LaunchCtx&, const XcdSplit&, bool, int32_t, float, bool, bool,
                       int32_t, float) {
  return hipSuccess;
}
hipError_t launch_prod_wide(const LaunchCtx&, const XcdSplit&, int32_t, float, bool, bool) {
  return hipSuccess;
}
hipError_t noalloc_scratch(char**) { return hipErrorInvalidSymbol; }
hipError_t launch_quant8(const LaunchCtx&, int32_t, int32_t, int32_t) { return hipSuccess; }
hipError_t launch_gram8(const LaunchCtx&, const XcdSplit&, float, bool) { return hipSuccess; }
hipError_t launch_poly8(const LaunchCtx&, const XcdSplit&, float, float) { return hipSuccess; }
hipError_t launch_prod8(const LaunchCtx&, const XcdSplit&, int32_t, float, bool) {
  return hipSuccess;
}
hipError_t launch_put_bytes(const void* from, size_t n, void* to, hipStream_t) {
  ++written;
  std::memcpy(to, from, n);
  return hipSuccess;
}
int64_t adamw_blocks(int64_t n) { return (n + 1023) / 1024; }
hipError_t launch_adamw(const AdamCtx&, int32_t, bool, const AdamParams&) { return hipSuccess; }
}  // namespace muon

namespace {

enum Call { kNs, kStep, kScaled, kHost };

// Pointer number k of the matrices.
void* fake(int32_t k) {
  return reinterpret_cast<void*>((intptr_t{1} << 56) + (static_cast<intptr_t>(k) << 24));
}

// Runs a call over a ragged batch; returns its status and the bytes of the tables.
int32_t run_call(Call which, int32_t batch, std::vector<char>& table) {
  std::vector<int64_t> rows(batch), cols(batch);
  std::vector<void*> w(batch), g(batch), m(batch);
  for (int32_t i = 0; i < batch; ++i) {
    rows[i] = 64 + 33 * (i % 9);
    cols[i] = 200 + 71 * (i % 5);
    w[i] = fake(4 * i + 1);
    g[i] = fake(4 * i + 2);
    m[i] = fake(4 * i + 3);
  }
  const size_t bytes = muon_workspace_bytes_ex(batch, rows.data(), cols.data(), 0,
                                               which == kHost ? MUON_WS_MOMENTUM_HOST : 0);
  table.assign(bytes + 256, 0);
  char* const ws =
      reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(table.data()) + 255) / 256 * 256);
  muon_step_params p{};
  p.lr = 0.02f;
  p.beta = 0.95f;
  p.ns.steps = 5;
  p.ns.a = 3.4445f;
  p.ns.b = -4.775f;
  p.ns.c = 2.0315f;
  p.ns.eps = 1e-7f;
  p.momentum_host = which == kHost;
  const float* const factor = reinterpret_cast<const float*>(4096);
  copies = written = events = 0;
  int32_t st;
  if (which == kNs)
    st = muon_ns_batched(batch, rows.data(), cols.data(), g.data(), w.data(), 0, &p.ns, ws, bytes,
                         nullptr);
  else if (which == kScaled)
    st = muon_step_batched_scaled(batch, rows.data(), cols.data(), w.data(), g.data(), m.data(), 0,
                                  &p, factor, ws, bytes, nullptr);
  else
    st = muon_step_batched(batch, rows.data(), cols.data(), w.data(), g.data(), m.data(), 0, &p, ws,
                           bytes, nullptr);
  // the descriptors' pointers into the workspace differ from call to call: as offsets
  muon::MatDesc* const desc = reinterpret_cast<muon::MatDesc*>(ws);
  if (st == MUON_OK)
    for (int32_t i = 0; i < batch; ++i)
      for (void** q : {&desc[i].x[0], &desc[i].x[1], &desc[i].gram, &desc[i].poly})
        *q = reinterpret_cast<void*>(static_cast<char*>(*q) - ws);
  table.erase(table.begin(), table.begin() + (ws - table.data()));
  table.resize(bytes);
  return st;
}

}  // namespace

int main() {
  const struct {
    Call which;
    const char* name;
  } calls[] = {{kNs, "orthogonalization"}, {kStep, "step"}, {kScaled, "step with a factor"}};
  for (const auto& c : calls)
    for (const int32_t batch : {1, 7, 300}) {
      std::vector<char> eager, captured;
      capture = hipStreamCaptureStatusNone;
      expect(run_call(c.which, batch, eager) == MUON_OK, muon_last_error_detail(), c.name);
      expect(copies > 0 && events > 0 && written == 0, "an eager call copies its table", c.name);
      capture = hipStreamCaptureStatusActive;
      expect(run_call(c.which, batch, captured) == MUON_OK, muon_last_error_detail(), c.name);
      expect(copies == 0 && events == 0 && written > 0, "a captured call copies nothing", c.name);
      expect(eager == captured, "the tables differ", c.name);
    }
  std::vector<char> none;
  capture = hipStreamCaptureStatusActive;
  expect(run_call(kHost, 3, none) == MUON_ERR_UNSUPPORTED, "not refused", "momentum in host memory");
  expect(copies == 0 && events == 0 && written == 0, "enqueued something", "momentum in host memory");
  if (failures) return 1;
  std::puts("OK");
  return 0;
}
