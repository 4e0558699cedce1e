// Host-only check of where AdamW's table of tensors goes.
//
// Built with `hipcc --offload-host-only` against the ABI source itself, with stub
// kernel launchers and stub runtime calls (no kernel is compiled or run).  A call
// whose table fits the kernels' arguments, or that has enough blocks for several
// launches with such tables, copies nothing; any other call takes one copy from a
// pinned slot and one launch, and, on a stream that is being captured, kernels that
// carry the table instead of the copy.  In every case the launches together hold
// each tensor once, with its pointers and its first block.
// Prints "OK" and exits 0, or names the first failure and exits 1.
#include "muon_abi.hip"

#include <cstdio>
#include <cstdlib>

namespace {

int copies = 0, written = 0, launches = 0;
hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
hipError_t capture_error = hipSuccess;
std::vector<muon::AdamDesc> seen;
std::vector<int32_t> first_block;

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
hipError_t hipEventRecord(hipEvent_t, hipStream_t) { return hipSuccess; }
hipError_t hipEventQuery(hipEvent_t) { return hipSuccess; }
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipMemcpyAsync(void* to, const void* from, size_t n, hipMemcpyKind, hipStream_t) {
  ++copies;
  std::memcpy(to, from, n);
  return hipSuccess;
}
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus* s) {
  *s = capture;
  return capture_error;
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
hipError_t launch_adamw(const AdamCtx& c, int32_t nblocks, bool, const AdamParams&) {
  const char* const t = c.table != nullptr ? static_cast<const char*>(c.table)
                                           : reinterpret_cast<const char*>(c.args->bytes);
  const AdamDesc* const d = reinterpret_cast<const AdamDesc*>(t);
  const int32_t* const p = reinterpret_cast<const int32_t*>(t + c.prefix_off);
  const int32_t before = first_block.empty() ? 0 : first_block.back();
  if (first_block.empty()) first_block.push_back(0);
  for (int32_t i = 0; i < c.batch; ++i) {
    seen.push_back(d[i]);
    first_block.push_back(before + p[i + 1]);
  }
  expect(p[0] == 0 && p[c.batch] == nblocks, "the prefixes do not span the launch", "launch");
  ++launches;
  return hipSuccess;
}
}  // namespace muon

namespace {

void call(const char* where, int32_t batch, int64_t numel, bool enough, bool captured) {
  std::vector<int64_t> n(batch);
  std::vector<void*> p(batch), g(batch);
  std::vector<float*> m(batch), v(batch);
  for (int32_t i = 0; i < batch; ++i) {
    n[i] = i % 7 == 3 ? 0 : numel + i % 5;
    p[i] = reinterpret_cast<void*>((4 * static_cast<intptr_t>(i) + 1) << 12);
    g[i] = reinterpret_cast<void*>((4 * static_cast<intptr_t>(i) + 2) << 12);
    m[i] = reinterpret_cast<float*>((4 * static_cast<intptr_t>(i) + 3) << 12);
    v[i] = reinterpret_cast<float*>((4 * static_cast<intptr_t>(i) + 4) << 12);
  }
  const size_t bytes = muon_adamw_workspace_bytes(batch, n.data());
  std::vector<char> room(bytes + 256);
  char* const ws = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(room.data()) + 255) / 256 * 256);
  copies = written = launches = 0;
  seen.clear();
  first_block.clear();
  const muon_adamw_params prm{1e-3f, 0.9f, 0.95f, 1e-8f, 0.1f, 3};
  const int32_t st = muon_adamw_batched(batch, n.data(), p.data(), g.data(), m.data(), v.data(), 0,
                                        &prm, ws, bytes, nullptr);
  expect(st == MUON_OK, muon_last_error_detail(), where);
  const bool args = batch <= 83 || enough;
  expect(copies == (args || captured ? 0 : 1), "copies", where);
  expect((written > 0) == (!args && captured), "kernels that write the table", where);
  expect(launches == (args ? (batch + 82) / 83 : 1), "launches", where);
  expect(seen.size() == static_cast<size_t>(batch), "tensors", where);
  int32_t blocks = 0;
  for (int32_t i = 0; i < batch && failures == 0; ++i) {
    const muon::AdamDesc& d = seen[i];
    expect(first_block[i] == blocks, "first block", where);
    expect(d.numel == n[i], "numel", where);
    if (n[i] > 0)
      expect(d.p == p[i] && d.g == g[i] && d.m == m[i] && d.v == v[i], "pointers", where);
    blocks += static_cast<int32_t>((n[i] + 1023) / 1024);
  }
}

}  // namespace

int main() {
  for (const bool captured : {false, true}) {
    capture = captured ? hipStreamCaptureStatusActive : hipStreamCaptureStatusNone;
    call("one", 1, 1000, false, captured);
    call("83 small", 83, 1000, false, captured);
    call("84 small", 84, 1000, false, captured);
    call("4000 small", 4000, 100, false, captured);
    call("2000 of 5 blocks", 2000, 5000, false, captured);
    call("200 large", 200, 1 << 20, true, captured);
  }
  capture = hipStreamCaptureStatusNone;
  capture_error = hipErrorStreamCaptureImplicit;  // the null stream beside another's capture
  call("4000 beside a capture", 4000, 100, false, true);
  if (failures) return 1;
  std::puts("OK");
  return 0;
}
