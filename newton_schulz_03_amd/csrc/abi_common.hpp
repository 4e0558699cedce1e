// Host helpers shared by the C ABI's translation units (muon_abi.hip defines
// them): the error detail of a thread, alignment, per-kernel timing.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "muon_internal.hpp"

namespace muon {

// Records the detail string of this thread's last error; returns `status`.
int32_t fail(int32_t status, const char* fmt, ...);
int32_t hip_fail(hipError_t e, const char* what);
void clear_detail();

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Null, too small or misaligned workspaces, as every entry point reports them.
int32_t check_workspace(const void* ws, size_t ws_bytes, size_t need);

// A call's descriptor table: n descriptors of `desc_bytes` together, then a
// second array (prefixes, or pointers; align_up(desc_bytes, kAlign) on).  Where
// it fits it becomes the kernels' argument table; otherwise kernels that carry
// its pieces write it to `ws`.  *mem: where it lies (null: the argument table).
// Kernel launches only, so that calls can be captured into a graph.
int32_t place_table(const void* desc, size_t desc_bytes, const void* second, size_t second_bytes,
                    char* ws, hipStream_t stream, ArgTable& args, const void** mem);

// Brackets one launch with timing events when timing is enabled (and allowed:
// the allocation-free entry point never creates events).
struct TimedLaunch {
  int kernel;
  hipStream_t stream;
  hipEvent_t start = nullptr, stop = nullptr;
  TimedLaunch(int k, hipStream_t s, bool allowed = true);
  void done();
};

}  // namespace muon
