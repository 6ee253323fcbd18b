// host_workspace.cpp - how a stream's workspace grows, without a GPU: ns_host.cpp
// is linked with a HIP runtime that only counts bytes.
//
//   * sizes that rise slowly: few allocations, and what is held stays within
//     four times the largest size;
//   * a card with no room for twice the old buffer: the size that is needed;
//   * a failed allocation leaves the workspace as it was.
#include <hip/hip_runtime_api.h>

#include <cstdio>
#include <cstring>
#include <map>

#include "ns_host.h"
#include "ns_kernels.h"

namespace {
size_t g_held = 0, g_room = ~size_t(0);
std::map<void*, size_t> g_sizes;
}  // namespace

extern "C" {
hipError_t hipGetDevice(int* d) { return *d = 0, hipSuccess; }
hipError_t hipSetDevice(int) { return hipSuccess; }
hipError_t hipDeviceSynchronize() { return hipSuccess; }
hipError_t hipGetLastError() { return hipSuccess; }
const char* hipGetErrorString(hipError_t) { return "error"; }
hipError_t hipMalloc(void** p, size_t n) {
  static uintptr_t next = 0x7000000000000000ull;
  if (n > g_room - g_held) return hipErrorOutOfMemory;
  *p = (void*)next;
  next += (n + 4095) / 4096 * 4096;
  g_sizes[*p] = n;
  g_held += n;
  return hipSuccess;
}
hipError_t hipFree(void* p) {
  g_held -= g_sizes.at(p);
  g_sizes.erase(p);
  return hipSuccess;
}
hipError_t hipGetDeviceProperties(hipDeviceProp_t* p, int) {  // (a macro may give it a suffix)
  std::memset(p, 0, sizeof(*p));
  return hipSuccess;
}
hipError_t hipEventCreateWithFlags(hipEvent_t*, unsigned) { return hipErrorUnknown; }
hipError_t hipEventSynchronize(hipEvent_t) { return hipSuccess; }
hipError_t hipEventElapsedTime(float* ms, hipEvent_t, hipEvent_t) { return *ms = 0, hipSuccess; }
}

namespace ns {
void set_launch_events(hipEvent_t, hipEvent_t) {}
}  // namespace ns

namespace {
int g_bad = 0;
void check(bool ok, const char* what, size_t at) {
  if (ok) return;
  ++g_bad;
  std::printf("%s (at %zu bytes: %zu held in %zu buffers)\n", what, at, g_held, g_sizes.size());
}
int ask(size_t bytes, char** ptr = nullptr) {
  ns::Workspace w;
  const int s = ns::get_workspace((hipStream_t)0x100, bytes, &w);
  if (ptr) *ptr = w.ptr;
  if (s == NS_OK) check(g_sizes.at(w.ptr) >= bytes, "a buffer that is too small", bytes);
  return s;
}
}  // namespace

int main() {
  const size_t MB = size_t(1) << 20;
  const int64_t before = ns_workspace_allocations();
  for (size_t n = 1000 * MB; n <= 64000 * MB; n += 37 * MB) {  // 1703 sizes, 64 times as large in the end
    check(ask(n) == NS_OK, "refused", n);
    check(g_held <= 4 * n, "more than four times the size held", n);
  }
  const int64_t made = ns_workspace_allocations() - before;
  check(made <= 8, "more allocations than the size doubles", (size_t)made);
  check(ask(10 * MB) == NS_OK && ns_workspace_allocations() - before == made, "a warm call allocated", 10 * MB);
  check(ns_release_workspace() == NS_OK && g_held == 0, "not all freed", 0);

  check(ask(1000 * MB) == NS_OK && g_held == 1000 * MB, "the first buffer is of the size asked for", 1000 * MB);
  check(ask(5000 * MB) == NS_OK && g_held == 6000 * MB, "a much larger one too", 5000 * MB);
  g_room = 6000 * MB + 5300 * MB;  // no room for 10000 MB
  char *a = nullptr, *b = nullptr;
  check(ask(5200 * MB, &a) == NS_OK && g_held == 11200 * MB, "where there is no room for more: what is needed", 5200 * MB);
  check(ask(5400 * MB) == NS_ERR_OOM, "no room at all", 5400 * MB);
  check(ask(5200 * MB, &b) == NS_OK && a == b, "a failed call leaves the workspace as it was", 5200 * MB);
  check(ns_release_workspace() == NS_OK && g_held == 0, "not all freed", 0);
  std::printf("%d allocations for sizes 64 times as large in the end, %d faults\n", (int)made, g_bad);
  return g_bad != 0;
}
