// host_threads.cpp - the host drivers of the library under several threads,
// without a GPU: ns_host.cpp, ns_api.cpp and ns_sublayer.cpp are linked with
// a HIP runtime and kernel launches that only write down who launched, on
// which stream.
//
//   * calls of several threads on one stream: whatever a call enqueues with
//     the stream's workspace is one run of that stream, with no other call's
//     launches inside it;
//   * calls on different streams do not wait for each other.
#include <hip/hip_runtime_api.h>

#include <atomic>
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <mutex>
#include <set>
#include <thread>
#include <vector>

#include "ns_hip.h"
#include "ns_kernels.h"
#include "ns_sublayer.h"

namespace {

thread_local int t_call = 0;  // the call that this thread is inside, a number of its own
std::atomic<int> g_calls{0};
std::mutex g_mu;
std::map<void*, std::vector<int>> g_log;  // stream -> the call of each launch, in order

void* const kWaits = (void*)0x100;  // a call on this stream waits until one on kOther has ended
void* const kOther = (void*)0x200;
std::condition_variable g_cv;
bool g_other_done = false, g_waited_in_vain = false;

hipError_t launched(hipStream_t st, int launches = 1) {
  for (int i = 0; i < launches; ++i) {
    {
      std::unique_lock<std::mutex> lk(g_mu);
      g_log[(void*)st].push_back(t_call);
      if ((void*)st == kWaits && !g_other_done &&
          !g_cv.wait_for(lk, std::chrono::seconds(20), [] { return g_other_done; }))
        g_waited_in_vain = true;
    }
    std::this_thread::sleep_for(std::chrono::microseconds(50));  // where another thread could come in
  }
  return hipSuccess;
}

}  // namespace

// ------------------------------------------------------- the HIP runtime

extern "C" {
hipError_t hipGetDevice(int* d) { return *d = 0, hipSuccess; }
hipError_t hipSetDevice(int) { return hipSuccess; }
hipError_t hipDeviceSynchronize() { return hipSuccess; }
hipError_t hipGetLastError() { return hipSuccess; }
const char* hipGetErrorString(hipError_t) { return "error"; }
hipError_t hipMalloc(void** p, size_t n) {
  static std::atomic<uintptr_t> next{0x7000000000000000ull};
  return *p = (void*)next.fetch_add((n + 4095) / 4096 * 4096), hipSuccess;
}
hipError_t hipFree(void*) { return hipSuccess; }
hipError_t hipMemset(void*, int, size_t) { return hipSuccess; }
hipError_t hipMemsetAsync(void*, int, size_t, hipStream_t st) { return launched(st); }
hipError_t hipMemcpyAsync(void*, const void*, size_t, hipMemcpyKind, hipStream_t st) { return launched(st); }
hipError_t hipMemcpy(void*, const void*, size_t, hipMemcpyKind) { return hipSuccess; }
hipError_t hipGetDeviceProperties(hipDeviceProp_t* p, int) {  // (a macro may give it a suffix)
  std::memset(p, 0, sizeof(*p));
  std::strcpy(p->gcnArchName, "gfx950");
  return hipSuccess;
}
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) { return *v = 256, hipSuccess; }
hipError_t hipEventCreate(hipEvent_t*) { return hipErrorUnknown; }
hipError_t hipEventCreateWithFlags(hipEvent_t*, unsigned) { return hipErrorUnknown; }
hipError_t hipEventDestroy(hipEvent_t) { return hipSuccess; }
hipError_t hipEventRecord(hipEvent_t, hipStream_t) { return hipSuccess; }
hipError_t hipEventSynchronize(hipEvent_t) { return hipSuccess; }
hipError_t hipEventElapsedTime(float* ms, hipEvent_t, hipEvent_t) { return *ms = 0, hipSuccess; }
}

// ------------------------------------------------- the kernels' launches

namespace ns {
void set_launch_events(hipEvent_t, hipEvent_t) {}
hipError_t launch_gemm(int, const StageKind&, const GemmArgs&, hipStream_t st) { return launched(st); }
hipError_t launch_gemm_grouped(int, const StageKind&, const GemmArgs*, int, hipStream_t st) { return launched(st); }
hipError_t launch_sumsq(int, const NormArgs&, int, hipStream_t st) { return launched(st); }
hipError_t launch_sumsq_grouped(int, const NormArgs*, const int*, int, hipStream_t st) { return launched(st); }
hipError_t launch_scale(int, const NormArgs&, int, hipStream_t st) { return launched(st); }
hipError_t launch_pad_sumsq(int, const PadArgs&, const NormArgs&, int, hipStream_t st) { return launched(st); }
hipError_t launch_unpad(int, const PadArgs&, hipStream_t st) { return launched(st); }
hipError_t noalloc_scratch(int, char** p) { return *p = (char*)0x1000, hipSuccess; }
hipError_t launch_mfma_peak(int, int, int, float*, unsigned long long*, hipStream_t st) { return launched(st); }
long long mfma_peak_flops_per_inst(int) { return 1; }
int mfma_peak_acc() { return 1; }
hipError_t launch_layer_norm(int, const LayerNormArgs&, hipStream_t st) { return launched(st); }
hipError_t launch_layer_norm_backward(int, const LayerNormGradArgs&, int, hipStream_t st) { return launched(st, 2); }
hipError_t launch_route(int, const RouteArgs&, hipStream_t st) { return launched(st, 3); }
hipError_t launch_route_backward(int, const RouteGradArgs&, hipStream_t st) { return launched(st); }
const char* experts_config(int, ExpertsMode, const ExpertsArgs&) { return "%s"; }
hipError_t launch_experts(int, ExpertsMode, const ExpertsArgs&, hipStream_t st) { return launched(st); }
hipError_t launch_combine(int, const CombineArgs&, hipStream_t st) { return launched(st); }
hipError_t launch_combine_backward(int, const CombineGradArgs&, hipStream_t st) { return launched(st); }
}  // namespace ns

// ------------------------------------------------------------- the calls

namespace {

char* at(int i) { return reinterpret_cast<char*>(0x10000000ll * (i + 1)); }  // far apart, 16-byte aligned

int call(int what, void* st) {
  int* const ids = reinterpret_cast<int*>(at(1));
  float* const f = reinterpret_cast<float*>(at(2));
  switch (what) {
    case 0:
      return ns_route(at(0), 64, nullptr, ids, f, ids + 65536, ids + 131072, ids + 262144, 5000, 64, 4, 1, 1, 2, 0, 1,
                      1.0f, 0, st);
    case 1:
      return ns_layer_norm_backward(at(0), 64, at(1), 64, at(3), f, f + 65536, at(4), at(5), at(6), 500, 64, 1, 0, st);
    case 2: return ns_orthogonalize(at(0), at(1), 2, 72, 100, 1, 3, 1, 1, 1, st);
    case 3: {
      const void* in[] = {at(0), at(1)};
      void* out[] = {at(2), at(1)};
      const int64_t batch[] = {1, 2}, rows[] = {64, 128}, cols[] = {128, 60};
      return ns_orthogonalize_grouped(2, in, out, batch, rows, cols, 1, 3, 1, 1, 1, st);
    }
    default: return ns_stage_normalize(at(0), at(1), nullptr, 2, 64, 128, 0, st);
  }
}
constexpr int kKinds = 5;

int run(int what, void* st) {
  t_call = ++g_calls;
  const int s = call(what, st);
  if (s != NS_OK) std::printf("call %d: status %d: %s\n", what, s, ns_last_error());
  return s;
}

}  // namespace

int main() {
  std::atomic<int> errors{0};
  for (int poison = 0; poison < 2; ++poison) {
    ns_set_workspace_poison(poison);
    std::vector<std::thread> threads;
    for (int t = 0; t < 4; ++t)
      threads.emplace_back([&, t] {
        for (int i = 0; i < 20; ++i) errors += run((i + t) % kKinds, (void*)(uintptr_t)(0x300 + i / 10)) != NS_OK;
      });
    for (auto& t : threads) t.join();
  }
  int mixed = 0;
  for (auto& stream : g_log) {
    std::set<int> ended;
    int last = 0;
    for (int c : stream.second) {
      if (c == last) continue;
      mixed += ended.count(c) != 0;
      if (last) ended.insert(last);
      last = c;
    }
  }
  std::printf("errors %d, calls whose launches another call's divide: %d\n", errors.load(), mixed);

  std::thread waits([&] { errors += run(0, kWaits) != NS_OK; });
  std::thread other([&] {
    errors += run(0, kOther) != NS_OK;
    std::lock_guard<std::mutex> lk(g_mu);
    g_other_done = true;
    g_cv.notify_all();
  });
  waits.join();
  other.join();
  std::printf("a stream that waited for another: %d\n", (int)g_waited_in_vain);
  return errors.load() != 0 || mixed != 0 || g_waited_in_vain;
}
