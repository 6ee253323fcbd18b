// ns_host.cpp - what the host drivers of the entry points share, and the
// entry points that report on it (errors, workspace, timing).
#include "ns_host.h"

#include <cstdio>
#include <cstring>
#include <map>
#include <mutex>
#include <utility>
#include <vector>

#include "ns_kernels.h"

namespace ns {

thread_local std::string t_err;
thread_local std::string t_cfg;
thread_local Config t_lazy_cfg;
thread_local bool t_untimed = false;
std::atomic<int> g_poison{0};

int fail(int status, const std::string& msg) {
  t_err = msg;
  return status;
}

int check_hip(hipError_t e, const char* what) {
  if (e == hipSuccess) return NS_OK;
  return fail(NS_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
}

// ---------------------------------------------------------------- checks

int check_dtype(int dtype) {
  if (dtype != NS_DTYPE_F32 && dtype != NS_DTYPE_BF16)
    return fail(NS_ERR_DTYPE, "dtype must be 0 (fp32) or 1 (bf16), got " + std::to_string(dtype));
  return NS_OK;
}

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const char* pa = static_cast<const char*>(a);
  const char* pb = static_cast<const char*>(b);
  return pa < pb + nb && pb < pa + na;
}

int check_ptr(const void* p, const char* name) {
  if (p == nullptr) return fail(NS_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (reinterpret_cast<uintptr_t>(p) % 16 != 0)
    return fail(NS_ERR_ALIGNMENT, std::string(name) + " is not 16-byte aligned");
  return NS_OK;
}

namespace {
std::mutex g_arch_mu;
std::map<int, int> g_arch;  // device -> NS_OK or NS_ERR_ARCH
}  // namespace

int check_arch() {
  int dev = 0;
  if (int s = check_hip(hipGetDevice(&dev), "hipGetDevice")) return s;
  std::lock_guard<std::mutex> lk(g_arch_mu);
  auto it = g_arch.find(dev);
  if (it == g_arch.end()) {
    hipDeviceProp_t prop;
    if (int s = check_hip(hipGetDeviceProperties(&prop, dev), "hipGetDeviceProperties")) return s;
    const int ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? NS_OK : NS_ERR_ARCH;
    it = g_arch.emplace(dev, ok).first;
    if (ok != NS_OK) t_err = std::string("device is ") + prop.gcnArchName + ", this library is built for gfx950";
  }
  if (it->second != NS_OK) return fail(NS_ERR_ARCH, "current device is not gfx950");
  return NS_OK;
}

// ------------------------------------------------------------- workspace

namespace {
struct Ws {
  void* ptr = nullptr;
  size_t bytes = 0;
  std::mutex enqueueing;  // held from taking the buffer to the last launch that uses it
};
std::mutex g_ws_mu;  // the containers below (taken after an `enqueueing`, never before one)
std::map<std::pair<int, void*>, Ws> g_ws;
// Buffers replaced by a larger one.  Work queued earlier may still read
// them, so they are freed only by ns_release_workspace.
std::vector<std::pair<int, void*>> g_ws_retired;
std::atomic<int64_t> g_ws_allocs{0};
}  // namespace

int get_workspace(hipStream_t st, size_t bytes, Workspace* out) {
  int dev = 0;
  if (int s = check_hip(hipGetDevice(&dev), "hipGetDevice")) return s;
  Ws* found = nullptr;
  {
    std::lock_guard<std::mutex> lk(g_ws_mu);
    found = &g_ws[{dev, (void*)st}];  // (stays where it is until ns_release_workspace, which runs beside no call)
  }
  Ws& w = *found;
  std::unique_lock<std::mutex> held(w.enqueueing);
  if (w.bytes < bytes) {
    void* p = nullptr;
    if (hipMalloc(&p, bytes) != hipSuccess || p == nullptr) {
      (void)hipGetLastError();
      return fail(NS_ERR_OOM, "workspace allocation of " + std::to_string(bytes) + " bytes failed");
    }
    ++g_ws_allocs;
    if (w.ptr != nullptr) {
      std::lock_guard<std::mutex> lk(g_ws_mu);
      g_ws_retired.emplace_back(dev, w.ptr);
    }
    w.ptr = p;
    w.bytes = bytes;
  }
  out->ptr = static_cast<char*>(w.ptr);
  out->held = std::move(held);
  return NS_OK;
}

// ---------------------------------------------------------------- timing

namespace {
struct TimingRec {
  int kind;
  hipEvent_t a, b;
};
std::mutex g_t_mu;
int g_t_mask = 0;
int g_t_every = 1, g_t_offset = 0;     // launch i of a kind is timed when i % every == offset
int64_t g_t_count[NS_KIND_COUNT] = {};  // launches of each kind since the last reset
std::vector<TimingRec> g_t_recs;
std::vector<hipEvent_t> g_t_pool;

hipEvent_t take_event() {
  if (!g_t_pool.empty()) {
    hipEvent_t e = g_t_pool.back();
    g_t_pool.pop_back();
    return e;
  }
  // Timing-only events: no system-scope fence when recorded.  With the
  // default flags every record writes back and invalidates the caches, which
  // costs the timed kernels time of their own and slows the kernel after
  // them.  Their timestamps are only read after the stream has been
  // synchronised (ns_timing_query).
  hipEvent_t e = nullptr;
  if (hipEventCreateWithFlags(&e, hipEventDisableSystemFence) != hipSuccess) return nullptr;
  return e;
}
}  // namespace

LaunchTimer::LaunchTimer(int k) : kind(k) {
  std::lock_guard<std::mutex> lk(g_t_mu);
  on = ((g_t_mask >> kind) & 1) && g_t_count[kind]++ % g_t_every == g_t_offset;
  if (!on) return;
  a = take_event();
  b = take_event();
  if (a && b) set_launch_events(a, b);
}

void LaunchTimer::done(hipError_t e) {
  if (!on) return;
  set_launch_events(nullptr, nullptr);
  std::lock_guard<std::mutex> lk(g_t_mu);
  if (a && b && e == hipSuccess) {
    g_t_recs.push_back(TimingRec{kind, a, b});
  } else {  // nothing recorded them: back to the pool
    if (a) g_t_pool.push_back(a);
    if (b) g_t_pool.push_back(b);
  }
}

}  // namespace ns

// =================================================================== C ABI

using namespace ns;

extern "C" {

int ns_release_workspace(void) {
  t_err.clear();
  std::lock_guard<std::mutex> lk(g_ws_mu);
  int status = NS_OK;
  int cur = 0;
  (void)hipGetDevice(&cur);
  std::vector<std::pair<int, void*>> bufs = g_ws_retired;
  for (auto& kv : g_ws)
    if (kv.second.ptr != nullptr) bufs.emplace_back(kv.first.first, kv.second.ptr);
  std::map<int, bool> synced;
  for (auto& db : bufs) {
    if (hipSetDevice(db.first) != hipSuccess) {
      status = fail(NS_ERR_HIP, "hipSetDevice failed");
      continue;
    }
    if (!synced[db.first]) {
      (void)hipDeviceSynchronize();
      synced[db.first] = true;
    }
    if (hipFree(db.second) != hipSuccess) status = fail(NS_ERR_HIP, "hipFree failed");
  }
  g_ws.clear();
  g_ws_retired.clear();
  (void)hipSetDevice(cur);
  return status;
}

int64_t ns_workspace_allocations(void) { return g_ws_allocs.load(); }

const char* ns_status_string(int status) {
  switch (status) {
    case NS_OK: return "NS_OK";
    case NS_ERR_INVALID_ARG: return "NS_ERR_INVALID_ARG: invalid argument";
    case NS_ERR_DTYPE: return "NS_ERR_DTYPE: unsupported dtype";
    case NS_ERR_ALIGNMENT: return "NS_ERR_ALIGNMENT: pointers must be 16-byte aligned (stage exports: dims multiples of 8)";
    case NS_ERR_ARCH: return "NS_ERR_ARCH: device is not gfx950";
    case NS_ERR_OOM: return "NS_ERR_OOM: workspace allocation failed";
    case NS_ERR_HIP: return "NS_ERR_HIP: HIP runtime error";
    case NS_ERR_SCRATCH: return "NS_ERR_SCRATCH: the call needs more than the fixed no-alloc scratch";
    default: return "unknown status";
  }
}

const char* ns_last_error(void) { return t_err.c_str(); }

int ns_query_last_config(char* buf, size_t n) {
  if (t_lazy_cfg.fmt != nullptr) {
    const Config& c = t_lazy_cfg;
    char text[512];
    std::snprintf(text, sizeof(text), c.fmt, c.text, c.v[0], c.v[1], c.v[2], c.v[3], c.v[4], c.v[5], c.v[6], c.v[7]);
    t_cfg = text;
    t_lazy_cfg.fmt = nullptr;
  }
  if (buf != nullptr && n > 0) {
    std::strncpy(buf, t_cfg.c_str(), n - 1);
    buf[n - 1] = '\0';
  }
  return (int)t_cfg.size();
}

int ns_timing_enable(int mask) {
  std::lock_guard<std::mutex> lk(g_t_mu);
  g_t_mask = mask;
  return NS_OK;
}

int ns_timing_sample(int every, int offset) {
  t_err.clear();
  if (every < 1 || offset < 0 || offset >= every)
    return fail(NS_ERR_INVALID_ARG, "timing sample needs every >= 1 and 0 <= offset < every");
  std::lock_guard<std::mutex> lk(g_t_mu);
  g_t_every = every;
  g_t_offset = offset;
  return NS_OK;
}

int ns_timing_reset(void) {
  std::lock_guard<std::mutex> lk(g_t_mu);
  for (auto& c : g_t_count) c = 0;
  for (auto& r : g_t_recs) {
    g_t_pool.push_back(r.a);
    g_t_pool.push_back(r.b);
  }
  g_t_recs.clear();
  return NS_OK;
}

int ns_timing_query(int kind, double* total_ms, int64_t* launches) {
  t_err.clear();
  if (kind < 0 || kind >= NS_KIND_COUNT || total_ms == nullptr || launches == nullptr)
    return fail(NS_ERR_INVALID_ARG, "bad timing query");
  std::lock_guard<std::mutex> lk(g_t_mu);
  double sum = 0.0;
  int64_t count = 0;
  for (auto& r : g_t_recs) {
    if (r.kind != kind) continue;
    if (hipEventSynchronize(r.b) != hipSuccess) return fail(NS_ERR_HIP, "hipEventSynchronize failed");
    float ms = 0.0f;
    if (hipEventElapsedTime(&ms, r.a, r.b) != hipSuccess) return fail(NS_ERR_HIP, "hipEventElapsedTime failed");
    sum += ms;
    ++count;
  }
  *total_ms = sum;
  *launches = count;
  return NS_OK;
}

int ns_set_workspace_poison(int on) {
  g_poison.store(on != 0);
  return NS_OK;
}

}  // extern "C"
