// ns_host.h - what the host drivers of the entry points share: the thread's
// error and configuration texts, argument checks, the workspace of a (device,
// stream) and the timed launch.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>
#include <exception>
#include <mutex>
#include <new>
#include <string>

#include "../../include/ns_hip.h"

namespace ns {

extern thread_local std::string t_err;  // ns_last_error
extern thread_local std::string t_cfg;  // ns_query_last_config
// Set while the allocation-free entry point enqueues: its launches are
// neither timed nor counted (timing may create events).
extern thread_local bool t_untimed;
extern std::atomic<int> g_poison;       // ns_set_workspace_poison

// The same as a format of one text and up to eight numbers, filled in only
// when ns_query_last_config asks (it counts beside a short launch).
struct Config {
  const char* fmt = nullptr;
  const char* text = "";
  long long v[8] = {};
};
extern thread_local Config t_lazy_cfg;  // fmt null: t_cfg holds the text
template <typename... A>
void set_config(const char* fmt, const char* text, A... v) {
  static_assert(sizeof...(v) <= 8, "at most eight numbers");
  t_lazy_cfg = Config{fmt, text, {(long long)v...}};
}

int fail(int status, const std::string& msg);
int check_hip(hipError_t e, const char* what);
int check_dtype(int dtype);
int check_ptr(const void* p, const char* name);  // not null, 16-byte aligned
int check_arch();
bool overlaps(const void* a, size_t na, const void* b, size_t nb);

// The workspace of (current device, st), grown to at least `bytes`.  A warm
// workspace is returned without any HIP call, so calls on a stream that has
// seen a call of the same or a larger size enqueue only kernels and copies
// (graph capture needs exactly that).  It is the calling thread's own while
// `held` lives: an entry point keeps it until the last launch that uses the
// workspace is enqueued, so that calls of several threads on one stream are
// ordered by that stream as a whole, not launch by launch.
struct Workspace {
  char* ptr = nullptr;
  std::unique_lock<std::mutex> held;
};
int get_workspace(hipStream_t st, size_t bytes, Workspace* out);

// Timing of one launch of a kind: events that travel in the kernel's dispatch
// packet (set_launch_events), so timing adds no packets between the kernels
// of a call.
struct LaunchTimer {
  int kind;
  bool on = false;
  hipEvent_t a = nullptr, b = nullptr;
  explicit LaunchTimer(int kind);
  void done(hipError_t e);
};
template <typename F>
hipError_t timed_launch(int kind, hipStream_t, F&& f) {
  if (t_untimed) return f();
  LaunchTimer t(kind);
  const hipError_t e = f();
  t.done(e);
  return e;
}

// Runs the body of a C entry point: no C++ exception leaves it.
template <typename F>
int entry(F&& f) {
  try {
    t_err.clear();
    return f();
  } catch (const std::bad_alloc&) {
    return NS_ERR_OOM;
  } catch (const std::exception& e) {
    try {
      return fail(NS_ERR_HIP, e.what());
    } catch (...) {
      return NS_ERR_HIP;
    }
  }
}

}  // namespace ns
