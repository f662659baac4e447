// Host helpers shared by the C ABI's translation units: the thread's last
// error, alignment checks and the optional per-kernel event timing.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <map>
#include <mutex>
#include <string>
#include <utility>
#include <vector>

#include "moe_w4a16.h"

namespace moe {

// --------------------------------------------------------------------------
// Errors
// --------------------------------------------------------------------------

inline thread_local std::string g_err;

inline moe_status_t fail(moe_status_t st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_err = buf;
  return st;
}

inline moe_status_t ok() {
  g_err.clear();
  return MOE_OK;
}

inline moe_status_t hip_fail(hipError_t e, const char* what) {
  return fail(MOE_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// --------------------------------------------------------------------------
// Kernel timing
// --------------------------------------------------------------------------

struct Profiler {
  std::mutex mu;
  bool on = false;
  struct Pending {
    const char* name;
    hipEvent_t a, b;
  };
  std::vector<Pending> pending;
  std::vector<hipEvent_t> pool;
  std::map<std::string, std::pair<long, double>> totals;

  hipEvent_t get() {
    if (!pool.empty()) {
      hipEvent_t e = pool.back();
      pool.pop_back();
      return e;
    }
    hipEvent_t e = nullptr;
    // timing only: without the system-scope fence, recording an event
    // neither writes back nor invalidates the caches, which would change
    // the speed of the launch that follows it
    if (hipEventCreateWithFlags(&e, hipEventDisableSystemFence) != hipSuccess) return nullptr;
    return e;
  }
  void drain() {   // caller holds mu
    for (auto& p : pending) {
      float ms = 0.f;
      (void)hipEventSynchronize(p.b);
      (void)hipEventElapsedTime(&ms, p.a, p.b);
      auto& t = totals[p.name];
      t.first += 1;
      t.second += ms;
      pool.push_back(p.a);
      pool.push_back(p.b);
    }
    pending.clear();
  }
};

inline Profiler& prof() {
  static Profiler* p = new Profiler();   // never destroyed: events outlive static teardown
  return *p;
}

template <class F>
hipError_t run(const char* name, hipStream_t s, F&& f) {
  Profiler& P = prof();
  bool on;
  {
    std::lock_guard<std::mutex> g(P.mu);
    on = P.on;
  }
  if (!on) return f();
  hipEvent_t a, b;
  {
    std::lock_guard<std::mutex> g(P.mu);
    if (P.pending.size() > 4096) P.drain();
    a = P.get();
    b = P.get();
  }
  if (a) (void)hipEventRecord(a, s);
  hipError_t e = f();
  if (b) (void)hipEventRecord(b, s);
  if (a && b) {
    std::lock_guard<std::mutex> g(P.mu);
    P.pending.push_back({name, a, b});
  }
  return e;
}

}  // namespace moe
