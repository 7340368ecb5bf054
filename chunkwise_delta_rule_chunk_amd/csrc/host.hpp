// Host-side pieces shared by the translation units behind the C ABI: the
// error text, argument checks and the tracing hook around every launch.
#pragma once
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <vector>

#include "kernels.hpp"
#include "rewy.h"

#define REWY_API extern "C" __attribute__((visibility("default")))

namespace rewy {

// Records the thread's error text and returns `code`.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

constexpr size_t ALIGN = 256;
inline size_t up(size_t x) { return (x + ALIGN - 1) / ALIGN * ALIGN; }
inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline int hip_check(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(REWY_EHIP, "%s: %s", what, hipGetErrorString(e));
  return REWY_OK;
}

// ---- tracing: event pairs around every launch, per thread ------------------
struct TraceRec {
  const void* fn;  // host stub of the launched kernel
  hipStream_t s;
  hipEvent_t e0, e1;
};
struct Tracer {
  bool on = false;
  char only[64] = {0};  // empty: every launch
  std::vector<TraceRec> recs;
  std::vector<hipEvent_t> pool;
  size_t used = 0;
  hipEvent_t ev() {
    if (used == pool.size()) {
      hipEvent_t e;
      if (hipEventCreate(&e) != hipSuccess) return nullptr;
      pool.push_back(e);
    }
    return pool[used++];
  }
};
extern thread_local Tracer g_tr;

// `stage` is the kernel's template name, which rewy_trace_select matches
template <typename F>
hipError_t traced(const char* stage, hipStream_t s, F&& launch) {
  if (!g_tr.on || (g_tr.only[0] && strcmp(g_tr.only, stage) != 0)) return launch();
  TraceRec r{nullptr, s, g_tr.ev(), g_tr.ev()};
  if (r.e0) hipEventRecord(r.e0, s);
  last_kernel() = nullptr;
  const hipError_t e = launch();
  if (r.e1) hipEventRecord(r.e1, s);
  r.fn = last_kernel();
  if (r.e0 && r.e1 && r.fn) g_tr.recs.push_back(r);
  return e;
}

}  // namespace rewy
