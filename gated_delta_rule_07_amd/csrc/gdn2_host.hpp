// gdn2_host.hpp -- what the C-ABI files share on the host: the last error's
// text, pointer checks, and the timing of launches.
#pragma once

#include "../../include/gdn2.h"

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <mutex>
#include <string>
#include <utility>
#include <vector>

// hidden: every library built from these files has its own state
namespace gdn2 __attribute__((visibility("hidden"))) {
namespace host {

inline thread_local std::string g_last_error;

inline gdn2_status_t fail(gdn2_status_t st, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return st;
}

inline gdn2_status_t ok() {
  g_last_error.clear();
  return GDN2_OK;
}


inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// ------------------------------------------------------------- profiling --
// Kernel names are string literals of the library, so the pointers handed out
// by gdn2_profile_read stay valid for the life of the library.
struct prof_rec {
  const char *name;
  hipEvent_t start, stop;
};
inline std::mutex g_prof_mu;
inline bool g_prof_on = false;
inline std::vector<prof_rec> g_prof_pending;
inline std::vector<std::pair<const char *, std::pair<double, int>>> g_prof_total;

struct prof_scope {
  hipStream_t st;
  bool on;
  prof_rec rec;
  prof_scope(const char *name, hipStream_t s) : st(s), on(false) {
    std::lock_guard<std::mutex> lk(g_prof_mu);
    if (!g_prof_on)
      return;
    // no system-scope fence: a fenced event would write back the L2 between
    // the two passes and slow down the very launches being timed
    if (hipEventCreateWithFlags(&rec.start, hipEventDisableSystemFence) != hipSuccess)
      return;
    if (hipEventCreateWithFlags(&rec.stop, hipEventDisableSystemFence) != hipSuccess) {
      (void)hipEventDestroy(rec.start);
      return;
    }
    rec.name = name;
    on = hipEventRecord(rec.start, st) == hipSuccess;
    if (!on) {
      (void)hipEventDestroy(rec.start);
      (void)hipEventDestroy(rec.stop);
    }
  }
  ~prof_scope() {
    if (!on)
      return;
    (void)hipEventRecord(rec.stop, st);
    std::lock_guard<std::mutex> lk(g_prof_mu);
    g_prof_pending.push_back(rec);
  }
};

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace host
}  // namespace gdn2
