// lq_plan.h — launch plans: while a host thread has a PlanRecorder installed,
// every launch wrapper appends the name of the kernel it would launch and the
// grid and block sizes, instead of launching. lq_call_kernels and
// lq_linear_kernels report the kernels of a call from the dispatch code itself
// with it.
#pragma once
#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

namespace lqd {

struct PlanRecorder {
  char* buf;      // may be null (count only)
  size_t cap;     // bytes at buf
  size_t len;     // bytes written, without the terminating NUL
  int count;      // kernels recorded
};
extern thread_local PlanRecorder* g_plan;

__attribute__((format(printf, 3, 4))) inline hipError_t plan_add(int64_t nwg, int nthreads, const char* fmt, ...) {
  PlanRecorder* r = g_plan;
  char line[256];
  va_list ap;
  va_start(ap, fmt);
  int n = vsnprintf(line, sizeof line, fmt, ap);
  va_end(ap);
  if (n < 0) n = 0;
  char grid[48];
  const int g = snprintf(grid, sizeof grid, "\t%lld\t%d\n", (long long)nwg, nthreads);
  if (r->buf && r->len + (size_t)n + (size_t)g < r->cap) {
    memcpy(r->buf + r->len, line, (size_t)n);
    memcpy(r->buf + r->len + n, grid, (size_t)g);
    r->len += (size_t)n + (size_t)g;
    r->buf[r->len] = '\0';
  }
  r->count++;
  return hipSuccess;
}
inline const char* tf(bool b) { return b ? "true" : "false"; }

// Installs a recorder on this thread for the lifetime of the object.
struct PlanScope {
  PlanRecorder rec;
  PlanScope(char* buf, size_t bytes) {
    rec.buf = (buf && bytes) ? buf : nullptr;
    rec.cap = bytes;
    rec.len = 0;
    rec.count = 0;
    if (rec.buf) rec.buf[0] = '\0';
    g_plan = &rec;
  }
  ~PlanScope() { g_plan = nullptr; }
};

}  // namespace lqd
