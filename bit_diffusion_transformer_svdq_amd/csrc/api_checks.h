// Argument checks shared by the C ABI's entry points (api.cpp, block_api.cpp, fp8_api.cpp).
// Host only.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdarg>
#include <cstddef>
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "svdq.h"

// the thread's error message (api.cpp)
svdq_status svdq_internal_fail(svdq_status s, const char* msg);
svdq_status svdq_internal_ok();

namespace svdq_api {

inline svdq_status fail(svdq_status s, const char* fmt, ...) {
  char msg[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return svdq_internal_fail(s, msg);
}

inline svdq_status ok() { return svdq_internal_ok(); }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline svdq_status check_current_device() {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e == hipSuccess) return svdq_check_device(dev);  // cached per device
  (void)hipGetLastError();
  int count = 0;
  if (hipGetDeviceCount(&count) != hipSuccess || count <= 0) {
    (void)hipGetLastError();
    return fail(SVDQ_STATUS_NO_DEVICE, "no HIP device visible");
  }
  return fail(SVDQ_STATUS_HIP_ERROR, "hipGetDevice: %s", hipGetErrorString(e));
}

// A device byte range an entry point reads or writes.  Inputs may share memory
// with each other; an output may share memory with nothing else the call
// touches (the kernels read inputs while other workgroups already write).
struct Span {
  const void* p;
  size_t n;
  const char* name;
};

inline bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.n && b0 < a0 + a.n;
}

inline svdq_status check_disjoint(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    for (auto i = ins.begin(); i != ins.end(); ++i)
      if (overlap(*o, *i)) return fail(SVDQ_STATUS_INVALID_VALUE, "output %s overlaps input %s", o->name, i->name);
    for (auto o2 = o + 1; o2 != outs.end(); ++o2)
      if (overlap(*o, *o2)) return fail(SVDQ_STATUS_INVALID_VALUE, "outputs %s and %s overlap", o->name, o2->name);
  }
  return SVDQ_STATUS_SUCCESS;
}

// A call that needs `need` bytes of workspace gets them from the caller.
inline svdq_status check_workspace(const void* ws, size_t ws_bytes, size_t need, const char* query) {
  if (need == 0) return SVDQ_STATUS_SUCCESS;
  if (!ws) return fail(SVDQ_STATUS_INVALID_VALUE, "this shape needs a workspace of %zu bytes (%s)", need, query);
  if (ws_bytes < need)
    return fail(SVDQ_STATUS_INVALID_VALUE, "workspace of %zu bytes, this shape needs %zu (%s)", ws_bytes, need, query);
  if (!aligned16(ws)) return fail(SVDQ_STATUS_INVALID_VALUE, "workspace must be 16-byte aligned");
  return SVDQ_STATUS_SUCCESS;
}

// rows of `width` bytes, `stride` bytes apart
struct Rows {
  const void* p;
  size_t stride, width, rows;
  const char* name;
};

inline size_t extent(const Rows& r) { return r.rows == 0 ? 0 : (r.rows - 1) * r.stride + r.width; }

// Whether two sets of rows may share a byte.  Rows of one stride can interleave
// (the Q and K columns of one projection's output): their places within a
// stride decide.
inline bool meet(const Rows& a, const Rows& b) {
  if (!a.p || !b.p) return false;
  if (!overlap({a.p, extent(a), a.name}, {b.p, extent(b), b.name})) return false;
  if (a.stride != b.stride || a.stride == 0) return true;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  const size_t d = (size_t)((b0 >= a0 ? (b0 - a0) % a.stride : a.stride - (a0 - b0) % a.stride) % a.stride);
  return d < a.width || d + b.width > a.stride;
}

inline svdq_status check_rows(const Rows& out, std::initializer_list<Rows> others) {
  for (const Rows& o : others)
    if (meet(out, o)) return fail(SVDQ_STATUS_INVALID_VALUE, "output %s overlaps %s", out.name, o.name);
  return SVDQ_STATUS_SUCCESS;
}

inline bool bad_ptr(const void* p) { return p && !aligned16(p); }

inline svdq_status launched(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(SVDQ_STATUS_HIP_ERROR, "%s launch: %s", what, hipGetErrorString(e));
  return ok();
}

constexpr int64_t kMaxRows = 1ll << 24;

inline size_t sz(int64_t a, int64_t b = 1, int64_t c = 1) { return (size_t)a * (size_t)b * (size_t)c; }

}  // namespace svdq_api
