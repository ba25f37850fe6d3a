// api_common.hpp -- what every entry point of the C ABI shares: the
// thread-local failure text, descriptor views and their checks, and the
// device check.  Host only.
#pragma once
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>

#include "../../include/sl.h"

namespace sl {
namespace host {

// the text of the calling thread's last failure
inline thread_local std::string g_msg;

inline sl_status fail(sl_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline sl_status fail(sl_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_msg = buf;
  return s;
}

inline int elem_size(int32_t dt) {
  switch (dt) {
    case SL_F16: return 2;
    case SL_BF16: return 2;
    case SL_F32: return 4;
    case SL_F8_E4M3: return 1;
    case SL_E8M0: return 1;
    case SL_F4_E2M1: return 1;  // two elements per byte: byte_range halves the span
    case SL_F6_E2M3:
    case SL_F6_E3M2: return 1;  // four elements per three bytes: byte_range scales the span
    default: return 0;
  }
}

// A matrix view (batch stride, row stride, column stride) of a descriptor.
struct View {
  const sl_tensor* t;
  int64_t batch;  // 1 for rank 2
  int64_t rows, cols;
  int64_t bs, rs, cs;
  bool present;
};

inline sl_status make_view(const char* name, const sl_tensor& t, View* v) {
  v->t = &t;
  v->present = true;
  const sl_layout& L = t.layout;
  if (L.rank != 2 && L.rank != 3) return fail(SL_ERR_LAYOUT, "%s: rank %d (expected 2 or 3)", name, L.rank);
  for (int i = 0; i < L.rank; ++i) {
    if (L.shape[i] < 0) return fail(SL_ERR_SHAPE, "%s: negative size %lld", name, (long long)L.shape[i]);
    if (L.stride[i] < 0) return fail(SL_ERR_LAYOUT, "%s: negative stride %lld", name, (long long)L.stride[i]);
  }
  if (L.rank == 3) {
    v->batch = L.shape[0];
    v->rows = L.shape[1];
    v->cols = L.shape[2];
    v->bs = L.stride[0];
    v->rs = L.stride[1];
    v->cs = L.stride[2];
  } else {
    v->batch = 1;
    v->rows = L.shape[0];
    v->cols = L.shape[1];
    v->bs = 0;
    v->rs = L.stride[0];
    v->cs = L.stride[1];
  }
  return SL_OK;
}

// [lo, hi) byte range a view can touch, for `batch` batches.
inline void byte_range(const View& v, int64_t batch, uintptr_t* lo, uintptr_t* hi) {
  const int es = elem_size(v.t->dtype);
  const int64_t nb = v.t->layout.rank == 3 ? batch : 1;
  int64_t last = 0;
  if (nb > 0 && v.rows > 0 && v.cols > 0) last = (nb - 1) * v.bs + (v.rows - 1) * v.rs + (v.cols - 1) * v.cs;
  *lo = (uintptr_t)v.t->data;
  if (v.t->dtype == SL_F4_E2M1)
    *hi = (uintptr_t)v.t->data + (uintptr_t)(last / 2 + 1);
  else if (v.t->dtype == SL_F6_E2M3 || v.t->dtype == SL_F6_E3M2)
    *hi = (uintptr_t)v.t->data + (uintptr_t)((6 * last + 5) / 8 + 1);
  else
    *hi = (uintptr_t)v.t->data + (uintptr_t)((last + 1) * es);
}

// Distinct (batch, row, col) must map to distinct addresses.
inline bool injective(const View& v, int64_t batch) {
  struct Dim {
    int64_t n, s;
  } d[3] = {{batch, v.bs}, {v.rows, v.rs}, {v.cols, v.cs}};
  Dim live[3];
  int k = 0;
  for (auto& x : d)
    if (x.n > 1) live[k++] = x;
  std::sort(live, live + k, [](const Dim& a, const Dim& b) { return a.s < b.s; });
  int64_t span = 0;  // largest offset reached by the faster dims
  for (int i = 0; i < k; ++i) {
    if (live[i].s <= span) return false;
    span += live[i].s * (live[i].n - 1);
  }
  return true;
}

inline bool same_layout(const sl_tensor& x, const sl_tensor& y) {
  if (x.layout.rank != y.layout.rank) return false;
  for (int i = 0; i < x.layout.rank; ++i)
    if (x.layout.shape[i] != y.layout.shape[i] || x.layout.stride[i] != y.layout.stride[i]) return false;
  return true;
}

// HIP's limit: a launch has fewer than 2^32 work items along its grid.  (In
// floating point: the product of three counts can pass 64 bits.)
inline bool grid_fits(int64_t batch, int64_t tiles_m, int64_t tiles_n, int32_t threads) {
  return (double)batch * (double)tiles_m * (double)tiles_n * (double)threads < 0x1p32;
}

// gfx950 check, cached per device
inline sl_status check_arch() {
  static std::mutex mu;
  static int known[64] = {0};  // 0 unknown, 1 ok, -1 not gfx950
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return fail(SL_ERR_LAUNCH, "hipGetDevice failed");
  if (dev < 0 || dev >= 64) return fail(SL_ERR_ARCH, "device index %d out of range", dev);
  std::lock_guard<std::mutex> g(mu);
  if (known[dev] == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return fail(SL_ERR_LAUNCH, "hipGetDeviceProperties failed");
    known[dev] = strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : -1;
  }
  if (known[dev] < 0) return fail(SL_ERR_ARCH, "device %d is not gfx950", dev);
  return SL_OK;
}

}  // namespace host
}  // namespace sl
