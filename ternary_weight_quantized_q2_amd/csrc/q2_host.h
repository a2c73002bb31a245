// q2_host.h - argument checks, the error detail and the device check shared by
// the host files of the C ABI.
#pragma once
#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "q2.h"

namespace q2host {

inline thread_local char g_detail[320];

inline int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_detail, sizeof g_detail, fmt, ap);
  va_end(ap);
  return code;
}

inline int ok() {
  g_detail[0] = '\0';
  return Q2_OK;
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// pointer must be non-NULL when the buffer is non-empty, and aligned
inline int check_ptr(const void* p, bool nonempty, size_t align, const char* name) {
  if (nonempty && p == nullptr) return fail(Q2_ERR_ARG, "%s is NULL for a non-empty buffer", name);
  if (p != nullptr && !aligned(p, align)) return fail(Q2_ERR_ALIGN, "%s is not %zu-byte aligned", name, align);
  return Q2_OK;
}

// keep every element index inside int64 with room to spare
inline bool sizes_fit(int64_t M, int64_t N, int64_t K) {
  const int64_t lim = (int64_t)1 << 46;
  return M <= lim && N <= lim && K <= lim && (M <= 0 || (K <= lim / M && N <= lim / M)) && (N <= 0 || K <= lim / N);
}

inline int check_sizes(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0) return fail(Q2_ERR_ARG, "negative size (M=%lld N=%lld K=%lld)", (long long)M,
                                           (long long)N, (long long)K);
  if (K % 128 != 0) return fail(Q2_ERR_SHAPE, "K=%lld is not a multiple of 128", (long long)K);
  if (!sizes_fit(M, N, K)) return fail(Q2_ERR_ARG, "sizes too large");
  return Q2_OK;
}

// The linear kernels address one tile's activation rows and weight columns
// with 32-bit offsets; K up to 2^24 keeps them in range for every tile shape.
constexpr int64_t kMostK = (int64_t)1 << 24;
inline int check_linear_k(int64_t K) {
  if (K > kMostK) return fail(Q2_ERR_SHAPE, "K=%lld exceeds 16777216", (long long)K);
  return Q2_OK;
}

inline std::atomic<int> g_arch_ok[64];

inline int check_device() {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail(Q2_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(e));
  const int slot = (dev >= 0 && dev < 64) ? dev : -1;
  if (slot >= 0) {
    const int st = g_arch_ok[slot].load(std::memory_order_relaxed);
    if (st == 1) return Q2_OK;
    if (st == -1) return fail(Q2_ERR_DEVICE, "device %d is not gfx950", dev);
  }
  hipDeviceProp_t prop;
  e = hipGetDeviceProperties(&prop, dev);
  if (e != hipSuccess) return fail(Q2_ERR_HIP, "hipGetDeviceProperties: %s", hipGetErrorString(e));
  const bool good = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
  if (slot >= 0) g_arch_ok[slot].store(good ? 1 : -1, std::memory_order_relaxed);
  if (!good) return fail(Q2_ERR_DEVICE, "device %d is %s, not gfx950", dev, prop.gcnArchName);
  return Q2_OK;
}

inline int hip_status(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(Q2_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

}  // namespace q2host
