// api_util.h -- argument checks and the NVTX range shared by the C entry points.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "fa_internal.h"

namespace mfa {

constexpr size_t kAlign = 256;

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

inline int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// An activation/cache tensor: bf16 or fp16, rank, unit head-dim stride,
// other strides multiples of 8 elements (16 bytes), 16-byte aligned base.
inline int check_bf16(const fa_tensor* t, int ndim) {
  if (!t || !t->data) return FA_ERR_INVALID_ARG;
  if ((t->dtype != FA_DTYPE_BF16 && t->dtype != FA_DTYPE_F16) || t->ndim != ndim) return FA_ERR_INVALID_ARG;
  for (int i = 0; i < ndim; ++i)
    if (t->shape[i] < 0) return FA_ERR_INVALID_ARG;
  if (t->stride[ndim - 1] != 1) return FA_ERR_INVALID_ARG;
  for (int i = 0; i < ndim - 1; ++i)
    if (t->stride[i] < 0 || (t->stride[i] % 8) != 0) return FA_ERR_INVALID_ARG;
  if (!aligned16(t->data)) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

inline int check_i32_vec(const fa_tensor* t, int64_t len) {
  if (!t || !t->data || t->dtype != FA_DTYPE_I32 || t->ndim != 1) return FA_ERR_INVALID_ARG;
  if (t->shape[0] != len || t->stride[0] != 1) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// The device must be an sm_103 part (checked once per device).
inline int check_device() {
  static std::atomic<int> cached[64];  // 0 unknown, 1 ok, 2 bad
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_NO_DEVICE;
  if (dev < 0 || dev >= 64) return FA_ERR_NO_DEVICE;
  int c = cached[dev].load(std::memory_order_relaxed);
  if (c == 0) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
      cudaGetLastError();
      return FA_ERR_NO_DEVICE;
    }
    c = (major == 10 && minor == 3) ? 1 : 2;
    cached[dev].store(c, std::memory_order_relaxed);
  }
  return c == 1 ? FA_OK : FA_ERR_NO_DEVICE;
}

// SMs of the current device (152 on GB300, which a plan without a device assumes).
inline int sm_count() {
  static std::atomic<int> cached[64];
  int dev = 0, v = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return 152;
  }
  const int n = cached[dev].load(std::memory_order_relaxed);
  if (n > 0) return n;
  if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0) {
    cudaGetLastError();
    return 152;
  }
  cached[dev].store(v, std::memory_order_relaxed);
  return v;
}

// NVTX range around the host-side enqueue of one stage (a profiler's trace
// shows it beside the stage's kernels); none while g_trace_ranges is off.
struct TraceRange {
  bool on;
  explicit TraceRange(const char* name) : on(mfa::g_trace_ranges) {
    if (on) nvtxRangePushA(name);
  }
  ~TraceRange() {
    if (on) nvtxRangePop();
  }
  TraceRange(const TraceRange&) = delete;
  TraceRange& operator=(const TraceRange&) = delete;
};

}  // namespace mfa
