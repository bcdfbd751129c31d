// api_util.cuh -- host helpers shared by the translation units of the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include <initializer_list>
#include <mutex>

#include "../../include/nvfp4.h"

namespace nvfp4 {

constexpr int kMaxDevices = 64;

// SMs of the current device, looked up once per device.
inline int sm_count() {
  static int sms[kMaxDevices];
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
  std::lock_guard<std::mutex> lk(mu);
  if (sms[dev] == 0) {
    int s = 0;
    cudaDeviceGetAttribute(&s, cudaDevAttrMultiProcessorCount, dev);
    sms[dev] = s > 0 ? s : 148;
  }
  return sms[dev];
}

// Product of sizes that must each be non-negative, or -1 when one is negative or the product does not
// fit in int64 (so that no later size arithmetic can wrap round and pass a check).
inline int64_t checked_prod(std::initializer_list<int64_t> v) {
  int64_t p = 1;
  for (int64_t a : v) {
    if (a < 0 || __builtin_mul_overflow(p, a, &p)) return -1;
  }
  return p;
}

inline cudaStream_t S(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool dtype_ok(int dt) { return dt == NVFP4_F32 || dt == NVFP4_BF16 || dt == NVFP4_F16; }
inline int esize(int dt) { return dt == NVFP4_F32 ? 4 : 2; }
inline int last_error() { return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }

}  // namespace nvfp4
