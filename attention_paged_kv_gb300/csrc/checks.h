// Argument checks that the C entry points over device tables share.
#pragma once

#include <atomic>
#include <cstdint>

#include "internal.h"

namespace pa {

inline bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// log2 of a page size, or -1 where it is none
inline int page_shift(int32_t ps) {
  for (int s = 0; s <= 7; ++s)
    if (ps == (1 << s)) return s;
  return -1;
}

// SMs of the current device (asked once per device).
inline pagedattn_status device_sms(int* sms) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_err(e, "cudaGetDevice");
  int n = dev >= 0 && dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_err(e, "cudaDeviceGetAttribute");
    if (dev >= 0 && dev < 64) known[dev].store(n, std::memory_order_relaxed);
  }
  *sms = n;
  return PA_OK;
}

inline pagedattn_status check_heads(int32_t Hq, int32_t Hkv, int32_t D) {
  if (Hkv < 1 || Hq < 1 || Hq % Hkv)
    return set_err(PA_ERR_INVALID_ARG, "num_qo_heads must be a positive multiple of num_kv_heads");
  if (Hq / Hkv > 128 || Hq > 65535) return set_err(PA_ERR_UNSUPPORTED, "more than 128 query heads a kv head");
  if (D != 64 && D != 128 && D != 256) return set_err(PA_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256");
  return PA_OK;
}

inline pagedattn_status check_dtype(pagedattn_dtype d) {
  if (d != PA_FP16 && d != PA_BF16) return set_err(PA_ERR_UNSUPPORTED, "dtype must be PA_FP16 or PA_BF16");
  return PA_OK;
}

}  // namespace pa
