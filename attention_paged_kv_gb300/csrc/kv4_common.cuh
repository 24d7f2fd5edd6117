// Device helpers that the 4-bit kernels share: the batch as they read it, and
// the conversions of codes and scales.
#pragma once

#include <climits>

#include "common.cuh"
#include "kv4.h"

namespace pa {

// ---------------------------------------------------------------------------
// the batch

struct Req {
  int qo_start, qo_len, page_start, kv_len;
};

// Request b, checked: one whose entries cannot be is empty (its rows are not
// written) and raises PA_DEV_BAD_INDEX.
__device__ __forceinline__ Req load_req(const Kv4Params& p, int b) {
  const int q0 = p.qo_indptr[b], q1 = p.qo_indptr[b + 1];
  const int p0 = p.page_indptr[b], p1 = p.page_indptr[b + 1];
  const int last = p.last_page_len[b];
  const long long kv = p1 > p0 ? static_cast<long long>(p1 - p0 - 1) * p.g.ps + last : 0;
  const bool ok = q0 >= 0 && q1 >= q0 && q1 <= p.num_tokens && p0 >= 0 && p1 >= p0 && p1 <= p.num_page_indices &&
                  (p1 == p0 || (last >= 1 && last <= p.g.ps)) && kv <= INT_MAX - 256;
  if (!ok) {
    atomicOr(p.status, PA_DEV_BAD_INDEX);
    return Req{0, 0, 0, 0};
  }
  return Req{q0, q1 - q0, p0, static_cast<int>(kv)};
}

// ---------------------------------------------------------------------------
// codes and scales

// The 8 codes of a word as four (even, odd) fp16 pairs.
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// The e4m3 values of the low two bytes (the upper two are ignored).
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t two) {
  uint32_t h;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(two));
  return h;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
  const __half2 r = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The power of two (as its exponent) that brings a bf16 row whose largest
// magnitude has the bits `top` to [2^13, 2^14), where fp16 holds it; 0 for
// rows of zeros, subnormals, infinities or NaN.
__device__ __forceinline__ int bf16_row_shift(uint32_t top) {
  const int e = static_cast<int>(top >> 7);
  return (e == 0 || e == 255) ? 0 : min(140 - e, 126);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

}  // namespace pa
