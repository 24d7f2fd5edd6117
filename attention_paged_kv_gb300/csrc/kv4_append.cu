// Appends the step's K and V rows to a 4-bit paged cache (pagedattn_kv4_append).
//
// Blocks of 16 values along head_dim share an e4m3 scale; with g the cache's
// fp32 scale of K or V, each step rounded once (to nearest, ties to even):
//   s    = e4m3(amax / (6 g)), at most 448        6 is the largest e2m1 value
//   code = e2m1(x / (s g)), beyond 6 to 6; 0 where s is 0
//   value read back = code * s * g
// The divisions are correctly rounded fp32 ones: a multiplication by a
// reciprocal would move values that lie on a border between two codes.  They
// share a block's divisor, so each is the reciprocal's product put right by one
// residual (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990): with r = 1/b correctly rounded and q = a r, the
// sum q + r (a - q b), in two fused steps, is a / b correctly rounded, as long
// as nothing over- or underflows.  It does neither here where it matters:
// quotients are clamped to 8 (codes end at 6), and where the residual
// underflows the quotient is far below the first border.  A block with a NaN
// gets the NaN scale, so that it reads back as NaN; an infinity saturates to
// the block's largest value.
//
// HBM-bound: 2 bytes read and 0.5625 written an element (2 more where the
// values are wanted).  A thread takes 8 values, one 16-byte load, and its
// neighbour the block's other half (one shuffle joins their maxima), so every
// access of a warp is to consecutive 16-byte (codes: 4-byte) pieces.
#include <cstring>

#include "common.cuh"
#include "internal.h"
#include "kv4.h"

namespace pa {
namespace {

constexpr int kAppendThreads = 256;

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Two e2m1 codes in a byte, the first value low.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 c;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %2, %1;\n\tmov.b32 %0, {c, 0, 0, 0};\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 e2m1x2_values(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 c, z1, z2, z3;\n\tmov.b32 {c, z1, z2, z3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}"
      : "=r"(h)
      : "r"(byte));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}
__device__ __forceinline__ uint32_t e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(x), "f"(0.f));
  return r & 0xFFu;
}
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(byte)));
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
}

// a / b for a >= 0, given r = 1 / b rounded to nearest.
__device__ __forceinline__ float quotient(float a, float b, float r) {
  const float q = __fmul_rn(a, r);
  return __fmaf_rn(__fmaf_rn(-q, b, a), r, q);
}

template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads) kv4_append_kernel(const Kv4AppendParams p) {
  constexpr int TPR = D / 8;  // threads of a row
  pdl_wait();
  const int64_t pieces = static_cast<int64_t>(p.n) * p.g.Hkv * TPR;
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kAppendThreads; i0 < pieces;
       i0 += static_cast<int64_t>(gridDim.x) * kAppendThreads) {
    const int64_t i = i0 + threadIdx.x;  // TPR is even and pieces a multiple of it: a block's two threads go together
    const bool in = i < pieces;
    const int c = static_cast<int>(i % TPR);
    const int64_t th = i / TPR;
    const int h = static_cast<int>(th % p.g.Hkv);
    const int tok = static_cast<int>(th / p.g.Hkv);
    const int half = blockIdx.y;
    int64_t slot = in ? p.slots[tok] : -1;
    if (slot >= static_cast<int64_t>(p.g.num_pages) << p.g.ps_shift) {
      atomicOr(p.status, PA_DEV_BAD_INDEX);
      slot = -1;
    }
    const bool live = slot >= 0;
    const T* src = static_cast<const T*>(half ? p.v : p.k) + tok * (half ? p.v_stride : p.k_stride) +
                   static_cast<int64_t>(h) * D + c * 8;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (live) w = *reinterpret_cast<const uint4*>(src);
    float x[8];
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = Elt<T>::to_f2(ws[j]);
      x[2 * j] = f.x;
      x[2 * j + 1] = f.y;
    }
    // the largest magnitude, as bits: a NaN is above every number
    uint32_t mb = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) mb = max(mb, abs_bits(x[j]));
    mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
    const float g = half ? p.v_scale : p.k_scale;
    const bool nan = mb > 0x7F800000u;
    // (an infinite or NaN maximum would make the residual NaN)
    const float amax = fminf(__uint_as_float(mb), 3.0e38f);
    const uint32_t sb = nan ? 0x7Fu : e4m3(__fdiv_rn(amax, 6.f * g));
    const float per = __fmul_rn(e4m3_value(sb), g);  // value of code 1
    uint32_t codes = 0;
    if (per > 0.f) {  // false for a NaN scale as well
      const float r = __frcp_rn(per), most = 8.f * per;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float lo = quotient(fminf(fabsf(x[2 * j]), most), per, r);
        const float hi = quotient(fminf(fabsf(x[2 * j + 1]), most), per, r);
        codes |= e2m1x2(copysignf(lo, x[2 * j]), copysignf(hi, x[2 * j + 1])) << (8 * j);
      }
    }
    if (!live) continue;
    const int64_t page = slot >> p.g.ps_shift;
    const int at = static_cast<int>(slot) & (p.g.ps - 1);
    const int64_t row = (page * 2 + half) * (static_cast<int64_t>(p.g.ps) * p.g.Hkv) +
                        static_cast<int64_t>(at) * p.g.slot_rows + static_cast<int64_t>(h) * p.g.head_rows;
    *reinterpret_cast<uint32_t*>(p.codes + row * (D / 2) + c * 4) = codes;
    if (!(c & 1)) p.scales[row * (D / 16) + (c >> 1)] = static_cast<uint8_t>(sb);
    T* values = static_cast<T*>(half ? p.v_values : p.k_values);
    if (values) {
      uint32_t o[4];
      const float s = e4m3_value(sb);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 q = e2m1x2_values((codes >> (8 * j)) & 0xFFu);
        o[j] = Elt<T>::from_f2(__fmul_rn(q.x * s, g), __fmul_rn(q.y * s, g));  // code * s is exact
      }
      *reinterpret_cast<uint4*>(values + th * D + c * 8) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

template <typename T>
cudaError_t launch_t(const Kv4AppendParams& p, int D, int num_sms, cudaStream_t stream) {
  const int64_t pieces = static_cast<int64_t>(p.n) * p.g.Hkv * (D / 8);
  const int64_t blocks = (pieces + kAppendThreads - 1) / kAppendThreads, most = int64_t(num_sms) * 64;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(static_cast<unsigned>(blocks < most ? blocks : most), 2);
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  std::memset(attr, 0, sizeof(attr));
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
#ifndef PA_NO_PDL
  attr[0].val.programmaticStreamSerializationAllowed = 1;
#endif
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  switch (D) {
    case 64: return cudaLaunchKernelEx(&cfg, kv4_append_kernel<T, 64>, p);
    case 128: return cudaLaunchKernelEx(&cfg, kv4_append_kernel<T, 128>, p);
    default: return cudaLaunchKernelEx(&cfg, kv4_append_kernel<T, 256>, p);
  }
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendParams& p, int D, int dtype, int num_sms, cudaStream_t stream) {
  return dtype == PA_BF16 ? launch_t<__nv_bfloat16>(p, D, num_sms, stream) : launch_t<__half>(p, D, num_sms, stream);
}

}  // namespace pa
