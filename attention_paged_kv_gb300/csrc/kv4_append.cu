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
// 2 bytes read and 0.5625 written an element (2 more where the values are
// wanted); the instructions come close to the bytes' time.  A thread takes a
// whole block of 16 values, so that the scale, its reciprocal and the row's
// address are found once a block (16000 tokens of 8 heads, 128 dims and
// values, 150 MB: 30 us, 74 % of the copy rate; with 8 values a thread 44.9).
#include <cstring>

#include "common.cuh"
#include "internal.h"
#include "kv4.h"

namespace pa {
namespace {

constexpr int kAppendThreads = 256;

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

// A CTA takes kAppendThreads / W tokens at a time (W blocks of 16 values make a
// token), or one token in several passes: which block is a thread's takes
// divisions once, not for every block.
template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads) kv4_append_kernel(const Kv4AppendParams p) {
  constexpr int TPR = D / 16;  // threads of a row
  pdl_wait();
  const int W = p.g.Hkv * TPR;
  const int tokens = W < kAppendThreads ? kAppendThreads / W : 1;
  const int mine = W < kAppendThreads ? static_cast<int>(threadIdx.x) / W : 0;
  const int piece0 = static_cast<int>(threadIdx.x) - mine * W;
  const int half = blockIdx.y;
  const T* rows = static_cast<const T*>(half ? p.v : p.k);
  const int64_t stride = half ? p.v_stride : p.k_stride;
  T* values = static_cast<T*>(half ? p.v_values : p.k_values);
  const float g = half ? p.v_scale : p.k_scale;
  const float g6 = 6.f * g, r6 = __frcp_rn(g6);
  const int64_t page_rows = static_cast<int64_t>(p.g.ps) * p.g.Hkv;
  const int64_t slots_end = static_cast<int64_t>(p.g.num_pages) << p.g.ps_shift;
  for (int tok0 = blockIdx.x * tokens; tok0 < p.n; tok0 += gridDim.x * tokens) {
    const int tok = tok0 + mine;
    int64_t slot = mine < tokens && tok < p.n ? p.slots[tok] : -1;
    if (slot >= slots_end) {
      atomicOr(p.status, PA_DEV_BAD_INDEX);
      slot = -1;
    }
    const int64_t row0 = ((slot >> p.g.ps_shift) * 2 + half) * page_rows +
                         static_cast<int64_t>(static_cast<int>(slot) & (p.g.ps - 1)) * p.g.slot_rows;
    for (int p0 = 0; p0 < W; p0 += kAppendThreads) {
      const int piece = p0 + piece0;
      if (slot < 0 || piece >= W) continue;
      const int h = piece / TPR, c = piece % TPR;
      const uint4* src = reinterpret_cast<const uint4*>(rows + tok * stride + static_cast<int64_t>(piece) * 16);
      const uint4 w0 = __ldg(src), w1 = __ldg(src + 1);
      const uint32_t ws[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
      // the largest magnitude by its 16 bits: a NaN is above every number
      uint32_t m2 = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) m2 = __vmaxu2(m2, ws[j] & 0x7FFF7FFFu);
      const uint32_t mb = max(m2 & 0xFFFFu, m2 >> 16);
      const bool nan = mb > (Elt<T>::kBf16 ? 0x7F80u : 0x7C00u);
      const float amax = Elt<T>::to_f2(mb).x;
      const uint32_t sb = nan ? 0x7Fu : e4m3(quotient(fminf(amax, 500.f * g6), g6, r6));
      const float s = e4m3_value(sb);
      const float per = __fmul_rn(s, g);  // value of code 1
      uint32_t codes[2] = {0, 0};
      if (per > 0.f) {  // false for a NaN scale as well
        const float r = __frcp_rn(per), most = 8.f * per;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 x = Elt<T>::to_f2(ws[j]);
          const float lo = quotient(fminf(fabsf(x.x), most), per, r);
          const float hi = quotient(fminf(fabsf(x.y), most), per, r);
          codes[j >> 2] |= e2m1x2(copysignf(lo, x.x), copysignf(hi, x.y)) << (8 * (j & 3));
        }
      }
      const int64_t row = row0 + static_cast<int64_t>(h) * p.g.head_rows;
      *reinterpret_cast<uint2*>(p.codes + row * (D / 2) + c * 8) = make_uint2(codes[0], codes[1]);
      p.scales[row * (D / 16) + c] = static_cast<uint8_t>(sb);
      if (values) {
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 q = e2m1x2_values((codes[j >> 2] >> (8 * (j & 3))) & 0xFFu);
          o[j] = Elt<T>::from_f2(__fmul_rn(q.x * s, g), __fmul_rn(q.y * s, g));  // code * s is exact
        }
        uint4* dst = reinterpret_cast<uint4*>(values + (static_cast<int64_t>(tok) * W + piece) * 16);
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
  }
}

template <typename T>
cudaError_t launch_t(const Kv4AppendParams& p, int D, int num_sms, cudaStream_t stream) {
  const int W = p.g.Hkv * (D / 16);
  const int tokens = W < kAppendThreads ? kAppendThreads / W : 1;
  const int64_t blocks = (int64_t(p.n) + tokens - 1) / tokens, most = int64_t(num_sms) * 16;
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
