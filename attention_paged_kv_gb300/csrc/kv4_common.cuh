// Device helpers that the 4-bit kernels share: the batch as they read it, and
// the conversions of codes and scales.
#pragma once

#include <cfloat>
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

// Three-input maximum (one instruction).
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// base + a * b in one instruction.
__device__ __forceinline__ const uint8_t* offset_by(const uint8_t* base, uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mad.wide.u32 %0, %1, %2, %3;" : "=l"(r) : "r"(a), "r"(b), "l"(reinterpret_cast<uint64_t>(base)));
  return reinterpret_cast<const uint8_t*>(r);
}

// The power of two (as its exponent) that brings a bf16 row whose largest
// magnitude has the bits `top` to [2^13, 2^14), where fp16 holds it; 0 for
// rows of zeros, subnormals, infinities or NaN.
__device__ __forceinline__ int bf16_row_shift(uint32_t top) {
  const int e = static_cast<int>(top >> 7);
  return (e == 0 || e == 255) ? 0 : min(140 - e, 126);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// The factor from a row's scores (of q * 2^up) to its logits, kept a normal
// number: a score is 0, or of a size in [2^-34, 2^34], or -inf where its key is
// masked.  Below fp32's range the factor would be 0, and 0 * -inf a NaN; the
// logits are below 2^-92 either way.  Above, it would be infinite, and a NaN
// for scores of 0; the logits of other scores pass 2^93 either way, and the
// largest alone counts (or passes fp32's range).
__device__ __forceinline__ float row_factor(float scale_log2, float down) {  // down = 2^-up
  return fminf(fmaxf(scale_log2 * down, FLT_MIN), FLT_MAX);
}

// n / G and n % G for n < 512 (G <= 128): G's reciprocal in 16 bits, rounded up
// (its error, below G / 2^16 a unit, stays below one for such n).
struct DivG {
  int G;
  uint32_t m;
  __device__ explicit DivG(int g) : G(g), m((65535u + g) / g) {}
  __device__ __forceinline__ int div(int n) const { return static_cast<int>((static_cast<uint32_t>(n) * m) >> 16); }
};

// ---------------------------------------------------------------------------
// softmax weights

// P is 2^(logit - m) with the reference m this far (in log2 units) below the
// largest logit when it is set; it is set again when a logit passes it by
// kPMost, so a row's largest P lies in [2^7, 2^15] and fp16 rounds P to 2^-11
// of it down to 2^-14: 2^-21 of the row's largest weight or above.  Smaller
// ones are off by at most 2^-25, or 2^-32 of the largest (with m the largest
// logit itself, keys below 2^-25 of it were lost: a row with one dominant key
// lost all others).
constexpr float kPHead = 7.f, kPMost = 15.f;

// ---------------------------------------------------------------------------
// partial states

// Joins `parts` states of `rows` rows: o = sum_k 2^(lse_k - lse) o_k, in the
// parts' order, by `threads` threads of which this one is `rank`.  Part k's
// rows begin at part_row(k) of part_o / part_lse; out_row(n) is row n of out.
// A thread has K parts of U columns in flight at a time: one by one, each
// would wait for two dependent loads.
template <typename T, int D, int U, int K, typename PartRow, typename OutRow>
__device__ __forceinline__ void join_parts(const Kv4Params& p, int rank, int threads, int rows, int parts,
                                           PartRow part_row, OutRow out_row) {
  constexpr int COLS = D / 4;  // float4 columns of a row
  const int n_items = rows * COLS;
  for (int i0 = rank; i0 < n_items; i0 += U * threads) {
    int at[U];  // row * COLS + column, the last one again past the end
    float top[U], sum[U];
    float4 acc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      at[u] = min(i0 + u * threads, n_items - 1);
      top[u] = -3.0e38f;
      sum[u] = 0.f;
      acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll K
    for (int k = 0; k < parts; ++k) {
      const float* lse = p.part_lse + part_row(k);
#pragma unroll
      for (int u = 0; u < U; ++u) top[u] = fmaxf(top[u], __ldcg(lse + at[u] / COLS));
    }
#pragma unroll K
    for (int k = 0; k < parts; ++k) {
      const int64_t row = part_row(k);
      float4 v[U];
      float a[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        v[u] = __ldcg(reinterpret_cast<const float4*>(p.part_o + row * D) + at[u]);
        a[u] = __ldcg(p.part_lse + row + at[u] / COLS);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float w;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(a[u] - top[u]));
        sum[u] += w;
        acc[u].x += w * v[u].x;
        acc[u].y += w * v[u].y;
        acc[u].z += w * v[u].z;
        acc[u].w += w * v[u].w;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u * threads >= n_items) break;
      const int col = at[u] % COLS;
      // a row that sees no key: zeros, and -inf as its lse
      const float inv = sum[u] == 0.f ? 0.f : p.v_scale / sum[u];
      const int64_t row = out_row(at[u] / COLS);
      *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + row * D + col * 4) =
          make_uint2(Elt<T>::from_f2(acc[u].x * inv, acc[u].y * inv), Elt<T>::from_f2(acc[u].z * inv, acc[u].w * inv));
      if (col == 0 && p.lse)
        p.lse[row] = sum[u] == 0.f ? -INFINITY : (top[u] + log2f(sum[u])) * 0.6931471805599453f;
    }
  }
}

}  // namespace pa
