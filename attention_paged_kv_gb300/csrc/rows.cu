// Rotary positions, rows appended to the 16-bit paged cache with the rotation
// on the way, and the bounds of a page's keys (pagedattn_rope,
// pagedattn_kv_append, pagedattn_kv_bounds).
//
// Rotation.  Pair (a, b) of a head at position x becomes
//   (a cos - b sin, b cos + a sin),  angle = 2 pi frac(x f)
// with f the pair's turns a position as a 64-bit fraction of a turn: x * f
// modulo 2^64 is exact in integers, so a position of 10^6 has as good an angle
// as one of 10, where a product in fp32 would be off by 0.1 rad; its top 32
// bits go to sincospi, in fp32 (off by 2^-26 turns).  Angles cost no table and no loads but the position.
//
// Bytes bound it (2 read and 2 written a value).  A thread takes 8 pairs of one
// token, two 16-byte pieces of a head, and goes through the heads of a group
// with the same 8 cosines and sines.  16000 tokens of 64 / 8 heads of 128 with V
// (656 MB): 102 us, 6.4 TB/s; 12001 tokens of 32 / 8 heads, three axes, pairs side
// by side (246 MB): 41 us, 6.0 TB/s; 64 tokens 2.4 to 2.6 us, a launch's time.  In
// CTAs of 256 threads 104, 42.2 and 2.8.
//
// Bounds: a page's keys are read once, D / 8 lanes a row.  8 prompts of 1001 to
// 4000 tokens (39 MB) 9.9 us: slots, then two rounds of 16 rows, each a memory
// latency; 256 decodes 2.8.  16 loads in flight in the place of 8 did not help
// (11.7 and 3.2).
#include <cstring>

#include "common.cuh"
#include "internal.h"
#include "paged.h"

namespace pa {
namespace {

constexpr int kRowsThreads = 128;

// cos and sin of x * turn / 2^64 turns.
__device__ __forceinline__ float2 turned(int32_t x, uint64_t turn) {
  const uint64_t t = static_cast<uint64_t>(static_cast<int64_t>(x)) * turn;
  float s, c;
  sincospif(static_cast<float>(static_cast<int32_t>(t >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31 half turns
  return make_float2(c, s);
}

// Two 16-byte pieces of a head, rotated: `lo` holds the pairs' first values and
// `hi` their second ones, or each holds four pairs side by side.
template <typename T, bool kInterleaved>
__device__ __forceinline__ void rotate(uint4& lo, uint4& hi, const float (&c)[8], const float (&s)[8]) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  if constexpr (kInterleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = Elt<T>::to_f2(w[i]);
      w[i] = Elt<T>::from_f2(v.x * c[i] - v.y * s[i], v.y * c[i] + v.x * s[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = Elt<T>::to_f2(w[i]), b = Elt<T>::to_f2(w[4 + i]);
      w[i] = Elt<T>::from_f2(a.x * c[2 * i] - b.x * s[2 * i], a.y * c[2 * i + 1] - b.y * s[2 * i + 1]);
      w[4 + i] = Elt<T>::from_f2(b.x * c[2 * i] + a.x * s[2 * i], b.y * c[2 * i + 1] + a.y * s[2 * i + 1]);
    }
  }
  lo = make_uint4(w[0], w[1], w[2], w[3]);
  hi = make_uint4(w[4], w[5], w[6], w[7]);
}

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kRowsThreads) rows_kernel(const RowsParams p) {
  constexpr int U = 4;  // heads in flight
  pdl_wait();
  const int lanes = p.D / 16, tokens = kRowsThreads / lanes;
  const int mine = static_cast<int>(threadIdx.x) / lanes, j = static_cast<int>(threadIdx.x) - mine * lanes;
  const int64_t tok = static_cast<int64_t>(blockIdx.x) * tokens + mine;
  if (mine >= tokens || tok >= p.n) return;
  int group = blockIdx.y, which = 0;
  while (which < 2 && group >= p.part[which].groups) group -= p.part[which++].groups;
  const RowsPart part = p.part[which];
  const int h0 = group * p.group_heads, heads = min(p.group_heads, part.heads - h0);

  T* out;
  int64_t out_step = p.D;  // between heads
  if (part.out) {
    out = static_cast<T*>(part.out) + tok * part.out_stride;
  } else {
    const int64_t slot = p.slots[tok];
    if (slot < 0) return;
    if (slot >= static_cast<int64_t>(p.g.num_pages) << p.g.ps_shift) {
      atomicOr(p.status, PA_DEV_BAD_INDEX);
      return;
    }
    const int64_t row = ((slot >> p.g.ps_shift) * 2 + part.half) * p.g.ps * p.g.Hkv +
                        static_cast<int64_t>(static_cast<int>(slot) & (p.g.ps - 1)) * p.g.slot_rows;
    out = static_cast<T*>(p.cache) + row * p.D;
    out_step = static_cast<int64_t>(p.g.head_rows) * p.D;
  }
  const T* in = static_cast<const T*>(part.in) + tok * part.in_stride;

  // the thread's two pieces, and its 8 pairs' angles
  const bool turns = part.rotate && j < p.pairs / 8;
  const bool halves = turns && !kInterleaved;
  const int lo = halves ? 8 * j : 16 * j, hi = halves ? p.pairs + 8 * j : 16 * j + 8;
  float c[8], s[8];
  if (turns) {
    int32_t x[8];
    if (p.axes) {
      int axis[8];
      bool sound = true;
#pragma unroll
      for (int i = 0; i < 8; ++i) axis[i] = p.axes[8 * j + i];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool in = static_cast<unsigned>(axis[i]) < static_cast<unsigned>(p.num_axes);
        sound = sound && in;
        x[i] = p.positions[(in ? axis[i] : 0) * p.position_stride + tok];
      }
      if (!sound && p.status) atomicOr(p.status, PA_DEV_BAD_INDEX);
    } else {
      x[0] = p.positions[tok];
#pragma unroll
      for (int i = 1; i < 8; ++i) x[i] = x[0];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 cs = turned(x[i], p.turns[8 * j + i]);
      c[i] = cs.x * p.scale;
      s[i] = cs.y * (p.scale * p.sign);
    }
  }
  for (int a = 0; a < heads; a += U) {
    uint4 v[U], w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const T* row = in + static_cast<int64_t>(h0 + min(a + u, heads - 1)) * p.D;
      v[u] = *reinterpret_cast<const uint4*>(row + lo);
      w[u] = *reinterpret_cast<const uint4*>(row + hi);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (a + u >= heads) break;
      if (turns) rotate<T, kInterleaved>(v[u], w[u], c, s);
      T* row = out + (h0 + a + u) * out_step;
      *reinterpret_cast<uint4*>(row + lo) = v[u];
      *reinterpret_cast<uint4*>(row + hi) = w[u];
    }
  }
}

// ---------------------------------------------------------------------------
// bounds

template <typename T> struct Pair;
template <> struct Pair<__half> { using type = __half2; };
template <> struct Pair<__nv_bfloat16> { using type = __nv_bfloat162; };

// Largest and smallest of packed pairs; a NaN stays one.
template <typename T>
__device__ __forceinline__ uint32_t most2(uint32_t a, uint32_t b) {
  using P = typename Pair<T>::type;
  const P r = __hmax2_nan(*reinterpret_cast<const P*>(&a), *reinterpret_cast<const P*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <typename T>
__device__ __forceinline__ uint32_t least2(uint32_t a, uint32_t b) {
  using P = typename Pair<T>::type;
  const P r = __hmin2_nan(*reinterpret_cast<const P*>(&a), *reinterpret_cast<const P*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

constexpr int kBoundsWarps = 4;

// The slot of a warp's token base + lane (lane < warp_tokens) where it is the last of its
// page, that is, where the next row that has a slot is of another page; otherwise -1.
// Rows without a slot, and those beyond the cache, may stand between two rows of a page, which
// would otherwise both write its bounds.  The next row is looked for among 64 slots that
// the warp loads at once.  Only where they hold none, and the last row of the warp does not fill
// its page, is it looked for among the CTA's later tokens, and behind them by all warps, 2048 slots
// at a time (64 tokens with 8128 rows of padding 16.7 us, by one warp 25.1).
struct BoundsShared {
  int64_t first[kBoundsWarps];  // slot of the first row of a warp's tokens that has one
  unsigned long long behind;    // index of the first such row behind the CTA's tokens
};
__device__ __forceinline__ int64_t end_of_page(const BoundsParams& p, BoundsShared& sh) {
  constexpr int U = 16;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t cta = static_cast<int64_t>(blockIdx.x) * kBoundsWarps * p.warp_tokens, base = cta + warp * p.warp_tokens;
  const int64_t end = static_cast<int64_t>(p.g.num_pages) << p.g.ps_shift;
  auto load = [&](int64_t i) { return i < p.n ? p.slots[i] : int64_t(-1); };
  auto counts = [&](int64_t s) { return s >= 0 && s < end; };
  const int64_t s0 = load(base + lane), s1 = load(base + 32 + lane);
  const unsigned m0 = __ballot_sync(0xffffffffu, counts(s0)), m1 = __ballot_sync(0xffffffffu, counts(s1));
  const unsigned later = m0 & (0xfffffffeu << lane);
  const int64_t next0 = __shfl_sync(0xffffffffu, s0, (__ffs(later) - 1) & 31);
  const int64_t next1 = __shfl_sync(0xffffffffu, s1, (__ffs(m1) - 1) & 31);
  int64_t next = later ? next0 : (m1 ? next1 : -1);
  int64_t slot = lane < p.warp_tokens ? s0 : -1;
  if (slot >= end) {
    atomicOr(p.status, PA_DEV_BAD_INDEX);
    slot = -1;
  }
  // (one lane of a warp at most)
  bool far = slot >= 0 && (later | m1) == 0 && (static_cast<int>(slot) & (p.g.ps - 1)) < p.g.ps - 1 && base + 64 < p.n;
  if (__syncthreads_or(far)) {
    const unsigned own = m0 & (0xffffffffu >> (32 - p.warp_tokens));
    const int64_t first = __shfl_sync(0xffffffffu, s0, (__ffs(own) - 1) & 31);
    if (lane == 0) sh.first[warp] = own ? first : -1;
    if (tid == 0) sh.behind = ~0ull;
    __syncthreads();
    for (int w = warp + 1; far && w < kBoundsWarps; ++w)
      if (sh.first[w] >= 0) next = sh.first[w], far = false;
    bool look = __syncthreads_or(far);  // (of one warp at most)
    for (int64_t i = cta + kBoundsWarps * p.warp_tokens; look && i < p.n; i += U * 32 * kBoundsWarps) {
      int64_t s[U];
#pragma unroll
      for (int u = 0; u < U; ++u) s[u] = load(i + u * 32 * kBoundsWarps + tid);
      unsigned long long found = ~0ull;
#pragma unroll
      for (int u = U - 1; u >= 0; --u)
        if (counts(s[u])) found = i + u * 32 * kBoundsWarps + tid;
      if (found != ~0ull) atomicMin(&sh.behind, found);
      look = !__syncthreads_or(found != ~0ull);
    }
    if (far && sh.behind != ~0ull) next = p.slots[sh.behind];
  }
  if (next >= 0 && (next >> p.g.ps_shift) == (slot >> p.g.ps_shift)) {
    if (next <= slot) atomicOr(p.status, PA_DEV_BAD_INDEX);  // out of order
    slot = -1;  // a later token's page
  }
  return slot;
}

// A warp looks at `warp_tokens` tokens for the last of each page, and for each
// reads one head's keys of that page: D / 8 lanes a row, 16 bytes each.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kBoundsWarps) bounds_kernel(const BoundsParams p) {
  constexpr int LANES = D / 8, ROWS = 32 / LANES, U = 8;
  __shared__ BoundsShared shared;
  pdl_wait();
  const int lane = threadIdx.x & 31, h = blockIdx.y;
  const int64_t slot = end_of_page(p, shared);
  for (unsigned todo = __ballot_sync(0xffffffffu, slot >= 0); todo; todo &= todo - 1) {
    const int64_t at = __shfl_sync(0xffffffffu, slot, __ffs(todo) - 1);
    const int64_t page = at >> p.g.ps_shift;
    const int rows = (static_cast<int>(at) & (p.g.ps - 1)) + 1;
    const T* keys = static_cast<const T*>(p.data) +
                    (page * 2 * p.g.ps * p.g.Hkv + static_cast<int64_t>(h) * p.g.head_rows) * D + (lane % LANES) * 8;
    const int64_t step = static_cast<int64_t>(p.g.slot_rows) * D;
    uint32_t top[4], low[4];
    for (int r0 = 0; r0 < rows; r0 += U * ROWS) {
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)  // rows past the last are the last again
        v[u] = *reinterpret_cast<const uint4*>(keys + min(r0 + u * ROWS + lane / LANES, rows - 1) * step);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          top[i] = r0 + u ? most2<T>(top[i], w[i]) : w[i];
          low[i] = r0 + u ? least2<T>(low[i], w[i]) : w[i];
        }
      }
    }
    float hi[8], lo[8], a = 0.f;
    bool sound = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int d = LANES; d < 32; d <<= 1) {
        top[i] = most2<T>(top[i], __shfl_xor_sync(0xffffffffu, top[i], d));
        low[i] = least2<T>(low[i], __shfl_xor_sync(0xffffffffu, low[i], d));
      }
      const float2 x = Elt<T>::to_f2(top[i]), y = Elt<T>::to_f2(low[i]);
      hi[2 * i] = x.x, hi[2 * i + 1] = x.y, lo[2 * i] = y.x, lo[2 * i + 1] = y.y;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float m = fmaxf(fabsf(hi[i]), fabsf(lo[i]));
      sound = sound && fabsf(hi[i]) < INFINITY && fabsf(lo[i]) < INFINITY;  // false for NaN too
      a = fmaxf(a, m);
    }
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
    sound = __all_sync(0xffffffffu, sound);
    if (a < 7.888609052210118e-31f) a = 0.f;  // 2^-100
    const float f = a > 0.f ? 127.f * __frcp_rn(a) : 0.f;
    uint32_t ct[2] = {0, 0}, cl[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = sound ? static_cast<int>(fminf(ceilf(hi[i] * f), 127.f)) : 127;
      const int l = sound ? static_cast<int>(fmaxf(floorf(lo[i] * f), -127.f)) : -127;
      ct[i >> 2] |= static_cast<uint32_t>(t & 0xFF) << (8 * (i & 3));
      cl[i >> 2] |= static_cast<uint32_t>(l & 0xFF) << (8 * (i & 3));
    }
    int8_t* codes = p.bounds + (page * p.g.Hkv + h) * (2 * D) + (lane % LANES) * 8;
    if (lane < LANES) {
      *reinterpret_cast<uint2*>(codes) = make_uint2(ct[0], ct[1]);
      *reinterpret_cast<uint2*>(codes + D) = make_uint2(cl[0], cl[1]);
    }
    if (lane == 0) p.scales[page * p.g.Hkv + h] = sound ? a * (1.f / 127.f) : INFINITY;
  }
}

template <typename... KArgs, typename... Args>
cudaError_t launch_2d(void (*kernel)(KArgs...), dim3 grid, unsigned block, cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  std::memset(attr, 0, sizeof(attr));
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
#ifndef PA_NO_PDL
  attr[0].val.programmaticStreamSerializationAllowed = 1;
#endif
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace

cudaError_t launch_rows(RowsParams p, int parts, bool interleaved, int dtype, int num_sms, cudaStream_t stream) {
  const int tokens = kRowsThreads / (p.D / 16);
  const int64_t blocks = (int64_t(p.n) + tokens - 1) / tokens;
  int heads = 0;
  for (int i = 0; i < parts; ++i) heads += p.part[i].heads;
  // The angles are made once a group: of 8 heads where the card is full without
  // more (16000 tokens 102 us, of 4 heads 109), of 4 for few tokens (64 tokens 2.3 us,
  // of 8 2.8).
  p.group_heads = blocks * heads >= int64_t(num_sms) * 128 ? 8 : 4;
  unsigned groups = 0;
  for (int i = 0; i < 3; ++i) {
    p.part[i].groups = i < parts ? (p.part[i].heads + p.group_heads - 1) / p.group_heads : 0;
    groups += p.part[i].groups;
  }
  const dim3 grid(static_cast<unsigned>(blocks), groups);
  if (dtype == PA_BF16)
    return interleaved ? launch_2d(rows_kernel<__nv_bfloat16, true>, grid, kRowsThreads, stream, p)
                       : launch_2d(rows_kernel<__nv_bfloat16, false>, grid, kRowsThreads, stream, p);
  return interleaved ? launch_2d(rows_kernel<__half, true>, grid, kRowsThreads, stream, p)
                     : launch_2d(rows_kernel<__half, false>, grid, kRowsThreads, stream, p);
}

cudaError_t launch_bounds(BoundsParams p, int D, int dtype, int num_sms, cudaStream_t stream) {
  // A warp a token where there are few (each may end a page: 256 decodes 2.8 us,
  // 31 with 32 tokens a warp), up to 32 where most do not (8 prompts 10 us, 22
  // with one).
  p.warp_tokens = 1;
  while (p.warp_tokens < 32 && int64_t(p.n) * p.g.Hkv > int64_t(num_sms) * 32 * p.warp_tokens) p.warp_tokens *= 2;
  const int64_t per_block = int64_t(p.warp_tokens) * kBoundsWarps;
  const dim3 grid(static_cast<unsigned>((p.n + per_block - 1) / per_block), p.g.Hkv);
  const unsigned block = 32 * kBoundsWarps;
  if (dtype == PA_BF16) {
    if (D == 64) return launch_2d(bounds_kernel<__nv_bfloat16, 64>, grid, block, stream, p);
    if (D == 128) return launch_2d(bounds_kernel<__nv_bfloat16, 128>, grid, block, stream, p);
    return launch_2d(bounds_kernel<__nv_bfloat16, 256>, grid, block, stream, p);
  }
  if (D == 64) return launch_2d(bounds_kernel<__half, 64>, grid, block, stream, p);
  if (D == 128) return launch_2d(bounds_kernel<__half, 128>, grid, block, stream, p);
  return launch_2d(bounds_kernel<__half, 256>, grid, block, stream, p);
}

}  // namespace pa
