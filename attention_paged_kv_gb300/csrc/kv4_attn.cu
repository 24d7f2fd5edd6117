// Attention over a paged cache held in 4 bits, through device tables
// (pagedattn_kv4_run): the small-query kernel and the merge of its splits.
//
// Number formats.  K and V are e2m1 codes with an e4m3 scale per 16 values
// along head_dim.  code * scale has at most 6 significant bits and lies in
// [2^-10, 2688], so it is exact in fp16: every product below is an fp16 MMA
// over the exact cache values, for fp16 and bf16 queries alike.  A bf16 query
// row is multiplied by the power of two that brings its largest value to
// [2^13, 2^14) first (bf16's 8 significant bits fit fp16's 11; what falls
// below fp16's range is 2^-38 of the row's largest value) and the logits by
// its inverse.  The cache's own fp32 scales go into the logit factor (K) and
// the epilogue (V).  P is rounded to fp16 (2^-11 relative) for the P V
// product, whatever the type of q: a bf16 P would cost 2^-8.
//
// Work.  A unit is 64 keys of one row tile (8 * NT packed rows: token major,
// the G query heads of the kv head minor) of one request.  The units of the
// batch, in request order, are cut into equal slices, one per CTA and kv
// head, whatever the requests' boundaries, so that one request of 10^5 keys
// and 10^3 requests of 100 keys load the SMs alike with no plan from the
// host: every CTA sums the units of all requests itself (one block scan) and
// so finds where its slice begins.  CTAs of one slice and different kv heads
// are adjacent: they read the same pages at the same time, and in the NHD
// layout the 32-byte sectors of scales that 4 heads share come from L2.
// A row tile that a slice boundary cuts leaves fp32 partial states.
//
// A warp takes 16 keys at a time and computes S^T = K q^T and O^T = V^T P^T
// with m16n8k16, so that keys (or dims) fill the 16-row side and 8 packed
// rows the other.  Both contractions are free in the order of their index:
//   S^T  lane (g, t) takes dims [t D/4, (t+1) D/4) of keys g and g + 8: one
//        16-byte load a key (head_dim 128), codes converted in the order they
//        lie in memory; q's fragments are loaded in the same order.
//   O^T  lane (g, t) takes dims [g D/8, (g+1) D/8) of keys 2t, 2t+1, 2t+8 and
//        2t+9: the codes of two keys are merged nibble by nibble (two
//        bitfield selects for 16 values) so that one conversion gives the
//        fragment's (key, key + 1) pair.
// So the cache goes from global memory to registers and into the MMA without
// shared memory.
#include <cstring>

#include "internal.h"
#include "kv4_common.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnitKeys = 64;
constexpr int kMinUnits = 4;  // of a slice: below 256 keys a split costs more than it spreads
constexpr float kLn2f = 0.6931471805599453f;

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ int row_tiles(const Kv4Params& p, const Req& r, int tile_rows) {
  const int rows = r.qo_len * p.G;
  return rows > p.small_rows ? 0 : (rows + tile_rows - 1) / tile_rows;
}
__device__ __forceinline__ int key_units(const Req& r) { return max(1, (r.kv_len + kUnitKeys - 1) / kUnitKeys); }

// ---------------------------------------------------------------------------
// 4-bit fragments

// (a & m) | (b & ~m): low nibbles of a, high nibbles of b.
__device__ __forceinline__ uint32_t select_nibbles(uint32_t a, uint32_t b) {
  return (a & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int BYTES> struct Piece;  // a lane's contiguous codes of one row
template <> struct Piece<4> { uint32_t w[1]; };
template <> struct Piece<8> { uint32_t w[2]; };
template <> struct Piece<16> { uint32_t w[4]; };
template <> struct Piece<32> { uint32_t w[8]; };

template <int BYTES>
__device__ __forceinline__ Piece<BYTES> load_piece(const uint8_t* src) {
  Piece<BYTES> r;
  if constexpr (BYTES == 4) {
    r.w[0] = __ldg(reinterpret_cast<const uint32_t*>(src));
  } else if constexpr (BYTES == 8) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
    r.w[0] = v.x;
    r.w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + i);
      r.w[4 * i] = v.x;
      r.w[4 * i + 1] = v.y;
      r.w[4 * i + 2] = v.z;
      r.w[4 * i + 3] = v.w;
    }
  }
  return r;
}
template <int BYTES>
__device__ __forceinline__ uint32_t load_scales(const uint8_t* src) {
  if constexpr (BYTES == 1) return __ldg(src);
  if constexpr (BYTES == 2) return __ldg(reinterpret_cast<const unsigned short*>(src));
  return __ldg(reinterpret_cast<const uint32_t*>(src));
}

// What a lane holds of 16 keys.
template <int D>
struct KeyStep {
  static constexpr int KB = D / 8;                      // bytes of a K row: D/4 dims
  static constexpr int VB = D / 16;                     // bytes of a V row: D/8 dims
  static constexpr int KS = D / 64;                     // their scales
  static constexpr int VS = D >= 128 ? D / 128 : 1;
  Piece<KB> k[2];  // keys g, g + 8
  Piece<VB> v[4];  // keys 2t, 2t + 1, 2t + 8, 2t + 9
  uint32_t ks[2], vs[4];
};

template <int D, int NT>
struct SmallCfg {
  static constexpr int ROWS = 8 * NT;
  static constexpr int O_STRIDE = D + 4;  // floats of a row in the combine buffer
  static constexpr int SMEM = kWarps * ROWS * O_STRIDE * 4 + 2 * kWarps * ROWS * 4;
  static constexpr int CTAS = D == 256 ? 1 : 2;  // of an SM
};

// Sum over the block (every thread gets it).
__device__ __forceinline__ long long block_sum(long long v, long long* scratch) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  long long s = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += scratch[w];
  __syncthreads();
  return s;
}

template <typename T, int D, int NT, bool kSmallPage>
__global__ void __launch_bounds__(kThreads, SmallCfg<D, NT>::CTAS) kv4_small_kernel(const Kv4Params p) {
  using C = SmallCfg<D, NT>;
  using Step = KeyStep<D>;
  extern __shared__ float smem_f[];
  float* o_s = smem_f;                                    // [warps][rows][O_STRIDE]
  float* m_s = smem_f + kWarps * C::ROWS * C::O_STRIDE;   // [warps][rows]
  float* l_s = m_s + kWarps * C::ROWS;                    // [warps][rows]
  __shared__ long long scratch[kWarps];
  __shared__ long long found_u;
  __shared__ int found_b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int h = blockIdx.x % p.g.Hkv, slice = blockIdx.x / p.g.Hkv;
  pdl_wait();

  // ---- the slice's units [u, u_end) and the request that they begin in
  auto units_of = [&](int b) -> long long {
    const Req r = load_req(p, b);
    return static_cast<long long>(row_tiles(p, r, C::ROWS)) * key_units(r);
  };
  long long mine = 0;
  for (int b = tid; b < p.batch; b += kThreads) mine += units_of(b);
  const long long total = block_sum(mine, scratch);
  const long long per_slice = max(static_cast<long long>(kMinUnits), (total + p.slices - 1) / p.slices);
  long long u = slice * per_slice;
  const long long u_end = min(total, u + per_slice);
  if (h == 0 && tid == 0 && (u >= u_end || slice == 0)) p.splits[slice].valid = 0;
  if (u >= u_end) return;
  long long base = 0;  // units before the chunk of requests
  for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
    const long long v = b0 + tid < p.batch ? (p.batch <= kThreads ? mine : units_of(b0 + tid)) : 0;
    long long x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    long long before = base, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += scratch[w];
      all += scratch[w];
    }
    const long long first = before + x - v;
    if (v > 0 && first <= u && u < first + v) {
      found_b = b0 + tid;
      found_u = first;
    }
    __syncthreads();
    base += all;
    if (u < base) break;
  }
  int b = found_b;  // always found: u < total
  long long req_u = found_u;  // the request's first unit
  Req rq = load_req(p, b);

  // ---- row tiles, one after the other
  bool first_segment = true;
  while (u < u_end) {
    const int kts = key_units(rq);
    const int rt = static_cast<int>((u - req_u) / kts);
    const long long tile_u = req_u + static_cast<long long>(rt) * kts;
    const int unit0 = static_cast<int>(u - tile_u);
    const long long seg_end = min(u_end, tile_u + kts);
    const int rows = min(C::ROWS, rq.qo_len * p.G - rt * C::ROWS);
    const int row0 = rt * C::ROWS;
    // keys that some row of the tile sees, and those that every row sees
    const int shift = rq.kv_len - rq.qo_len + 1;
    const int seen_end = p.causal ? max(0, shift + (row0 + rows - 1) / p.G) : rq.kv_len;
    const int all_end = p.causal ? shift + row0 / p.G : rq.kv_len;
    const int key_a = unit0 * kUnitKeys;
    const int key_b = min(static_cast<int>(seg_end - tile_u) * kUnitKeys, seen_end);
    const int steps = key_b > key_a ? (key_b - key_a + 15) / 16 : 0;

    if (h == 0 && tid == 0 && first_segment && slice > 0) {
      Kv4Split s;
      s.valid = u > tile_u;
      s.qo_row0 = rq.qo_start;
      s.rows = rq.qo_len * p.G;
      s.row_tile = rt;
      s.u0 = tile_u;
      s.u1 = tile_u + kts;
      s.per_slice = per_slice;
      p.splits[slice] = s;
    }

    // page ids two steps ahead, codes one
    const int32_t* page_ids = p.pages + rq.page_start;
    auto step_page = [&](int s) -> int {  // kSmallPage: of key (lane & 15) of the step
      if (s >= steps) return 0;
      const int key = key_a + s * 16;
      int pid;
      if constexpr (kSmallPage)
        pid = __ldg(page_ids + (min(key + (lane & 15), rq.kv_len - 1) >> p.g.ps_shift));
      else
        pid = __ldg(page_ids + (key >> p.g.ps_shift));
      return pid;
    };
    const int64_t half_rows = static_cast<int64_t>(p.g.ps) * p.g.Hkv;
    const int64_t head_off = static_cast<int64_t>(h) * p.g.head_rows;
    auto load_step = [&](Step& f, int s, int pid) {
      if (s >= steps) return;
      if (static_cast<unsigned>(pid) >= static_cast<unsigned>(p.g.num_pages)) {
        atomicOr(p.status, PA_DEV_BAD_INDEX);
        pid = 0;
      }
      const int key = key_a + s * 16;
      if constexpr (kSmallPage) {
        auto row_of = [&](int i, int half) {
          const int id = __shfl_sync(0xffffffffu, pid, i);
          const int slot = min(key + i, rq.kv_len - 1) & (p.g.ps - 1);
          return (static_cast<int64_t>(id) * 2 + half) * half_rows + static_cast<int64_t>(slot) * p.g.slot_rows +
                 head_off;
        };
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int64_t row = row_of(g + 8 * i, 0);
          f.k[i] = load_piece<Step::KB>(p.codes + row * (D / 2) + t * Step::KB);
          f.ks[i] = load_scales<Step::KS>(p.scales + row * (D / 16) + t * Step::KS);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t row = row_of(2 * t + (i & 1) + 8 * (i >> 1), 1);
          f.v[i] = load_piece<Step::VB>(p.codes + row * (D / 2) + g * Step::VB);
          f.vs[i] = load_scales<Step::VS>(p.scales + row * (D / 16) + (g * D / 8) / 16);
        }
      } else {
        // pages of 16 slots or more: the step's 16 slots are all in one page
        // (those past the last key too, so nothing has to be clamped)
        const int64_t row = static_cast<int64_t>(pid) * 2 * half_rows +
                            static_cast<int64_t>(key & (p.g.ps - 1)) * p.g.slot_rows + head_off;
        const uint8_t* kc = p.codes + row * (D / 2);
        const uint8_t* ksc = p.scales + row * (D / 16);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = (g + 8 * i) * p.g.slot_rows;
          f.k[i] = load_piece<Step::KB>(kc + static_cast<int64_t>(r) * (D / 2) + t * Step::KB);
          f.ks[i] = load_scales<Step::KS>(ksc + static_cast<int64_t>(r) * (D / 16) + t * Step::KS);
        }
        const uint8_t* vc = kc + half_rows * (D / 2);
        const uint8_t* vsc = ksc + half_rows * (D / 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = (2 * t + (i & 1) + 8 * (i >> 1)) * p.g.slot_rows;
          f.v[i] = load_piece<Step::VB>(vc + static_cast<int64_t>(r) * (D / 2) + g * Step::VB);
          f.vs[i] = load_scales<Step::VS>(vsc + static_cast<int64_t>(r) * (D / 16) + (g * D / 8) / 16);
        }
      }
    };
    int pid0 = step_page(warp), pid1 = step_page(warp + kWarps);
    Step cur, nxt;
    load_step(cur, warp, pid0);

    // q fragments (row n = g of each 8-row group, dims [t D/4, (t+1) D/4)) and
    // the logit factors of rows 2t, 2t + 1
    uint32_t qf[NT][D / 16][2];
    float fac[NT][2];
    int lim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int n = nt * 8 + g, r = row0 + n;
      float my = p.scale_log2;
      if (n < rows) {
        const T* src = static_cast<const T*>(p.q) + static_cast<int64_t>(rq.qo_start + r / p.G) * p.q_stride +
                       static_cast<int64_t>(h * p.G + r % p.G) * D + t * (D / 4);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          const uint4 w = *(reinterpret_cast<const uint4*>(src) + c);
          qf[nt][2 * c][0] = w.x;
          qf[nt][2 * c][1] = w.y;
          qf[nt][2 * c + 1][0] = w.z;
          qf[nt][2 * c + 1][1] = w.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < D / 16; ++j) qf[nt][j][0] = qf[nt][j][1] = 0;
      }
      if constexpr (Elt<T>::kBf16) {
        uint32_t top = 0;  // the largest magnitude's bf16 bits
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            top = max(top, max(qf[nt][j][i] & 0x7FFFu, (qf[nt][j][i] >> 16) & 0x7FFFu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int up = bf16_row_shift(top);
        const float mul = pow2(up);
        my *= pow2(-up);
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 f = Elt<T>::to_f2(qf[nt][j][i]);
            qf[nt][j][i] = pack_f16x2(f.x * mul, f.y * mul);
          }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        fac[nt][i] = __shfl_sync(0xffffffffu, my, (2 * t + i) * 4);
        const int r2 = row0 + nt * 8 + 2 * t + i;
        lim[nt][i] = p.causal ? min(shift + r2 / p.G, rq.kv_len) : rq.kv_len;
      }
    }

    float o[NT][D / 16][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }

    auto compute = [&](Step& f, int s) {
      const int key = key_a + s * 16;
      float sc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
      for (int w = 0; w < Step::KB / 4; ++w) {  // 8 dims of each of the two keys
        uint32_t a[4], c[4];
        e2m1x8(f.k[0].w[w], a);
        e2m1x8(f.k[1].w[w], c);
        const uint32_t b0 = (f.ks[0] >> (8 * (w >> 1))) & 0xFFu, b1 = (f.ks[1] >> (8 * (w >> 1))) & 0xFFu;
        const uint32_t s0 = e4m3x2_f16(b0 * 0x101u), s1 = e4m3x2_f16(b1 * 0x101u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = mul_f16x2(a[i], s0);
          c[i] = mul_f16x2(c[i], s1);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16(sc[nt], a[0], c[0], a[1], c[1], qf[nt][2 * w][0], qf[nt][2 * w][1]);
          mma_f16(sc[nt], a[2], c[2], a[3], c[3], qf[nt][2 * w + 1][0], qf[nt][2 * w + 1][1]);
        }
      }
      uint32_t pb[NT][2];
      const bool edge = key + 16 > all_end;  // some row does not see every key of the step
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = sc[nt][e] * fac[nt][e & 1];
          if (edge && key + g + 8 * (e >> 1) >= lim[nt][e & 1]) x[e] = -INFINITY;
        }
        // the reference maximum moves when a logit passes it by 8 (in log2
        // units): P stays below 2^8, which fp16 and the fp32 sums carry
        const bool grow = fmaxf(x[0], x[2]) > m[nt][0] + 8.f || fmaxf(x[1], x[3]) > m[nt][1] + 8.f;
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float top = fmaxf(x[i], x[i + 2]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float now = fmaxf(m[nt][i], top);
            const float alpha = now == m[nt][i] ? 1.f : ex2f(m[nt][i] - now);
            m[nt][i] = now;
            l[nt][i] *= alpha;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              o[nt][j][i] *= alpha;
              o[nt][j][i + 2] *= alpha;
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float ref = m[nt][e & 1] == -INFINITY ? 0.f : m[nt][e & 1];
          x[e] = ex2f(x[e] - ref);
          l[nt][e & 1] += x[e];
        }
        pb[nt][0] = movmatrix(pack_f16x2(x[0], x[1]));
        pb[nt][1] = movmatrix(pack_f16x2(x[2], x[3]));
      }
      if (key + 16 > seen_end) {
        // slots past the last key may hold anything: a NaN scale would pass
        // through P = 0
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (key + 2 * t + (i & 1) + 8 * (i >> 1) >= seen_end) f.vs[i] = 0;
      }
#pragma unroll
      for (int w = 0; w < Step::VB / 4; ++w) {  // 8 dims of each of the four keys
        const int sh = 8 * (w >> 1);
        const uint32_t s01 = e4m3x2_f16(((f.vs[0] >> sh) & 0xFFu) | (((f.vs[1] >> sh) & 0xFFu) << 8));
        const uint32_t s89 = e4m3x2_f16(((f.vs[2] >> sh) & 0xFFu) | (((f.vs[3] >> sh) & 0xFFu) << 8));
        uint32_t a[4], b[4], c[4], d[4];
        e2m1x8(select_nibbles(f.v[0].w[w], f.v[1].w[w] << 4), a);
        e2m1x8(select_nibbles(f.v[0].w[w] >> 4, f.v[1].w[w]), b);
        e2m1x8(select_nibbles(f.v[2].w[w], f.v[3].w[w] << 4), c);
        e2m1x8(select_nibbles(f.v[2].w[w] >> 4, f.v[3].w[w]), d);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = mul_f16x2(a[i], s01);
          b[i] = mul_f16x2(b[i], s01);
          c[i] = mul_f16x2(c[i], s89);
          d[i] = mul_f16x2(d[i], s89);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt][4 * w + i], a[i], b[i], c[i], d[i], pb[nt][0], pb[nt][1]);
        }
      }
    };
    for (int s = warp; s < steps; s += 2 * kWarps) {
      pid0 = step_page(s + 2 * kWarps);
      load_step(nxt, s + kWarps, pid1);
      compute(cur, s);
      pid1 = step_page(s + 3 * kWarps);
      load_step(cur, s + 2 * kWarps, pid0);
      if (s + kWarps < steps) compute(nxt, s + kWarps);
    }

    // ---- the warps' states are joined
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], d);
        const int n = nt * 8 + 2 * t + i;
        if (g == 0) {
          m_s[warp * C::ROWS + n] = m[nt][i];
          l_s[warp * C::ROWS + n] = l[nt][i];
        }
        float* dst = o_s + (warp * C::ROWS + n) * C::O_STRIDE + g * (D / 8);
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
          *reinterpret_cast<float4*>(dst + 4 * j) = make_float4(o[nt][2 * j][i], o[nt][2 * j][i + 2],
                                                                o[nt][2 * j + 1][i], o[nt][2 * j + 1][i + 2]);
      }
    __syncthreads();
    const bool whole = unit0 == 0 && seg_end == tile_u + kts;
    const int64_t part = (static_cast<int64_t>(blockIdx.x) * 2 + (first_segment ? 0 : 1)) * C::ROWS;
    for (int i = tid; i < rows * (D / 4); i += kThreads) {
      const int n = i / (D / 4), d = (i % (D / 4)) * 4;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, m_s[w * C::ROWS + n]);
      const float ref = top == -INFINITY ? 0.f : top;
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float a = ex2f(m_s[w * C::ROWS + n] - ref);
        const float4 v = *reinterpret_cast<const float4*>(o_s + (w * C::ROWS + n) * C::O_STRIDE + d);
        sum += a * l_s[w * C::ROWS + n];
        acc.x += a * v.x;
        acc.y += a * v.y;
        acc.z += a * v.z;
        acc.w += a * v.w;
      }
      // a row that sees no key: zeros, and -inf as its lse
      const float inv = sum == 0.f ? 0.f : (whole ? p.v_scale : 1.f) / sum;
      const float lse2 = sum == 0.f ? -INFINITY : ref + log2f(sum);
      acc.x *= inv;
      acc.y *= inv;
      acc.z *= inv;
      acc.w *= inv;
      if (whole) {
        const int r = row0 + n;
        const int64_t row = static_cast<int64_t>(rq.qo_start + r / p.G) * p.Hq + h * p.G + r % p.G;
        *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + row * D + d) =
            make_uint2(Elt<T>::from_f2(acc.x, acc.y), Elt<T>::from_f2(acc.z, acc.w));
        if (d == 0 && p.lse) p.lse[row] = lse2 * kLn2f;
      } else {
        *reinterpret_cast<float4*>(p.part_o + (part + n) * D + d) = acc;
        if (d == 0) p.part_lse[part + n] = lse2;
      }
    }
    __syncthreads();  // the buffers are the next row tile's
    first_segment = false;
    u = seg_end;
    if (u < u_end && rt + 1 == row_tiles(p, rq, C::ROWS)) {  // on to the next request with units
      req_u += static_cast<long long>(row_tiles(p, rq, C::ROWS)) * kts;
      do {
        if (++b >= p.batch) return;
        rq = load_req(p, b);
      } while (row_tiles(p, rq, C::ROWS) == 0);
    }
  }
}

// One CTA per slice boundary and kv head: where the boundary is the first one
// inside a row tile, the partial states of all slices that the tile spans are
// joined, o = sum_s 2^(lse_s - lse) o_s.
constexpr int kMergeThreads = 512;

template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(kMergeThreads) kv4_merge_kernel(const Kv4Params p) {
  constexpr int COLS = D / 4;                        // float4 columns of a row
  constexpr int GROUPS = kMergeThreads / COLS;       // rows x part groups at a time
  constexpr int RP = GROUPS < ROWS ? GROUPS : ROWS;  // rows at a time
  constexpr int PG = GROUPS / RP;                    // groups that share a row's parts
  __shared__ float4 acc_s[kMergeThreads];
  __shared__ float sum_s[kMergeThreads], top_s[kMergeThreads];
  pdl_wait();
  const int h = blockIdx.x % p.g.Hkv, slice = blockIdx.x / p.g.Hkv + 1;
  const Kv4Split s = p.splits[slice];
  if (!s.valid) return;
  const int sa = static_cast<int>(s.u0 / s.per_slice), sb = static_cast<int>((s.u1 - 1) / s.per_slice);
  if (sa != slice - 1) return;  // an earlier boundary's
  const bool sa_first = s.u0 == sa * s.per_slice;
  auto part_row = [&](int sl) {
    const int which = (sl == sa && !sa_first) ? 1 : 0;
    return ((static_cast<int64_t>(sl) * p.g.Hkv + h) * 2 + which) * ROWS;
  };
  const int col = threadIdx.x % COLS, grp = threadIdx.x / COLS, pg = grp / RP;
  const int rows = min(ROWS, s.rows - s.row_tile * ROWS);
  for (int n0 = 0; n0 < rows; n0 += RP) {
    const int n = n0 + grp % RP;
    const bool in = n < rows && pg < PG;
    float top = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) {
      for (int sl = sa + pg; sl <= sb; sl += PG) top = fmaxf(top, p.part_lse[part_row(sl) + n]);
      const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll 4
      for (int sl = sa + pg; sl <= sb; sl += PG) {
        const int64_t row = part_row(sl) + n;
        const float a = ex2f(p.part_lse[row] - ref);
        const float4 v = *reinterpret_cast<const float4*>(p.part_o + row * D + col * 4);
        sum += a;
        acc.x += a * v.x;
        acc.y += a * v.y;
        acc.z += a * v.z;
        acc.w += a * v.w;
      }
    }
    acc_s[threadIdx.x] = acc;
    sum_s[threadIdx.x] = sum;
    top_s[threadIdx.x] = top;
    __syncthreads();
    if (in && pg == 0) {
      float all = -INFINITY;
#pragma unroll
      for (int k = 0; k < PG; ++k) all = fmaxf(all, top_s[threadIdx.x + k * RP * COLS]);
      const float ref = all == -INFINITY ? 0.f : all;
      sum = 0.f;
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < PG; ++k) {
        const int at = threadIdx.x + k * RP * COLS;
        const float a = ex2f(top_s[at] - ref);  // 0 where the group had no part
        const float4 v = acc_s[at];
        sum += a * sum_s[at];
        acc.x += a * v.x;
        acc.y += a * v.y;
        acc.z += a * v.z;
        acc.w += a * v.w;
      }
      const float inv = sum == 0.f ? 0.f : p.v_scale / sum;
      const int r = s.row_tile * ROWS + n;
      const int64_t row = static_cast<int64_t>(s.qo_row0 + r / p.G) * p.Hq + h * p.G + r % p.G;
      *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + row * D + col * 4) = make_uint2(
          Elt<T>::from_f2(acc.x * inv, acc.y * inv), Elt<T>::from_f2(acc.z * inv, acc.w * inv));
      if (col == 0 && p.lse) p.lse[row] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * kLn2f;
    }
    __syncthreads();
  }
}

// Packed rows of a tile: 8 where no request has more (or the registers of
// head_dim 256 allow no more), else 16.
int tile_rows(const Kv4Shape& s) { return s.max_rows <= 8 || s.D == 256 ? 8 : 16; }

template <typename T, int D, int NT>
cudaError_t launch_small(const Kv4Params& p, cudaStream_t stream) {
  using C = SmallCfg<D, NT>;
  const unsigned grid = static_cast<unsigned>(p.slices) * p.g.Hkv;
  static std::atomic<uint64_t> set_a{0}, set_b{0};
  cudaError_t e;
  if (p.g.ps < 16) {
    auto* k = kv4_small_kernel<T, D, NT, true>;
    e = set_smem_once(set_a, reinterpret_cast<const void*>(k), C::SMEM);
    if (e == cudaSuccess) e = launch_pdl(k, grid, unsigned(kThreads), size_t(C::SMEM), stream, p);
  } else {
    auto* k = kv4_small_kernel<T, D, NT, false>;
    e = set_smem_once(set_b, reinterpret_cast<const void*>(k), C::SMEM);
    if (e == cudaSuccess) e = launch_pdl(k, grid, unsigned(kThreads), size_t(C::SMEM), stream, p);
  }
  if (e != cudaSuccess || p.slices < 2) return e;
  return launch_pdl(kv4_merge_kernel<T, D, C::ROWS>, static_cast<unsigned>(p.slices - 1) * p.g.Hkv,
                    unsigned(kMergeThreads), size_t(0), stream, p);
}

template <typename T>
cudaError_t launch_t(const Kv4Params& p, const Kv4Shape& s, cudaStream_t stream) {
  const bool wide = tile_rows(s) == 16;
  switch (s.D) {
    case 64: return wide ? launch_small<T, 64, 2>(p, stream) : launch_small<T, 64, 1>(p, stream);
    case 128: return wide ? launch_small<T, 128, 2>(p, stream) : launch_small<T, 128, 1>(p, stream);
    default: return launch_small<T, 256, 1>(p, stream);
  }
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

Kv4Layout kv4_layout(const Kv4Shape& s) {
  Kv4Layout l;
  const int per_sm = s.D == 256 ? 1 : 2;
  const int slices = per_sm * s.num_sms / s.Hkv;
  l.slices = slices > 0 ? slices : 1;
  const size_t rows = size_t(l.slices) * s.Hkv * 2 * tile_rows(s);
  l.off_splits = 256;  // after the status word
  l.off_part_o = up256(l.off_splits + size_t(l.slices) * sizeof(Kv4Split));
  l.off_part_lse = up256(l.off_part_o + rows * s.D * sizeof(float));
  l.total = up256(l.off_part_lse + rows * sizeof(float));
  return l;
}

cudaError_t launch_kv4_attention(const Kv4Params& p, const Kv4Shape& s, int dtype, cudaStream_t stream) {
  return dtype == PA_BF16 ? launch_t<__nv_bfloat16>(p, s, stream) : launch_t<__half>(p, s, stream);
}

}  // namespace pa
