// Attention of each query over the pages on its list (pagedattn_blocks_run).
//
// Work.  An item is one query token and kv head (up to 16 of the group's heads,
// 8 at head_dim 256): its rows share every key.  A CTA takes an item, or where
// items are few a slice of its list; slices leave fp32 partial states that the
// last of them joins.  The CTA's warps take every fourth tile of 16 keys (32 at
// head_dim 64) and copy their own keys ahead (cp.async into a ring of their own),
// so that no warp waits for another until their states are joined at the end.
//
// S^T = K q^T and O^T = V^T P^T with m16n8k16: keys (or head dims) fill the
// 16-row side and the heads the other.  P is 2^(logit - m) with the reference m
// set 7 below the largest logit, in log2 units, and set again when a logit
// passes it by 15: a row's largest P lies in [2^7, 2^15], and the keys' ones
// down to 2^-21 of it are rounded like it.  P is split in two terms of the values' type and
// multiplied twice: by one term it would be off by 2^-8 in bf16 and 2^-11 in fp16 (64 decodes at
// 64 / 8 heads in fp16 75.9 us, with one 75.2; at 128 / 8 81.7 and 78.7).  Logits are scaled and rounded as m was
// before m is taken off (no fused step): however large they are, a key's is at most 15
// above m, and the largest not below it.
//
// What bounds it: HBM.  64 decodes of 2048 keys at 64 / 8 heads (464 MB) take 75
// us, 6.2 TB/s, 91 % of the copy rate; 3 requests of 4096 of up to 131071 keys (50 MB)
// 16.5, of them about 7 the copies, the rest tables, list, page ids and the first
// keys one after the other, and the join.  Steps on the way (us): a look-up of
// list and page for each row that is copied 89; whole pages 75.
#include <climits>
#include <cstring>

#include "internal.h"
#include "paged_common.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr float kNone = -3.0e38f;  // a maximum before any key: finite, so that it can be subtracted
constexpr float kHead = 7.f, kRise = 8.f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D, int NT>
struct Cfg {
  static constexpr int ROWS = 8 * NT;
  static constexpr int ROW = 2 * D;                  // bytes of a key's row
  // A tile: two pieces of 16 keys at head_dim 64, else one.  64 decodes of 2048 keys
  // at 64 / 8 heads of 64 take 44.0 us so and 45.3 with one piece (and three CTAs an
  // SM), 3 requests of 4096 keys 9.7 and 11.4.
  static constexpr int PIECES = D == 64 ? 2 : 1, TILE = 16 * PIECES;
  static constexpr int STAGE = 2 * TILE * ROW;       // K, then V
  static constexpr int STAGES = 3;
  static constexpr int RING = STAGES * STAGE;        // of a warp
  static constexpr int CTAS = D == 256 ? 1 : 2;
  static constexpr int SMEM = kWarps * RING;         // the list comes behind
  static constexpr int O_STRIDE = D + 4;             // floats of a row of a warp's state, in its ring's place
  static_assert(ROWS * (O_STRIDE + 2) * 4 <= RING, "a warp's state fits its ring");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
template <bool kTrans>
__device__ __forceinline__ void ldmatrix(uint32_t (&r)[4], uint32_t at) {
  if constexpr (kTrans)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
template <typename T>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (Elt<T>::kBf16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// A weight as two terms of its type: the first cut towards zero, the second what is left, never
// below kLeast (bf16 2^-100, fp16 its smallest number) of a weight above that: an infinity of V
// times terms of one sign, none of them zero, stays one.
template <typename T>
__device__ __forceinline__ uint32_t first_terms(float a, float b) {
  uint32_t r;
  if constexpr (Elt<T>::kBf16) asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  else asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
template <typename T>
__device__ __forceinline__ float second_term(float x, float first) {
  constexpr float kLeast = Elt<T>::kBf16 ? 0x1p-100f : 0x1p-24f;
  return fmaxf(x - first, fminf(x, kLeast));
}
template <int N> __device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Row `row` of a state: its four columns from `col` on as 16-bit values.
template <typename T>
__device__ __forceinline__ void store4(void* out, int64_t row, int D, int col, float4 v, float inv) {
  *reinterpret_cast<uint2*>(static_cast<T*>(out) + row * D + col) =
      make_uint2(Elt<T>::from_f2(v.x * inv, v.y * inv), Elt<T>::from_f2(v.z * inv, v.w * inv));
}

// Chunks whose items were cut along their keys (block_prefill.cu): the parts'
// states of each row joined, a row a warp, four rows in flight.
template <typename T, int D>
__device__ __forceinline__ void join_tiles(const BlockParams& p, int parts) {
  constexpr int V = D / 32, U = 4;  // columns of a lane
  const int TQ = 128 / p.G, lane = threadIdx.x & 31;
  const int per_item = p.tile_tokens * p.G, rows = p.tile_indptr[p.batch] * p.g.Hkv * per_item;
  const int tiles = p.tile_indptr[p.batch];
  for (int r0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * U; r0 < rows; r0 += gridDim.x * kWarps * U) {
    const float *lse[U], *o[U];
    int64_t out[U];  // rows of out, -1: none
    float top[U], sum[U], acc[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = min(r0 + u, rows - 1), place = r / per_item, rr = r - place * per_item, t = rr / p.G, g = rr - t * p.G;
      const int h = place % p.g.Hkv;
      const BlockItem* it = p.items + static_cast<int64_t>(tiles - 1 - place / p.g.Hkv) * p.g.Hkv + h;
      out[u] = r0 + u < rows && t < it->tokens ? (static_cast<int64_t>(it->token) + t) * p.Hq + h * p.G + g : -1;
      const int64_t row = static_cast<int64_t>(place) * parts * p.tile_rows + (out[u] < 0 ? 0 : t / TQ * 128 + t % TQ * p.G + g);
      lse[u] = p.part_lse + row;
      o[u] = p.part_o + row * D + lane * V;
      top[u] = kNone;
      sum[u] = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) acc[u][i] = 0.f;
    }
    for (int k = 0; k < parts; ++k)
#pragma unroll
      for (int u = 0; u < U; ++u) top[u] = fmaxf(top[u], __ldcg(lse[u] + k * p.tile_rows));
#pragma unroll 2
    for (int k = 0; k < parts; ++k) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float w = ex2(__ldcg(lse[u] + k * p.tile_rows) - top[u]);
        const float* src = o[u] + static_cast<int64_t>(k) * p.tile_rows * D;
        float v[V];
        if constexpr (V == 2) {
          const float2 x = __ldcg(reinterpret_cast<const float2*>(src));
          v[0] = x.x, v[1] = x.y;
        } else {
#pragma unroll
          for (int i = 0; i < V; i += 4) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(src + i));
            v[i] = x.x, v[i + 1] = x.y, v[i + 2] = x.z, v[i + 3] = x.w;
          }
        }
        sum[u] += w;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[u][i] += w * v[i];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (out[u] < 0) continue;
      const float inv = sum[u] == 0.f ? 0.f : 1.f / sum[u];
#pragma unroll
      for (int i = 0; i < V; i += 2)
        *reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + out[u] * D + lane * V + i) =
            Elt<T>::from_f2(acc[u][i] * inv, acc[u][i + 1] * inv);
      if (lane == 0 && p.lse) p.lse[out[u]] = sum[u] == 0.f ? -INFINITY : (top[u] + log2f(sum[u])) * kLn2;
    }
  }
}

// One slice of one item: an item for each token, kv head and chunk of heads, or (listed) for those of the
// tokens that small_indptr counts.
template <typename T, int D, int NT>
__device__ __forceinline__ void attend_item(const BlockParams& p, unsigned work, int slices, uint8_t* smem,
                                            int (&count_s)[2][kWarps], int* last_s) {
  using C = Cfg<D, NT>;
  constexpr int CH = D / 8, RPI = 32 / CH;  // 16-byte pieces of a row; rows that a warp copies at a time
  constexpr int KS = D / 16;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  const int chunks = (p.G + C::ROWS - 1) / C::ROWS;
  const int slice = work % slices, item = work / slices;
  const int chunk = item % chunks, h = item / chunks % p.g.Hkv;
  int t = item / (chunks * p.g.Hkv), guess = t;
  if (p.listed) {
    guess = last_below(p.small_indptr, p.batch + 1, t);
    t = p.qo_indptr[guess] + t - p.small_indptr[guess];
  }
  const int heads = min(C::ROWS, p.G - chunk * C::ROWS);
  int32_t* list = reinterpret_cast<int32_t*>(smem + C::SMEM);

  // ---- the list: page ids of the blocks that the query sees, its own block marked by the top bit
  const int32_t* blocks = p.blocks + (static_cast<int64_t>(t) * p.g.Hkv + h) * p.num_blocks;
  int e = tid < p.num_blocks ? blocks[tid] : -1;  // (in flight beside the tables)
  int before = tid > 0 && tid < p.num_blocks ? blocks[tid - 1] : e - 1;
  const Query mine = find_query(p, t, guess);
  if (!mine.there) return;
  const int64_t q_row = static_cast<int64_t>(t) * p.Hq + h * p.G + chunk * C::ROWS;  // in out and lse
  uint32_t qf[NT][KS][2];
  {
    const T* q = static_cast<const T*>(p.q) + t * p.q_stride + (static_cast<int64_t>(h) * p.G + chunk * C::ROWS) * D;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const bool real = n * 8 + g < heads;
      const uint32_t* row = reinterpret_cast<const uint32_t*>(q + (real ? n * 8 + g : 0) * D) + t4;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qf[n][k][0] = real ? row[k * 8] : 0u;
        qf[n][k][1] = real ? row[k * 8 + 4] : 0u;
      }
    }
  }
  const int own = mine.pos < 0 ? -1 : mine.pos >> p.g.ps_shift, limit = mine.pos & (p.g.ps - 1);
  int count = 0;
  bool sound = true;
  for (int i0 = 0, turn = 0; i0 < p.num_blocks; i0 += kThreads, turn ^= 1) {
    if (i0) {
      e = i0 + tid < p.num_blocks ? blocks[i0 + tid] : -1;
      before = i0 + tid < p.num_blocks ? blocks[i0 + tid - 1] : -1;
    }
    if (e >= 0 && (e <= before || (before < 0 && i0 + tid > 0))) sound = false;
    if (e >= mine.pages) atomicOr(p.status, PA_DEV_BAD_INDEX);
    const bool seen = e >= 0 && e <= own;
    const int id = seen ? page_of(p, mine.page_start + e) : 0;
    const unsigned m = __ballot_sync(0xffffffffu, seen);
    if (lane == 0) count_s[turn][warp] = __popc(m);
    __syncthreads();
    int at = count + __popc(m & ((1u << lane) - 1));
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += count_s[turn][w];
      count += count_s[turn][w];
    }
    if (seen) list[at] = id | (e == own ? INT_MIN : 0);
  }
  // a list out of order, or a request longer than it may be: as an empty list
  if (__syncthreads_or(!sound || own >= p.max_pages)) {
    if (tid == 0) atomicOr(p.status, own >= p.max_pages ? PA_DEV_NO_ROOM : PA_DEV_BAD_INDEX);
    count = 0;
  }
  const int lo = static_cast<int>(static_cast<int64_t>(count) * slice / slices);
  const int entries = static_cast<int>(static_cast<int64_t>(count) * (slice + 1) / slices) - lo;
  list += lo;

  // ---- the warp's tiles
  const int keys = entries << p.g.ps_shift;
  const int pieces = (keys + 15) / 16, tiles = (pieces + C::PIECES - 1) / C::PIECES;
  const uint32_t ring = smem_u32(smem) + warp * C::RING;
  const int64_t v_off = static_cast<int64_t>(p.g.ps) * p.g.Hkv * C::ROW;
  const int64_t slot_bytes = static_cast<int64_t>(p.g.slot_rows) * C::ROW;
  const int row0 = lane / CH;  // of the rows that the lane copies, every RPI-th
  const uint8_t* data = static_cast<const uint8_t*>(p.data) + static_cast<int64_t>(h) * p.g.head_rows * C::ROW + lane % CH * 16;
  const bool whole = p.g.ps_shift >= 4;  // a piece lies in one page
  // Key i of the slice: the list's entry, and whether the query sees it.
  auto entry_of = [&](int i) { return list[min(i >> p.g.ps_shift, entries - 1)]; };
  auto seen = [&](int i, int word) { return i < keys && (word >= 0 || (i & (p.g.ps - 1)) <= limit); };
  // Of a piece in one page: its entry, and how many of its first rows the query sees.
  auto word_of = [&](int piece) { return list[min(piece, pieces - 1) >> (p.g.ps_shift - 4)]; };
  auto live_of = [&](int piece, int word) {
    return C::PIECES > 1 && piece >= pieces ? 0 : (word >= 0 ? 16 : limit + 1 - ((piece * 16) & (p.g.ps - 1)));
  };
  auto copy = [&](int tile, int stage) {
    if (tile < tiles) {
      const uint32_t chunk16 = (lane % CH) ^ row0;
#pragma unroll
      for (int m = 0; m < C::PIECES; ++m) {
        const uint32_t dst = ring + stage * C::STAGE + (m * 16 + row0) * C::ROW;
        const int piece = tile * C::PIECES + m;
        if (whole) {
          const int word = word_of(piece), slot0 = (piece * 16) & (p.g.ps - 1), live = live_of(piece, word);
          const uint8_t* k = data + static_cast<int64_t>(word & INT_MAX) * (2 * v_off) + (slot0 + row0) * slot_bytes;
          const uint8_t* v = k + v_off;
          if (live >= 16) {
#pragma unroll
            for (int i = 0; i < 16 / RPI; ++i) {
              const uint32_t at = dst + i * RPI * C::ROW + (chunk16 ^ (i * RPI & 7)) * 16;
              cp_async16(at, k + i * RPI * slot_bytes, 16);
              cp_async16(at + C::TILE * C::ROW, v + i * RPI * slot_bytes, 16);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16 / RPI; ++i) {
              const uint32_t at = dst + i * RPI * C::ROW + (chunk16 ^ (i * RPI & 7)) * 16;
              const uint32_t bytes = i * RPI + row0 < live ? 16 : 0;
              cp_async16(at, k + i * RPI * slot_bytes, bytes);
              cp_async16(at + C::TILE * C::ROW, v + i * RPI * slot_bytes, bytes);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16 / RPI; ++i) {
            const int key = piece * 16 + i * RPI + row0;
            const int word = entry_of(key);
            const uint32_t bytes = seen(key, word) ? 16 : 0;
            const uint8_t* src = data + static_cast<int64_t>(word & INT_MAX) * (2 * v_off) + (key & (p.g.ps - 1)) * slot_bytes;
            const uint32_t at = dst + i * RPI * C::ROW + (chunk16 ^ (i * RPI & 7)) * 16;
            cp_async16(at, src, bytes);
            cp_async16(at + C::TILE * C::ROW, src + v_off, bytes);
          }
        }
      }
    }
    cp_async_commit();
  };
  // Running reference m, and the score above which it is set again.
  float o[NT][KS][4], m[NT][2], l[NT][2], above[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m[n][0] = m[n][1] = kNone;
    above[n][0] = above[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][k][i] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < C::STAGES - 1; ++i) copy(warp + i * kWarps, i);
  int stage = 0;
  for (int tile = warp; tile < tiles; tile += kWarps) {
    cp_async_wait<C::STAGES - 2>();
    __syncwarp();
    copy(tile + (C::STAGES - 1) * kWarps, stage == 0 ? C::STAGES - 1 : stage - 1);
    const uint32_t at = ring + stage * C::STAGE;
    stage = stage == C::STAGES - 1 ? 0 : stage + 1;
    float s[NT][C::PIECES][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int m = 0; m < C::PIECES; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[n][m][i] = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
#pragma unroll
      for (int m = 0; m < C::PIECES; ++m) {
        uint32_t a[4];
        ldmatrix<false>(a, at + (m * 16 + (lane & 15)) * C::ROW + ((2 * k + (lane >> 4)) ^ (lane & 7)) * 16);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma<T>(s[n][m], a, qf[n][k][0], qf[n][k][1]);
      }
    }
#pragma unroll
    for (int m = 0; m < C::PIECES; ++m) {
      const int piece = tile * C::PIECES + m;
      bool see0 = true, see1 = true, masked = false;
      if (whole) {
        const int live = live_of(piece, word_of(piece));
        masked = live < 16;
        see0 = g < live, see1 = g + 8 < live;
      } else {
        const int k0 = piece * 16 + g;
        masked = true;
        see0 = seen(k0, entry_of(k0)), see1 = seen(k0 + 8, entry_of(k0 + 8));
      }
      if (masked) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[n][m][i] = (i < 2 ? see0 : see1) ? s[n][m][i] : -INFINITY;
      }
    }
    // the largest of a lane's keys for each of its heads
    auto largest = [&](int n, int i) {
      float top = fmaxf(s[n][0][i], s[n][0][i + 2]);
      if constexpr (C::PIECES > 1) top = fmaxf(top, fmaxf(s[n][1][i], s[n][1][i + 2]));
      return top;
    };
    bool over = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) over = over || largest(n, i) > above[n][i];
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float top = largest(n, i);
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
          if (top > above[n][i]) {
            const float next = __fmul_rn(top, p.scale_log2) - kHead, f = ex2(m[n][i] - next);
            above[n][i] = fabsf(next) < 0x1p20f ? top + kRise / p.scale_log2 : top;
            m[n][i] = next;
            l[n][i] *= f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              o[n][k][i] *= f;
              o[n][k][i + 2] *= f;
            }
          }
        }
      }
    }
#pragma unroll
    for (int w = 0; w < C::PIECES; ++w) {
      uint32_t b[NT][2], b_low[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float(&x)[4] = s[n][w];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = ex2(__fmul_rn(x[i], p.scale_log2) - m[n][i & 1]);
        l[n][0] += x[0] + x[2];
        l[n][1] += x[1] + x[3];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t both = first_terms<T>(x[2 * i], x[2 * i + 1]);
          const float2 r = Elt<T>::to_f2(both);
          b[n][i] = movmatrix(both);
          b_low[n][i] = movmatrix(Elt<T>::from_f2(second_term<T>(x[2 * i], r.x), second_term<T>(x[2 * i + 1], r.y)));
        }
      }
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t a[4];
        const int r = w * 16 + (lane & 7) + (lane >> 4) * 8;
        ldmatrix<true>(a, at + (C::TILE + r) * C::ROW + ((2 * k + ((lane >> 3) & 1)) ^ (lane & 7)) * 16);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma<T>(o[n][k], a, b[n][0], b[n][1]);
          mma<T>(o[n][k], a, b_low[n][0], b_low[n][1]);
        }
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();

  // ---- the warps' states, each in its ring's place
  float* state = reinterpret_cast<float*>(smem + warp * C::RING);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], d);
      const int row = n * 8 + 2 * t4 + i;
      if (g == 0) {
        state[C::ROWS * C::O_STRIDE + 2 * row] = m[n][i];
        state[C::ROWS * C::O_STRIDE + 2 * row + 1] = l[n][i];
      }
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        state[row * C::O_STRIDE + 16 * k + g] = o[n][k][i];
        state[row * C::O_STRIDE + 16 * k + g + 8] = o[n][k][i + 2];
      }
    }
  }
  __syncthreads();
  constexpr int COLS = D / 4;
  const int64_t part = p.part_base + static_cast<int64_t>(work) * C::ROWS;  // the slice's first partial row
  for (int i = tid; i < heads * COLS; i += kThreads) {
    const int row = i / COLS, col = i % COLS * 4;
    float mw[kWarps], lw[kWarps], top = kNone, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float* st = reinterpret_cast<const float*>(smem + w * C::RING) + C::ROWS * C::O_STRIDE + 2 * row;
      mw[w] = st[0];
      lw[w] = st[1];
      top = fmaxf(top, mw[w]);
    }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + w * C::RING) + row * C::O_STRIDE + col);
      const float f = ex2(mw[w] - top);
      sum += f * lw[w];
      acc.x += f * v.x, acc.y += f * v.y, acc.z += f * v.z, acc.w += f * v.w;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (slices == 1) {
      store4<T>(p.out, q_row + row, D, col, acc, inv);
      if (col == 0 && p.lse) p.lse[q_row + row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
    } else {
      *reinterpret_cast<float4*>(p.part_o + (part + row) * D + col) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      if (col == 0) p.part_lse[part + row] = sum == 0.f ? -INFINITY : top + log2f(sum);
    }
  }
  if (slices == 1) {
    __syncthreads();  // the list and the states have been read
    return;
  }

  // ---- the last slice of the item joins the parts
  __threadfence();
  __syncthreads();
  if (tid == 0) {
    *last_s = atomicAdd(p.counters + item, 1) == slices - 1;
    if (*last_s) p.counters[item] = 0;
  }
  __syncthreads();
  if (!*last_s) return;
  __threadfence();
  const int64_t first = p.part_base + static_cast<int64_t>(item) * slices * C::ROWS;
  for (int i = tid; i < heads * COLS; i += kThreads) {
    const int row = i / COLS, col = i % COLS * 4;
    float top = kNone, sum = 0.f;
    for (int k = 0; k < slices; ++k) top = fmaxf(top, __ldcg(p.part_lse + first + k * C::ROWS + row));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < slices; ++k) {
      const int64_t r = first + k * C::ROWS + row;
      const float f = ex2(__ldcg(p.part_lse + r) - top);
      const float4 v = __ldcg(reinterpret_cast<const float4*>(p.part_o + r * D + col));
      sum += f;
      acc.x += f * v.x, acc.y += f * v.y, acc.z += f * v.z, acc.w += f * v.w;
    }
    store4<T>(p.out, q_row + row, D, col, acc, sum == 0.f ? 0.f : 1.f / sum);
    if (col == 0 && p.lse) p.lse[q_row + row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
  }
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT>::CTAS) attend_kernel(const BlockParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int count_s[2][kWarps];
  __shared__ int last_s;
  pdl_wait();
  unsigned works = gridDim.x;
  int slices = p.slices;
  if (p.listed) {
    const int parts = p.small_indptr[p.batch + 1], rows = Cfg<D, NT>::ROWS;
    if (parts > 1) join_tiles<T, D>(p, parts);
    const int items = p.small_indptr[p.batch] * p.g.Hkv * ((p.G + rows - 1) / rows);
    slices = items > 0 ? max(1, min(p.slices, p.ctas / items)) : 1;
    works = unsigned(items) * slices;
  }
  for (unsigned work = blockIdx.x; work < works; work += gridDim.x)
    attend_item<T, D, NT>(p, work, slices, smem, count_s, &last_s);
}

template <typename T, int D, int NT>
cudaError_t launch_nt(const BlockParams& p, unsigned grid, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const int most = Cfg<D, NT>::SMEM + kMaxListed * 4;
  const cudaError_t e = set_smem_once(done, reinterpret_cast<const void*>(attend_kernel<T, D, NT>), most);
  if (e != cudaSuccess) return e;
  return launch_pdl(attend_kernel<T, D, NT>, grid, kThreads, Cfg<D, NT>::SMEM + p.num_blocks * 4, stream, p);
}

template <typename T>
cudaError_t launch_t(const BlockParams& p, int D, int rows, unsigned grid, cudaStream_t stream) {
  if (D == 256) return launch_nt<T, 256, 1>(p, grid, stream);
  if (D == 128) return rows == 8 ? launch_nt<T, 128, 1>(p, grid, stream) : launch_nt<T, 128, 2>(p, grid, stream);
  return rows == 8 ? launch_nt<T, 64, 1>(p, grid, stream) : launch_nt<T, 64, 2>(p, grid, stream);
}

}  // namespace

constexpr int kMaxSlices = 64;

AttendShape attend_shape(const BlockShape& s) {
  AttendShape a;
  a.rows = s.D == 256 || s.G <= 8 ? 8 : 16;
  a.chunks = (s.G + a.rows - 1) / a.rows;
  a.ctas = s.num_sms * (s.D == 256 ? 1 : 2);
  // slices of 128 keys or more (3 requests of 4096 keys 16.4 us, in one slice each 34.5)
  int64_t n = int64_t(s.num_blocks) * s.page_size / 128;
  if (n > s.num_blocks) n = s.num_blocks;
  if (n > kMaxSlices) n = kMaxSlices;
  a.slices = n < 1 ? 1 : int(n);
  return a;
}

int64_t attend_part_rows(const BlockShape& s) {
  return int64_t(s.num_sms) * 2 * 16;  // no more slices in all than CTAs that fit the card
}

cudaError_t launch_block_attention(BlockParams p, const BlockShape& s, int dtype, cudaStream_t stream) {
  const AttendShape a = attend_shape(s);
  const int64_t items = int64_t(s.num_tokens) * s.Hkv * a.chunks;
  p.slices = a.slices;
  p.ctas = a.ctas;
  int64_t grid;
  if (p.listed) {
    // how many tokens are listed the host does not know: CTAs for a full card or
    // two, slice after slice (which the kernel cuts by the number that it finds)
    grid = items * a.slices < 2 * a.ctas ? items * a.slices : 2 * a.ctas;
  } else {
    // as many slices as the card has room for CTAs
    const int64_t fit = a.ctas / items;
    p.slices = fit < 1 ? 1 : (fit < a.slices ? int(fit) : a.slices);
    grid = items * p.slices;
  }
  return dtype == PA_BF16 ? launch_t<__nv_bfloat16>(p, s.D, a.rows, unsigned(grid), stream)
                          : launch_t<__half>(p, s.D, a.rows, unsigned(grid), stream);
}

}  // namespace pa
