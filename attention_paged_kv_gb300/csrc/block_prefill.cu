// Attention over selected pages for requests of many query tokens (tcgen05).
//
// Every token of a chunk has a list of its own, but a page read for one of them
// costs the tensor cores no more for all: a key of a pair of row tiles, 256
// packed rows, takes 100 ps of the whole card, and the small-query kernel 38 for the
// key of one token and kv head.  So a CTA takes the tokens of two row tiles (256 / G of them), the union of their
// lists, and masks each row to its own list: whatever the lists share is read
// and multiplied once, and what they do not share costs less than by itself.
//
//   order_requests  (select.cu) cumulative counts of row-tile pairs and of the tokens
//                   that are left to the small-query kernel, over the requests
//   union_lists     per row-tile pair and kv head: the union of the lists, in
//                   ascending order, and for each 128 of its keys and each token
//                   a mask of 16 bits, one for 8 keys
//   attend_tiles    the attention: warps 0-3 and 4-7 the softmax of a row tile
//                   each (thread = row = TMEM lane), warp 8 copies Q and K, warp
//                   10 V (TMA, a page a lane), warp 9 issues the MMAs
//
// Items that do not fill the card are cut along their keys (order_requests); the
// single tokens' kernel, which comes last, joins their parts.
//
// What bounds it: 1000 tokens behind 7000 with 64 of 250 pages of 32 each, by
// chance, at 64 / 8 heads: 225 us, of them 214 the tiles.  The lists of 32 tokens hold
// all pages between them, so that four times the selected products are made: 1150
// TFLOP/s of these (tensor pipe 66 %), as the dense prefill kernel with its masks
// would; where all lists are alike it takes 80 us.  Each token by itself takes
// 603 us.  256 items are two waves of 152 CTAs for work of 1.7.
//
// P is rounded to the values' type (the MMA takes both operands of one type): by
// at most 2^-8 of each weight in bf16.  In fp16 the reference that is subtracted from the logits
// is set 7 below the running maximum, as the single tokens' kernel does: a weight is
// rounded by 2^-11 of it down to 2^-21 of the row's largest, below that by 2^-32 of the largest,
// and the largest stays below 2^15.  The reference is moved only when the maximum
// grows by more than 2^8.  Over many keys these roundings average out; items with a
// token of fewer than 128 keys (a prompt's first tokens, short lists) hold P in two terms of the
// type, side by side in TMEM, and multiply V twice (8 prompts of 300 tokens 84 us, with one
// term 75; longer requests as with one).
//
// A key that a row's mask leaves out is given a weight of exactly 0 by its
// exponent's addend; a NaN or an infinity of K or V reaches the tokens of its row
// tiles all the same.
#include <climits>
#include <cstring>
#include <type_traits>

#include "internal.h"
#include "paged_common.cuh"

namespace pa {
namespace {

constexpr float kLn2f = 0.6931471805599453f;
constexpr float kHead = 7.f;  // fp16: the reference below the maximum
constexpr int kUnionThreads = 256;

// ---------------------------------------------------------------------------
// unions

// words[block * W + token / 32]: the tokens that list the block.
__global__ void __launch_bounds__(kUnionThreads) union_lists_kernel(const BlockParams p) {
  extern __shared__ uint32_t words[];
  __shared__ uint32_t bad[8];
  __shared__ int warp_count[2][kUnionThreads / 32];
  __shared__ int full;  // tokens that see 128 keys or more
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tile = blockIdx.x / p.g.Hkv, h = blockIdx.x % p.g.Hkv;
  pdl_wait();
  if (tile >= p.tile_indptr[p.batch]) return;
  const int b = last_below(p.tile_indptr, p.batch + 1, tile);
  const Span r = load_span(p, b, false);
  const int q0 = (tile - p.tile_indptr[b]) * p.tile_tokens;
  const int tokens = min(p.tile_tokens, r.qo_len - q0);
  const int W = (p.tile_tokens + 31) / 32;
  int32_t* listed = reinterpret_cast<int32_t*>(words + p.max_pages * W);  // the union's blocks
  const int pos0 = r.kv_len - r.qo_len + q0;  // of the first token
  const int end = pos0 + tokens - 1;
  const int blocks = end < 0 ? 0 : min(end / p.g.ps + 1, p.max_pages);
  if (end >= 0 && end / p.g.ps + 1 > p.max_pages && tid == 0) atomicOr(p.status, PA_DEV_NO_ROOM);
  for (int i = tid; i < blocks * W; i += kUnionThreads) words[i] = 0;
  if (tid < 8) bad[tid] = 0;
  if (tid == 0) full = 0;
  __syncthreads();
  // 32 entries of a list at a time, kBatch such strips of a warp's lists in flight
  constexpr int kUnionWarps = kUnionThreads / 32, kBatch = 8;
  const int strips = (p.num_blocks + 31) / 32, mine = (tokens - warp + kUnionWarps - 1) / kUnionWarps * strips;
  for (int j0 = 0; j0 < mine; j0 += kBatch) {
    int e[kBatch], before[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int j = j0 + k, t = warp + j / strips * kUnionWarps, i = j % strips * 32 + lane;
      const int32_t* list = p.blocks + (static_cast<int64_t>(r.qo_start + q0 + t) * p.g.Hkv + h) * p.num_blocks;
      const bool there = j < mine && i < p.num_blocks;
      e[k] = there ? list[i] : -1;
      before[k] = there && lane == 0 && i > 0 ? list[i - 1] : -1;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int j = j0 + k, t = warp + j / strips * kUnionWarps, i = j % strips * 32 + lane;
      if (j >= mine) break;
      const int pos = pos0 + t, own = pos < 0 ? -1 : pos / p.g.ps;
      const int up = __shfl_up_sync(0xffffffffu, e[k], 1), last = lane ? up : before[k];
      bool sound = own < p.max_pages;
      if (e[k] >= 0) {
        if (i > 0 && (last < 0 || e[k] <= last)) sound = false;
        if (e[k] >= r.pages) atomicOr(p.status, PA_DEV_BAD_INDEX);
        if (e[k] <= own && e[k] < blocks) {
          atomicOr(words + e[k] * W + (t >> 5), 1u << (t & 31));
          if (i == 128 / p.g.ps) atomicAdd(&full, 1);  // 128 keys in the pages before it
        }
      }
      if (!__all_sync(0xffffffffu, sound) && lane == 0) {
        atomicOr(bad + (t >> 5), 1u << (t & 31));
        if (own < p.max_pages) atomicOr(p.status, PA_DEV_BAD_INDEX);
      }
    }
  }
  __syncthreads();
  // the union, in ascending order: page id and block of each entry
  const int64_t item = blockIdx.x;
  int2* entries = p.entries + item * p.max_entries;
  int count = 0, diag = INT_MAX;
  for (int i0 = 0, turn = 0; i0 < blocks; i0 += kUnionThreads, turn ^= 1) {
    const int e = i0 + tid;
    bool any = false;
    if (e < blocks)
      for (int w = 0; w < W; ++w) any = any || (words[e * W + w] & ~bad[w]) != 0;
    const unsigned m = __ballot_sync(0xffffffffu, any);
    if (lane == 0) warp_count[turn][warp] = __popc(m);
    __syncthreads();
    int at = count + __popc(m & ((1u << lane) - 1));
#pragma unroll
    for (int w = 0; w < kUnionThreads / 32; ++w) {
      if (w < warp) at += warp_count[turn][w];
      count += warp_count[turn][w];
    }
    if (any) {
      entries[at] = make_int2(page_of(p, r.page_start + e), e);
      listed[at] = e;
    }
  }
  __syncthreads();
  pdl_launch();
  // masks, and the first 128-key step with a block that some token sees in part
  const int per = 128 / p.g.ps, bits = p.g.ps / 8;
  const int steps = (count + per - 1) / per;
  const int first_own = pos0 < 0 ? 0 : pos0 / p.g.ps;
  uint16_t* masks = p.masks + item * (p.max_entries / per) * p.tile_tokens;
  for (int i = tid; i < steps * p.tile_tokens; i += kUnionThreads) {
    const int s = i / p.tile_tokens, t = i - s * p.tile_tokens;
    uint32_t m = 0;
    if (t < tokens && !(bad[t >> 5] >> (t & 31) & 1)) {
      for (int k = 0; k < per && s * per + k < count; ++k) {
        const int e = listed[s * per + k];
        if (words[e * W + (t >> 5)] >> (t & 31) & 1) m |= ((1u << bits) - 1) << (k * bits);
        if (t == 0 && e >= first_own) diag = min(diag, s);
      }
    }
    masks[i] = static_cast<uint16_t>(m);
  }
  // (where token 0 is out, its part of the masks has not looked for the diagonal)
  if (bad[0] & 1) diag = 0;
  diag = __reduce_min_sync(0xffffffffu, diag);
  __shared__ int diag_s;
  if (tid == 0) diag_s = INT_MAX;
  __syncthreads();
  if (lane == 0) atomicMin(&diag_s, diag);
  __syncthreads();
  if (tid == 0) p.items[item] = BlockItem{r.qo_start + q0, tokens, count, diag_s, pos0, r.kv_len, full < tokens, 0};
}

// ---------------------------------------------------------------------------
// attention

template <int D, int NT>
struct TileCfg {
  static_assert(NT == 1 || (NT == 2 && D <= 128), "two tiles need 2 x (128 + D) <= 512 TMEM columns");
  static constexpr int WARP_K = 4 * NT, WARP_MMA = 4 * NT + 1, WARP_V = 4 * NT + 2;
  static constexpr int THREADS = 32 * (4 * NT + 3);
  static constexpr int NKB = D / 64;                // 128-byte column blocks of a row
  static constexpr int NST = D == 64 ? 4 : (D == 128 ? 2 : 1);
  static constexpr int BLK = 128 * 128;             // one 128-row x 128-byte block
  static constexpr int TILE = NKB * BLK;            // 128 rows of Q, K or V
  static constexpr int OFF_K = NT * TILE, OFF_V = OFF_K + NST * TILE, OFF_BAR = OFF_V + NST * TILE;
  static constexpr int SMEM = OFF_BAR + 256 + 1024;  // barriers, alignment slack
  static constexpr int O_COL = NT * 128;             // TMEM: S_x at 128 x, O_x behind the S columns
  static constexpr uint32_t TMEM_COLS = NT * (128 + D) <= 256 ? 256u : 512u;
  static_assert(SMEM <= 232448, "shared memory per CTA");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Bounded waits (see mbar_wait): of a whole warp; of the MMA thread, which
// polls without being suspended; and of what is in flight when a CTA ends.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int32_t* abort_flag, int32_t* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status, PA_WAIT_LIMIT_CYCLES));
}
__device__ __forceinline__ bool spin_wait(uint64_t* bar, uint32_t parity, volatile int32_t* abort_flag, int32_t* status) {
  const uint32_t a = smem_u32(bar);
  if (mbar_test_wait(a, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (mbar_test_wait(a, parity)) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > PA_WAIT_LIMIT_CYCLES) {
      *abort_flag = 1;
      atomicOr(status, PA_DEV_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  const long long t0 = clock64();
  while (!mbar_try_wait(a, parity))
    if (clock64() - t0 > PA_WAIT_LIMIT_CYCLES) break;
}

// A row tile's softmax over all steps, by a warpgroup (thread = row = TMEM lane): what it works on,
// and what it leaves.
struct RowArgs {
  uint64_t *s_full, *p_full, *full_v;  // s_full and p_full: the row tile's
  volatile int32_t* abort_flag;
  int32_t* status;
  const int2* entries;
  const uint16_t* masks;  // the row's token's
  uint8_t* smem;
  uint32_t s_col, o_col;
  int steps, count, diag, per, ps_shift, pos, kv_len, tile_tokens, x;
  float sl2;
  bool real;
};
struct RowState {
  float m_ref, l_sum;
  bool ok;
};
// kFew: P's second terms behind the first ones.
template <typename T, int D, int NT, bool kFew>
__device__ __forceinline__ RowState softmax_rows(const RowArgs& a) {
  using C = TileCfg<D, NT>;
  constexpr int NKB = C::NKB, NST = C::NST;
  const int r = threadIdx.x & 127, lane = threadIdx.x & 31, ps = 1 << a.ps_shift;
  float m_ref = -INFINITY, l_sum = 0.f;
  bool ok = true;
  uint32_t mask = a.real && a.steps > 0 ? a.masks[0] : 0u;
  for (int j = 0; j < a.steps; ++j) {
    const uint32_t next = a.real && j + 1 < a.steps ? a.masks[(j + 1) * a.tile_tokens] : 0u;
    ok = warp_wait(a.s_full, j & 1, a.abort_flag, a.status);
    if (!ok) break;
    tc_fence_after();
    uint32_t s[128];
    tmem_ld32(a.s_col + 0, *reinterpret_cast<uint32_t(*)[32]>(s + 0));
    tmem_ld32(a.s_col + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
    tmem_ld32(a.s_col + 64, *reinterpret_cast<uint32_t(*)[32]>(s + 64));
    tmem_ld32(a.s_col + 96, *reinterpret_cast<uint32_t(*)[32]>(s + 96));
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 128; ++i) asm volatile("" : "+r"(s[i]));
    if (j >= a.diag || j == a.steps - 1) {
      // keys behind the row's position, and what no page of the step holds
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const int e = j * a.per + (c * 8 >> a.ps_shift);
        const bool there = e < a.count && (mask >> c & 1);
        const int limit = there ? a.pos + 1 - (a.entries[min(e, a.count - 1)].y * ps + (c * 8 & (ps - 1))) : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i >= limit) s[8 * c + i] = __float_as_uint(-INFINITY);
      }
    }
    float top[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      auto f = [&](int i) { return __uint_as_float(s[8 * c + i]); };
      const float v = max3(max3(f(0), f(1), f(2)), max3(f(3), f(4), f(5)), fmaxf(f(6), f(7)));
      top[c] = mask >> c & 1 ? v : -INFINITY;
    }
    float most = top[15];
#pragma unroll
    for (int c = 0; c < 5; ++c) top[c] = max3(top[3 * c], top[3 * c + 1], top[3 * c + 2]);
    most = max3(max3(top[0], top[1], top[2]), max3(top[3], top[4], most), most) * a.sl2;
    float alpha = 1.f;
    bool resc = false;
    // (references of 2^20 and more are rounded by more than 2^-4: there they follow each growth)
    const float rise = Elt<T>::kBf16 ? 8.f : (fabsf(most) < 0x1p20f ? kHead + 8.f : kHead);
    if (most > m_ref + rise) {
      const float next = Elt<T>::kBf16 ? most : most - kHead;
      if (m_ref != -INFINITY) {
        alpha = ex2(m_ref - next);
        resc = true;
      }
      m_ref = next;
    }
    const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
    const float2 sc2 = make_float2(a.sl2, a.sl2);
    float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t ph[16], pl[16];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float nm = mask >> (4 * c + u) & 1 ? -m_use : -INFINITY;
        const float2 nm2 = make_float2(nm, nm);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int i = 4 * u + v, k = 32 * c + 2 * i;
          const float2 t2 = __ffma2_rn(make_float2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), sc2, nm2);
          const float y = ex2(t2.x), z = ex2(t2.y);
          acc[u & 1] = __fadd2_rn(acc[u & 1], make_float2(y, z));
          ph[i] = Elt<T>::from_f2(y, z);
          if constexpr (kFew) {
            const float2 hi = Elt<T>::to_f2(ph[i]);
            pl[i] = Elt<T>::from_f2(y - hi.x, z - hi.y);
          }
        }
      }
      tmem_st16(a.s_col + c * 16, ph);
      if constexpr (kFew) tmem_st16(a.s_col + 64 + c * 16, pl);
    }
    const float2 sum = __fadd2_rn(acc[0], acc[1]);
    // (P V of the step before is complete: S was issued behind it)
    if (__any_sync(0xffffffffu, resc)) {
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(a.o_col + c * 32, o);
        tmem_wait_ld(o);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
        tmem_st32(a.o_col + c * 32, o);
      }
    }
    // V rows of the last step that hold no key (0 * NaN would reach O)
    if (a.x == 0 && j == a.steps - 1) {
      const int last = a.count - 1 - j * a.per;
      const int valid = last * ps + min(ps, a.kv_len - a.entries[a.count - 1].y * ps);
      if (valid < 128) {
        const int st = j % NST;
        ok = warp_wait(&a.full_v[st], (j / NST) & 1, a.abort_flag, a.status);
        if (!ok) break;
        if (r >= valid) {
          uint8_t* row = a.smem + C::OFF_V + st * C::TILE + r * 128;
#pragma unroll
          for (int kb = 0; kb < NKB; ++kb)
#pragma unroll
            for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(row + kb * C::BLK + c * 16) = make_uint4(0, 0, 0, 0);
        }
      }
    }
    l_sum = l_sum * alpha + sum.x + sum.y;
    mask = next;
    tmem_wait_st();
    fence_proxy_async_smem();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(a.p_full);
  }
  return RowState{m_ref, l_sum, ok};
}
// Not in line: the registers of both loops in one function cost the usual one 2 to 7 %.
template <typename T, int D, int NT>
__device__ __noinline__ RowState softmax_rows_of_few(const RowArgs a) {
  return softmax_rows<T, D, NT, true>(a);
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(TileCfg<D, NT>::THREADS, 1)
    attend_tiles_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap q_map,
                        const BlockParams p) {
  using C = TileCfg<D, NT>;
  constexpr int NKB = C::NKB, NST = C::NST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* full_k = bars;             // [NST] K step landed
  uint64_t* full_v = bars + NST;       // [NST]
  uint64_t* empty_k = bars + 2 * NST;  // [NST] the S MMAs are done with it
  uint64_t* empty_v = bars + 3 * NST;  // [NST] the P V MMAs are
  uint64_t* q_full = bars + 4 * NST;
  uint64_t* s_full = q_full + 1;       // [2] S_x there
  uint64_t* p_full = s_full + 2;       // [2] P_x written, O_x corrected
  uint64_t* o_done = p_full + 2;       // [2] the last P V of x done
  uint64_t* fin = o_done + 2;          // all MMAs retired
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 26);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(tmem_slot + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  // the longest tiles of a chunk, its last ones, first
  const int tiles = p.tile_indptr[p.batch], parts = p.small_indptr[p.batch + 1];
  const int place = static_cast<int>(blockIdx.x) / parts, part = static_cast<int>(blockIdx.x) - place * parts;
  const int tile = tiles - 1 - place / p.g.Hkv, h = place % p.g.Hkv;
  if (tile < 0) return;
  const int64_t item = static_cast<int64_t>(tile) * p.g.Hkv + h;
  const BlockItem it = p.items[item];
  const int G = p.G, TQ = 128 / G;  // tokens of a row tile
  const bool has_b = NT == 2 && it.tokens > TQ;
  const int per = 128 >> p.g.ps_shift;  // pages of a step
  // the part's steps of 128 keys, and what they hold of the union
  const int all_steps = (it.entries + per - 1) / per;
  const int step0 = all_steps * part / parts, steps = all_steps * (part + 1) / parts - step0;
  const int count = min(it.entries - step0 * per, steps * per), diag = it.diag - step0;
  const int2* entries = p.entries + item * p.max_entries + step0 * per;

  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full_k[i], 1);
      mbar_init(&full_v[i], 1);
      mbar_init(&empty_k[i], 1);
      mbar_init(&empty_v[i], 1);
    }
    mbar_init(q_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_done[i], 1);
    }
    mbar_init(fin, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == C::WARP_MMA) tmem_alloc(tmem_slot, C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == C::WARP_K || warp == C::WARP_V) {
    // ---------------------------------------------------------------- copies
    const int half = warp == C::WARP_V;
    uint64_t* full = half ? full_v : full_k;
    uint64_t* empty = half ? empty_v : empty_k;
    const uint32_t ring = sbase + (half ? C::OFF_V : C::OFF_K);
    // the page of lane l of a step, read two steps ahead
    auto page = [&](int j) { return lane < per && j * per + lane < count ? entries[j * per + lane].x : 0; };
    if (!half && lane == 0 && steps > 0) {
      mbar_arrive_expect_tx(q_full, uint32_t((has_b ? 2 : 1) * NKB * TQ * G * 128));
#pragma unroll
      for (int kb = 0; kb < NKB; ++kb) {
        tma_load_3d(sbase + kb * C::BLK, &q_map, kb * 64, h * G, it.token, q_full);
        if (has_b) tma_load_3d(sbase + C::TILE + kb * C::BLK, &q_map, kb * 64, h * G, it.token + TQ, q_full);
      }
    }
    int id0 = page(0), id1 = page(1), issued = 0;
    bool ok = true;
    for (int j = 0; j < steps; ++j) {
      const int st = j % NST, id = id0;
      id0 = id1;
      id1 = page(j + 2);
      if (j >= NST) {
        if (lane == 0) ok = mbar_wait(&empty[st], ((j / NST) - 1) & 1, abort_flag, p.status, PA_WAIT_LIMIT_CYCLES);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
      }
      const int n = min(per, count - j * per);
      if (lane == 0) mbar_arrive_expect_tx(&full[st], uint32_t(n * p.g.ps * 128 * NKB));
      __syncwarp();
      if (lane < n) {
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb)
          tma_kv_rows(ring + st * C::TILE + kb * C::BLK + lane * p.g.ps * 128, &kv_map, kb * 64, h, 0, 2 * id + half,
                      &full[st], p.hnd);
      }
      issued = j + 1;
    }
    // copies in flight land before the CTA's memory goes away
    if (lane == 0) {
      if (!half && steps > 0) drain_wait(q_full, 0);
      for (int j = max(0, issued - NST); j < issued; ++j) drain_wait(&full[j % NST], (j / NST) & 1);
    }
    __syncwarp();
  } else if (warp == C::WARP_MMA) {
    // ---------------------------------------------------------------- MMAs
    if (lane == 0 && steps > 0) {
      const uint32_t id_s = idesc_f16(Elt<T>::kBf16, 0, 0, 128, 128);
      const uint32_t id_o = idesc_f16(Elt<T>::kBf16, 0, 1, 128, D);
      const uint64_t dq0 = smem_desc_sw128(sbase, 16, 1024);
      const uint64_t dk0 = smem_desc_sw128(sbase + C::OFF_K, 16, 1024);
      const uint64_t dv0 = smem_desc_sw128(sbase + C::OFF_V, C::BLK, 1024);
      auto issue_s = [&](int x, int st) {
        const uint64_t qd = dq0 + uint64_t(x) * (C::TILE >> 4), kd = dk0 + uint64_t(st) * (C::TILE >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * C::BLK + (k & 3) * 32) >> 4;
          tc_mma_ss(tmem + x * 128, qd + off, kd + off, id_s, k > 0 ? 1u : 0u);
        }
        tc_commit(&s_full[x]);
      };
      auto issue_pv = [&](int x, int j, int st, auto few) {
        const uint64_t vd = dv0 + uint64_t(st) * (C::TILE >> 4);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          tc_mma_ts(tmem + C::O_COL + x * 128, tmem + x * 128 + k * 8, vd + (k * 2048 >> 4), id_o, (j > 0 || k > 0) ? 1u : 0u);
        if constexpr (decltype(few)::value) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            tc_mma_ts(tmem + C::O_COL + x * 128, tmem + x * 128 + 64 + k * 8, vd + (k * 2048 >> 4), id_o, 1u);
        }
        if (j == steps - 1) tc_commit(&o_done[x]);
      };
      bool ok = spin_wait(q_full, 0, abort_flag, p.status);
      if (ok) ok = spin_wait(&full_k[0], 0, abort_flag, p.status);
      if (ok) {
        tc_fence_after();
        issue_s(0, 0);
        if (has_b) issue_s(1, 0);
        tc_commit(&empty_k[0]);
      }
      auto run = [&](auto few) {
        for (int j = 0; ok && j < steps; ++j) {
          const int st = j % NST, st1 = (j + 1) % NST;
          const bool more = j + 1 < steps;
          ok = spin_wait(&p_full[0], j & 1, abort_flag, p.status);
          if (ok) ok = spin_wait(&full_v[st], (j / NST) & 1, abort_flag, p.status);
          if (!ok) break;
          tc_fence_after();
          issue_pv(0, j, st, few);
          if (more) {
            ok = spin_wait(&full_k[st1], ((j + 1) / NST) & 1, abort_flag, p.status);
            if (!ok) break;
            tc_fence_after();
            issue_s(0, st1);
            if (!has_b) tc_commit(&empty_k[st1]);
          }
          if (has_b) {
            ok = spin_wait(&p_full[1], j & 1, abort_flag, p.status);
            if (!ok) break;
            tc_fence_after();
            issue_pv(1, j, st, few);
          }
          tc_commit(&empty_v[st]);
          if (has_b && more) {
            issue_s(1, st1);
            tc_commit(&empty_k[st1]);
          }
        }
      };
      if (it.few) run(std::true_type{});
      else run(std::false_type{});
      tc_commit(fin);
      drain_wait(fin, 0);
    }
    __syncwarp();
  } else if ((warp >> 2) == 0 || has_b) {
    // ---------------------------------------------------------------- softmax
    const int x = warp >> 2, r = tid & 127;
    const int t_local = r / G, g = r - t_local * G, t = x * TQ + t_local;  // token of the item
    const bool real = t_local < TQ && t < it.tokens;
    const int pos = it.pos + t;
    const uint16_t* masks = p.masks + (item * (p.max_entries / per) + step0) * p.tile_tokens + (real ? t : 0);
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lane_base + x * 128, o_col = tmem + lane_base + C::O_COL + x * 128;
    const RowArgs args{&s_full[x], &p_full[x], full_v, abort_flag, p.status, entries, masks, smem, s_col, o_col, steps, count,
                       diag, per, p.g.ps_shift, pos, it.kv_len, p.tile_tokens, x, p.scale_log2, real};
    const RowState state = it.few ? softmax_rows_of_few<T, D, NT>(args) : softmax_rows<T, D, NT, false>(args);
    const float m_ref = state.m_ref, l_sum = state.l_sum;
    bool ok = state.ok;
    if (ok && steps > 0) ok = warp_wait(&o_done[x], 0, abort_flag, p.status);
    pdl_launch();
    if (ok) {
      tc_fence_after();
      const float inv = l_sum == 0.f ? 0.f : 1.f / l_sum;
      const int64_t row0 = static_cast<int64_t>(it.token) * p.Hq + static_cast<int64_t>(h) * G;
      auto column = [&](int c4, uint32_t(&o)[32]) {  // 32 of the row's values
        if (steps > 0) {
          tmem_ld32(o_col + c4 * 32, o);
          tmem_wait_ld(o);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0;
        }
      };
      if (parts > 1) {  // a part's state: normalised, in fp32, with its log-sum in base 2
        const int64_t row = (static_cast<int64_t>(place) * parts + part) * (NT * 128) + x * 128 + r;
        if (real) p.part_lse[row] = l_sum == 0.f ? -INFINITY : m_ref + log2f(l_sum);
        // 64 columns at a time (32 at head_dim 64) through the warp's Q rows, free by
        // now, to leave in whole rows
        constexpr int TURN = D == 64 ? 32 : 64, BYTES = TURN * 4, LANES = TURN / 4;
        static_assert(4 * 32 * BYTES <= C::TILE, "four warps' rows fit a Q tile");
        uint8_t* own = smem + x * C::TILE + (warp & 3) * 32 * BYTES;
#pragma unroll
        for (int turn = 0; turn < D / TURN; ++turn) {
#pragma unroll
          for (int c4 = 0; c4 < TURN / 32; ++c4) {
            uint32_t o[32];
            column(turn * (TURN / 32) + c4, o);
#pragma unroll
            for (int v = 0; v < 8; ++v) {
              auto f = [&](int i) { return l_sum == 0.f ? 0.f : __uint_as_float(o[4 * v + i]) * inv; };
              *reinterpret_cast<float4*>(own + lane * BYTES + (((c4 * 8 + v) ^ (lane & 7)) << 4)) = make_float4(f(0), f(1), f(2), f(3));
            }
          }
          __syncwarp();
          const int c = lane % LANES;
#pragma unroll 4
          for (int i = lane / LANES; i < 32; i += 32 / LANES)
            *reinterpret_cast<float4*>(p.part_o + (row - lane + i) * D + turn * TURN + c * 4) =
                *reinterpret_cast<const float4*>(own + i * BYTES + ((c ^ (i & 7)) << 4));
          __syncwarp();
        }
      } else {
        if (real && p.lse)
          p.lse[row0 + static_cast<int64_t>(t) * p.Hq + g] =
              l_sum == 0.f ? -INFINITY : ((m_ref == -INFINITY ? 0.f : m_ref) + log2f(l_sum)) * kLn2f;
        // through the row tile's Q memory (free by now), whole rows at a time
        uint8_t* own = smem + x * C::TILE + r * 128;
#pragma unroll
        for (int c4 = 0; c4 < D / 32; ++c4) {
          uint32_t o[32];
          column(c4, o);
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int c = (c4 & 1) * 4 + v;
            auto f = [&](int i) { return __uint_as_float(o[8 * v + i]) * inv; };
            *reinterpret_cast<uint4*>(own + (c4 >> 1) * C::BLK + ((c ^ (r & 7)) << 4)) =
                l_sum == 0.f ? make_uint4(0, 0, 0, 0)
                             : make_uint4(Elt<T>::from_f2(f(0), f(1)), Elt<T>::from_f2(f(2), f(3)), Elt<T>::from_f2(f(4), f(5)),
                                          Elt<T>::from_f2(f(6), f(7)));
          }
        }
        __syncwarp();
        constexpr int LANES = D / 8;  // of a row
#pragma unroll 4
        for (int i = lane / LANES; i < 32; i += 32 / LANES) {
          const int rr = (warp & 3) * 32 + i, tl = rr / G, c = lane % LANES;
          if (tl < TQ && x * TQ + tl < it.tokens) {
            const uint4 w = *reinterpret_cast<const uint4*>(smem + x * C::TILE + (c >> 3) * C::BLK + rr * 128 + (((c & 7) ^ (rr & 7)) << 4));
            const int64_t row = row0 + static_cast<int64_t>(x * TQ + tl) * p.Hq + (rr - tl * G);
            *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + row * D + c * 8) = w;
          }
        }
      }
    }
  }
  // ---------------------------------------------------------------- the end
  if (warp < C::WARP_K) tmem_wait_st();
  tc_fence_before();
  __syncthreads();
  if (warp == C::WARP_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <typename T, int D, int NT>
cudaError_t launch_tiles(const CUtensorMap& kv_map, const CUtensorMap& q_map, const BlockParams& p, unsigned grid,
                         cudaStream_t stream) {
  using C = TileCfg<D, NT>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = set_smem_once(done, reinterpret_cast<const void*>(attend_tiles_kernel<T, D, NT>), C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(attend_tiles_kernel<T, D, NT>, grid, unsigned(C::THREADS), size_t(C::SMEM), stream, kv_map, q_map, p);
}
template <typename T>
cudaError_t launch_t(const CUtensorMap& kv_map, const CUtensorMap& q_map, const BlockParams& p, int D, unsigned grid,
                     cudaStream_t stream) {
  if (D == 64) return launch_tiles<T, 64, 2>(kv_map, q_map, p, grid, stream);
  if (D == 128) return launch_tiles<T, 128, 2>(kv_map, q_map, p, grid, stream);
  return launch_tiles<T, 256, 1>(kv_map, q_map, p, grid, stream);
}

}  // namespace

TileShape tile_shape(const BlockShape& s) {
  TileShape t;
  t.tokens = (s.D == 256 ? 1 : 2) * (128 / s.G);
  t.long_tokens = 32 / s.G + 1 > 2 ? 32 / s.G + 1 : 2;
  t.rows = (s.D == 256 ? 1 : 2) * 128;
  // A million keys of single tokens and kv heads: 64 tokens of 2048 keys at 8 kv
  // heads take 47 us in tiles (32 where their lists are alike) and 46 by
  // themselves, 32 tokens 43 (32) and 24, 128 tokens 63 (37) and 91.  That is behind 8000
  // keys.  The union grows with the keys, which the rule leaves out: 1000 tokens behind 32000,
  // 64000 and 128000 take 764, 1113 and 1385 us in tiles and 643, 798 and 958 by themselves where
  // lists are by chance; by the selection, of keys around a centre of their page, 494, 652 and 825 against 621,
  // 630 and 653; alike 90, 93 and 101 against 600.
  t.least_long = int32_t((1 << 20) / (int64_t(s.Hkv) * s.num_blocks * s.page_size) + 1);
  const int words = (t.tokens + 31) / 32;
  t.union_smem = int64_t(s.max_pages) * (words + 1) * 4;
  // pages of 8 slots or more (a TMA copy's rows keep the swizzle's period of 8),
  // and unions that shared memory holds (1000 tokens of 8 / 8 heads, 5688 pages and room for one
  // more: behind 32000 keys, by chance, 321 us and by themselves 622; behind 90000, by the selection, 707 and 780)
  t.use = s.max_qo_len >= t.long_tokens && s.num_tokens >= t.least_long && s.page_size >= 8 && t.union_smem <= 200 * 1024;
  if (!t.use) {
    t.max_tiles = t.max_entries = 0;
    return t;
  }
  const int64_t tokens = s.num_tokens, longs = tokens / t.long_tokens < s.batch ? tokens / t.long_tokens : s.batch;
  t.max_tiles = int32_t(tokens / t.tokens + longs);
  const int64_t most = int64_t(t.tokens) * s.num_blocks < s.max_pages ? int64_t(t.tokens) * s.num_blocks : s.max_pages;
  const int per = 128 / s.page_size;
  t.max_entries = int32_t((most + per - 1) / per * per);
  return t;
}

cudaError_t launch_block_tiles(BlockParams p, const BlockShape& s, const TileShape& t, const CUtensorMap& kv_map,
                               const CUtensorMap& q_map, int dtype, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = launch_order_requests(p, stream);
  if (e != cudaSuccess) return e;
  e = set_smem_once(done, reinterpret_cast<const void*>(union_lists_kernel), 200 * 1024);
  if (e != cudaSuccess) return e;
  const unsigned grid = unsigned(t.max_tiles) * unsigned(s.Hkv);
  if (grid == 0) return cudaSuccess;
  e = launch_pdl(union_lists_kernel, grid, unsigned(kUnionThreads), size_t(t.union_smem), stream, p);
  if (e != cudaSuccess) return e;
  // where items are few, up to two CTAs an SM for their parts
  const unsigned ctas = grid > 2u * s.num_sms ? grid : 2u * s.num_sms;
  return dtype == PA_BF16 ? launch_t<__nv_bfloat16>(kv_map, q_map, p, s.D, ctas, stream)
                          : launch_t<__half>(kv_map, q_map, p, s.D, ctas, stream);
}

}  // namespace pa
