// The pages that a query attends to (pagedattn_select_blocks).
//
// Score of a page for token t and kv head h, from the page's 8-bit bounds:
//   sum over channels of (c_u * largest + c_l * smallest), times the page's scale
// with c_u, c_l the group's summed positive and negative parts of q in 8 bits.
// The sums are of whole numbers, so they come out alike in any order, and the
// selection does not depend on how the work is cut.
//
// Single tokens: a CTA takes one query and kv head, or a slice of its pages where
// there are few of them; scores go to a scratch row as unsigned keys in their
// order, and the last slice to finish selects.  The k-th largest key is found by
// histograms over 2048 equal parts of the keys' range, then of the part that
// holds it, until one key (or a part taken whole) is left.
//
// Chunks: a CTA takes 16 tokens of a request, whose scores for 8 pages at a time
// are m16n8k32 products of 8-bit integers: the bounds are read once for all.
// Each warp then selects for tokens by itself, from keys in shared memory: a
// histogram over 256 parts, and the ranks of the keys of the part that holds the border.
//
// What bounds them.  64 decodes of 512 to 8192 keys (pages of 16, 8 kv heads, 34
// MB): 13.7 us, 5 at the copy rate; the rest is one dependent load after the
// other (tables, page ids, bounds) and the CTA's barriers.  A chunk of 2000
// tokens over 500 pages: 58 us, in two rounds of CTAs; in each, codes of q 3.6
// us, scores 10.4 (8-bit products: 36 cycles of a sub-partition each), the
// selection 8.6 (its instructions).  Measured without gain there: products in
// fp16 (bounds converted, 62), bounds loaded a step ahead (registers for two CTAs
// an SM: 79), scores and ranking in warps of their own a tile apart (72).
#include <cfloat>
#include <cstring>

#include "internal.h"
#include "paged_common.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kKept = kKeptKeys;
constexpr int kTileSmem = 100 * 1024;  // of a chunk's keys: two CTAs an SM
constexpr uint32_t kAlways = 0xFFFFFFFFu;  // above every score's key

// Scores as unsigned numbers of the same order; -0 is 0, NaN is infinity.
__device__ __forceinline__ uint32_t order_key(float s) {
  s = s != s ? INFINITY : s + 0.f;
  const uint32_t b = __float_as_uint(s);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The codes of the group's q: 2 * D bytes, c_u then c_l, made by a warp.
template <typename T, int D>
__device__ __forceinline__ void query_codes(const T* q, int G, int8_t* codes) {
  constexpr int LANES = D / 8, ROWS = 32 / LANES;
  constexpr int HELD = 4;  // rows of a lane that are kept between the two passes
  const int lane = threadIdx.x & 31, r = lane / LANES, c = lane % LANES;
  auto row = [&](int g) { return __ldg(reinterpret_cast<const uint4*>(q + g * D + c * 8)); };
  uint4 held[HELD];
#pragma unroll
  for (int i = 0; i < HELD; ++i) held[i] = r + i * ROWS < G ? row(r + i * ROWS) : make_uint4(0, 0, 0, 0);
  uint32_t top = 0;
  auto look = [&](const uint4& v) {
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                 __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
  };
#pragma unroll
  for (int i = 0; i < HELD; ++i) look(held[i]);
  for (int g = r + HELD * ROWS; g < G; g += ROWS) look(row(g));
  // magnitudes have the order of their bits
  top = __reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16));
  const float most = Elt<T>::to_f2(top).x;
  // sums of the values and of their magnitudes: u = (size + sum) / 2, l = (sum - size) / 2
  float sum[8], size[8], u[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = size[i] = 0.f;
  if (most > 0.f && most < INFINITY) {
    int e;
    frexpf(most, &e);
    e = 15 - e;
    // x * 2^e rounded to a whole number (to even): its size is at most 2^15, so
    // 3 * 2^22 added and taken away again does it.  2^e may pass fp32's range: in two steps.
    const float f1 = pow2f(e / 2), f2 = pow2f(e - e / 2);
    auto whole = [&](float x) { return fmaf(x * f1, f2, 12582912.f) - 12582912.f; };
    auto add = [&](const uint4& v) {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = Elt<T>::to_f2(w[i]);
        const float a = whole(x.x), b = whole(x.y);
        sum[2 * i] += a, size[2 * i] += fabsf(a);
        sum[2 * i + 1] += b, size[2 * i + 1] += fabsf(b);
      }
    };
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      if (i * ROWS < G) add(held[i]);
    for (int g = r + HELD * ROWS; g < G; g += ROWS) add(row(g));
  }
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int d = LANES; d < 32; d <<= 1) {
      sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], d);  // whole numbers up to 2^22: exact
      size[i] += __shfl_xor_sync(0xffffffffu, size[i], d);
    }
    u[i] = 0.5f * (size[i] + sum[i]);
    l[i] = 0.5f * (sum[i] - size[i]);
    m = fmaxf(m, fmaxf(u[i], -l[i]));
  }
  m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));  // (not negative: in the order of its bits)
  const float f = m > 0.f ? 127.f * __frcp_rn(m) : 0.f;
  if (lane < LANES) {
    uint32_t cu[2] = {0, 0}, cl[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cu[i >> 2] |= (static_cast<uint32_t>(static_cast<int>(rintf(u[i] * f))) & 0xFFu) << (8 * (i & 3));
      cl[i >> 2] |= (static_cast<uint32_t>(static_cast<int>(rintf(l[i] * f))) & 0xFFu) << (8 * (i & 3));
    }
    *reinterpret_cast<uint2*>(codes + c * 8) = make_uint2(cu[0], cu[1]);
    *reinterpret_cast<uint2*>(codes + D + c * 8) = make_uint2(cl[0], cl[1]);
  }
}

struct Scan {
  int warp_sum[kWarps];
};
// Exclusive sum over the CTA's threads, and the total.
__device__ __forceinline__ int sum_before(int v, int* all, Scan& s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 31) s.warp_sum[warp] = x;
  __syncthreads();
  int before = x - v, sum = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s.warp_sum[w];
    sum += s.warp_sum[w];
  }
  *all = sum;
  return before;
}

// The k largest of n > k keys, of equal ones the first, as ascending indices.
template <typename Key>
__device__ void select_largest(Key key, int n, int k, int32_t* out, int* bins, Scan& scan, uint32_t* range) {
  const int tid = threadIdx.x;
  // the range of the keys that are not always taken
  uint32_t least = 0xFFFFFFFFu, most = 0;
  int always = 0;
  for (int i = tid; i < n; i += kThreads) {
    const uint32_t x = key(i);
    if (x == kAlways) {
      ++always;
    } else {
      least = min(least, x);
      most = max(most, x);
    }
  }
  least = __reduce_min_sync(0xffffffffu, least);
  most = __reduce_max_sync(0xffffffffu, most);
  if (tid == 0) {
    range[0] = 0xFFFFFFFFu;
    range[1] = 0;
  }
  int forced;
  sum_before(always, &forced, scan);
  if ((tid & 31) == 0) {
    atomicMin(range, least);
    atomicMax(range + 1, most);
  }
  __syncthreads();
  uint32_t base = range[0];
  int need = k - forced;  // of the keys at or above `base` and below `top`; all above are taken
  uint64_t top = static_cast<uint64_t>(range[1]) + 1;
  while (need > 0 && top - base > 1) {
    // parts of 2^shift keys each
    const uint32_t span = static_cast<uint32_t>(top - 1 - base);
    const int shift = max(0, 32 - __clz(span) - 11);
    for (int i = tid; i < kBins; i += kThreads) bins[i] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      const uint32_t x = key(i);
      if (x >= base && x < top) atomicAdd(bins + ((x - base) >> shift), 1);
    }
    __syncthreads();
    // the part that holds the need-th largest, seen from above
    int mine[kBins / kThreads], sum = 0;
#pragma unroll
    for (int i = 0; i < kBins / kThreads; ++i) {
      mine[i] = bins[kBins - 1 - (tid * (kBins / kThreads) + i)];
      sum += mine[i];
    }
    int all, above = sum_before(sum, &all, scan);
#pragma unroll
    for (int i = 0; i < kBins / kThreads; ++i) {
      if (above < need && above + mine[i] >= need) {
        range[0] = kBins - 1 - (tid * (kBins / kThreads) + i);
        range[1] = need - above;  // still to take from this part
        range[2] = mine[i];
      }
      above += mine[i];
    }
    __syncthreads();
    const uint32_t part = range[0];
    need = range[1];
    const bool whole = need == static_cast<int>(range[2]);
    const uint64_t end = static_cast<uint64_t>(base) + ((static_cast<uint64_t>(part) + 1) << shift);
    base += part << shift;
    top = min(top, end);
    if (whole) {  // all of the part: everything from `base` on is taken
      top = base;
      need = 0;
    }
    __syncthreads();
  }
  // Now: keys >= top are taken, and of those equal to base (if top > base) the
  // first `need`.
  const int run = ((n + kThreads - 1) / kThreads) | 1;  // odd: no two threads' keys in one bank
  const int from = min(tid * run, n), to = min(from + run, n);
  int equal = 0, over = 0;
  for (int i = from; i < to; ++i) {
    const uint32_t x = key(i);
    if (x >= top) ++over;
    else if (x == base) ++equal;
  }
  int all;
  int equal_before = sum_before(equal, &all, scan);
  int taken = over + max(0, min(equal, need - equal_before));
  int at = sum_before(taken, &all, scan);
  for (int i = from; i < to; ++i) {
    const uint32_t x = key(i);
    bool take = x >= top;
    if (!take && x == base) take = equal_before++ < need;
    if (take) out[at++] = i;
  }
}

// One CTA: tile_indptr and small_indptr, [batch + 1] each, and the parts that
// an item's keys are cut into.  Where the long requests have fewer than
// least_long tokens in all, they are left to the kernel of single tokens.
__global__ void __launch_bounds__(1024) order_requests_kernel(const BlockParams p) {
  __shared__ int sums[2][32];
  __shared__ long long long_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) long_s = 0;
  __syncthreads();
  pdl_launch();  // (the next kernel's CTAs may take their places)
  pdl_wait();
  // (tokens and tiles are fewer than 2^30: limited to that, the sum of two counts fits 32 bits,
  // of requests that overlap too, in tables that cannot be)
  constexpr int kMost = (1 << 30) - 1;
  int mine = 0;
  for (int b = tid; b < p.batch; b += 1024) {
    const int n = load_span(p, b, true).qo_len;
    if (n >= p.long_tokens) mine = min(mine + n, kMost);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) mine = min(mine + __shfl_xor_sync(0xffffffffu, mine, d), kMost);
  if (lane == 0 && mine) atomicAdd(reinterpret_cast<unsigned long long*>(&long_s), static_cast<unsigned long long>(mine));
  __syncthreads();
  const int long_tokens = long_s < p.least_long ? INT_MAX : p.long_tokens;
  int base_t = 0, base_s = 0;
  if (tid == 0) p.tile_indptr[0] = p.small_indptr[0] = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 1024) {
    const int b = b0 + tid;
    int tiles = 0, small = 0;
    if (b < p.batch) {
      const int n = load_span(p, b, false).qo_len;
      if (n >= long_tokens) tiles = min((n + p.tile_tokens - 1) / p.tile_tokens, p.max_tiles);
      else small = n;
    }
    int t = tiles, s = small;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, t, d), c = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) t = min(t + a, p.max_tiles), s = min(s + c, p.num_tokens);
    }
    __syncthreads();
    if (lane == 31) sums[0][warp] = t, sums[1][warp] = s;
    __syncthreads();
    int all_t = 0, all_s = 0;
    // (requests that overlap may have more tiles than there is room for: what is past
    // it is left out)
    for (int w = 0; w < 32; ++w) {
      if (w < warp) t = min(t + sums[0][w], p.max_tiles), s = min(s + sums[1][w], p.num_tokens);
      all_t = min(all_t + sums[0][w], p.max_tiles), all_s = min(all_s + sums[1][w], p.num_tokens);
    }
    if (b < p.batch) {
      p.tile_indptr[b + 1] = min(base_t + t, p.max_tiles);
      p.small_indptr[b + 1] = min(base_s + s, p.num_tokens);
    }
    base_t = min(base_t + all_t, p.max_tiles);
    base_s = min(base_s + all_s, p.num_tokens);
  }
  if (tid == 0) {
    // Parts of an item: the number that gives the shortest run.  In units of an item
    // (85 us for 8000 keys): whole waves of parts, a part's start and end, and
    // the join of all parts' states.  1000 tokens behind 7000, us: 1 kv head (32 items)
    // whole 127, in 2 parts 85, 4 60, 8 (two waves) 69; 2 kv heads 130, 92, 97 (4);
    // 800 at 4 kv heads (100 items) 129, 148, 123 (3).
    const int items = base_t * p.g.Hkv;
    int parts = 1;
    float best = 3.0e38f;
    for (int n = 1; n <= kMaxParts && (n == 1 || items * n <= 2 * p.num_sms); ++n) {
      const float cost = static_cast<float>((items * n + p.num_sms - 1) / p.num_sms) * (1.f / n + 0.07f) +
                         (n > 1 ? static_cast<float>(items * n) * 0.0006f : 0.f);
      if (cost < best) best = cost, parts = n;
    }
    p.small_indptr[p.batch + 1] = parts;
  }
}

template <int D>
struct SelectShared {
  __align__(16) int8_t codes[kWarps][2 * D];
  int bins[kBins];
  Scan scan;
  uint32_t range[3];
  int last;
};

// One slice of one item: an item for each token and kv head, or (listed) for those of the tokens that
// small_indptr counts.  kept: the item's keys.
template <typename T, int D>
__device__ __forceinline__ void select_item(const BlockParams& p, unsigned work, int slices, uint32_t* kept,
                                            SelectShared<D>& sh) {
  constexpr int LPR = D / 32, RPW = 32 / LPR;  // lanes of a page's bounds, 64 bytes each; pages of a warp
  constexpr int U = D == 256 ? 4 : 2;  // 16 pages or more of a warp in flight
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int item = work / slices, slice = work % slices;
  const int h = item % p.g.Hkv;
  int t = p.token0 + item / p.g.Hkv, guess = t;
  if (p.listed) {
    guess = last_below(p.small_indptr, p.batch + 1, t);
    t = p.qo_indptr[guess] + t - p.small_indptr[guess];
  }
  const Query mine = find_query(p, t, guess);
  if (!mine.there) return;
  const int n = mine.pos < 0 ? 0 : mine.pos / p.g.ps + 1;
  int32_t* out = p.blocks + (static_cast<int64_t>(t) * p.g.Hkv + h) * p.num_blocks;
  if (n <= p.num_blocks || n > p.max_pages) {
    if (slice == 0)
      for (int i = tid; i < p.num_blocks; i += kThreads) out[i] = i < n && n <= p.max_pages ? i : -1;
    if (n > p.max_pages && tid == 0) atomicOr(p.status, PA_DEV_NO_ROOM);
    return;
  }
  const int lo = static_cast<int>(static_cast<int64_t>(n) * slice / slices);
  const int hi = static_cast<int>(static_cast<int64_t>(n) * (slice + 1) / slices);
  // 32 pages of a warp at a time: their ids in one load, a page's lanes then get
  // theirs (the first ones are on their way while q's codes are made)
  auto ids = [&](int b0) { return b0 < hi ? p.pages[mine.page_start + min(b0 + lane, hi - 1)] : 0; };
  int next = ids(lo + warp * 32);
  query_codes<T, D>(static_cast<const T*>(p.q) + t * p.q_stride + static_cast<int64_t>(h) * p.G * D, p.G, sh.codes[warp]);
  __syncwarp();
  int c[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int4 v = *reinterpret_cast<const int4*>(sh.codes[warp] + (i * LPR + lane % LPR) * 16);
    c[4 * i] = v.x, c[4 * i + 1] = v.y, c[4 * i + 2] = v.z, c[4 * i + 3] = v.w;
  }
  uint32_t* row = p.keys + static_cast<int64_t>(item) * p.max_pages;
  const bool own = slices == 1 && n <= kKept;  // the keys need not leave the CTA
  for (int b0 = lo + warp * 32; b0 < hi; b0 += kWarps * 32) {
    const int id = checked_page(p, next);
    next = ids(b0 + kWarps * 32);
#pragma unroll
    for (int w = 0; w < 32; w += U * RPW) {
      int4 v[U][4];
      float scale[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t at = static_cast<int64_t>(__shfl_sync(0xffffffffu, id, w + u * RPW + lane / LPR)) * p.g.Hkv + h;
        const int4* src = reinterpret_cast<const int4*>(p.bounds + at * (2 * D)) + lane % LPR;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[u][i] = __ldg(src + i * LPR);
        scale[u] = __ldg(p.bound_scales + at);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        int sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum = __dp4a(v[u][i].x, c[4 * i], sum);
          sum = __dp4a(v[u][i].y, c[4 * i + 1], sum);
          sum = __dp4a(v[u][i].z, c[4 * i + 2], sum);
          sum = __dp4a(v[u][i].w, c[4 * i + 3], sum);
        }
#pragma unroll
        for (int d = 1; d < LPR; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        const int b = b0 + w + u * RPW + lane / LPR;
        if (lane % LPR == 0 && b < hi) {
          const uint32_t x =
              b < p.first || b >= n - p.last ? kAlways : order_key(__fmul_rn(static_cast<float>(sum), scale[u]));
          if (own) kept[b] = x;
          else row[b] = x;
        }
      }
      if (b0 + w + U * RPW >= hi) break;
    }
  }
  if (slices > 1) {
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      int32_t* counter = p.counters + item;
      sh.last = atomicAdd(counter, 1) == slices - 1;
      if (sh.last) *counter = 0;
    }
    __syncthreads();
    if (!sh.last) return;
    __threadfence();
  } else {
    __syncthreads();
  }
  if (own) {
    select_largest([&](int i) { return kept[i]; }, n, p.num_blocks, out, sh.bins, sh.scan, sh.range);
  } else if (n <= kKept) {
    for (int i = tid; i < n; i += kThreads) kept[i] = __ldcg(row + i);
    __syncthreads();
    select_largest([&](int i) { return kept[i]; }, n, p.num_blocks, out, sh.bins, sh.scan, sh.range);
  } else {
    select_largest([&](int i) { return __ldcg(row + i); }, n, p.num_blocks, out, sh.bins, sh.scan, sh.range);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) select_kernel(const BlockParams p) {
  extern __shared__ __align__(16) uint32_t kept[];
  __shared__ SelectShared<D> shared;
  pdl_wait();
  unsigned works = gridDim.x;
  int slices = p.slices;
  if (p.listed) {
    const int items = p.small_indptr[p.batch] * p.g.Hkv;
    slices = items > 0 ? max(1, min(p.slices, 2 * p.num_sms / items)) : 1;
    works = unsigned(items) * slices;
  }
  for (unsigned work = blockIdx.x; work < works; work += gridDim.x) {
    __syncthreads();  // (shared memory of the item before)
    select_item<T, D>(p, work, slices, kept, shared);
  }
}

// ---------------------------------------------------------------------------
// chunks

constexpr int kTileRows = 16, kWarpBins = 256;

__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// As select_largest, by one warp: the first and last ones of n > k keys, and the
// largest of the others.  kRegs: of up to 32 * kRegs keys, held in registers; 0: of
// any number.
template <int kRegs>
__device__ __forceinline__ void warp_select(const uint32_t* key, int n, int k, int first, int last, int32_t* out, int* bins) {
  constexpr int STRIPS = kRegs ? kRegs : 1;
  const int lane = threadIdx.x & 31;
  const int lo = first, hi = n - last;
  int need = k - first - last;
  uint32_t held[STRIPS];  // 0, below every score's key, where there is none to choose
  auto load = [&](int i) { return i >= lo && i < hi ? key[i] : 0u; };
  if constexpr (kRegs > 0) {
#pragma unroll
    for (int s = 0; s < kRegs; ++s) held[s] = load(32 * s + lane);
  }
  // f(strip's first index, the lane's key of the strip)
  auto each = [&](auto&& f) {
    if constexpr (kRegs > 0) {
#pragma unroll
      for (int s = 0; s < kRegs; ++s)
        if (32 * s < n) f(32 * s, held[s]);
    } else {
#pragma unroll 4
      for (int i = 0; i < n; i += 32) f(i, load(i + lane));
    }
  };
  uint32_t least = 0xFFFFFFFFu, most = 0;
  each([&](int, uint32_t x) {
    least = min(least, x - 1);  // 0 is no key
    most = max(most, x);
  });
  const unsigned before = (1u << lane) - 1;
  uint32_t base = __reduce_min_sync(0xffffffffu, least) + 1, top = __reduce_max_sync(0xffffffffu, most) + 1;
  while (need > 0 && top - base > 1) {
    const int shift = max(0, 32 - __clz(top - 1 - base) - 8);
#pragma unroll
    for (int i = 0; i < kWarpBins / 32; ++i) bins[i * 32 + lane] = 0;
    __syncwarp();
    each([&](int, uint32_t x) {
      const uint32_t y = x - base;  // (of a key below base, and of 0, above all)
      if (y < top - base) atomicAdd(bins + (y >> shift), 1);
    });
    __syncwarp();
    int mine[kWarpBins / 32], sum = 0;  // lane l: the parts 255 - 8 l and down
    const int4 p0 = *reinterpret_cast<const int4*>(bins + 248 - 8 * lane), p1 = *reinterpret_cast<const int4*>(bins + 252 - 8 * lane);
    mine[0] = p1.w, mine[1] = p1.z, mine[2] = p1.y, mine[3] = p1.x, mine[4] = p0.w, mine[5] = p0.z, mine[6] = p0.y, mine[7] = p0.x;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += mine[i];
    int above = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, above, d);
      if (lane >= d) above += y;
    }
    above -= sum;
    int part = -1, still = 0, count = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (above < need && above + mine[i] >= need) part = 255 - 8 * lane - i, still = need - above, count = mine[i];
      above += mine[i];
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, part >= 0)) - 1;
    part = __shfl_sync(0xffffffffu, part, src);
    need = __shfl_sync(0xffffffffu, still, src);
    count = __shfl_sync(0xffffffffu, count, src);
    const uint64_t end = static_cast<uint64_t>(base) + ((static_cast<uint64_t>(part) + 1) << shift);
    base += static_cast<uint32_t>(part) << shift;
    if (end < top) top = static_cast<uint32_t>(end);
    __syncwarp();
    if (need == count) {  // the part whole
      top = base;
      need = 0;
    } else if (count <= 32) {  // a lane for each of its keys: the one with need - 1 larger ones is the border
      int at = 0;
      each([&](int, uint32_t x) {
        const bool in = x - base < top - base;
        const unsigned some = __ballot_sync(0xffffffffu, in);
        if (some) {
          if (in) bins[at + __popc(some & before)] = static_cast<int>(x);
          at += __popc(some);
        }
      });
      __syncwarp();
      const uint32_t x = lane < count ? static_cast<uint32_t>(bins[lane]) : 0u;
      int larger = 0, equal = 0;
      for (int i = 0; i < count; ++i) {
        const uint32_t y = __shfl_sync(0xffffffffu, x, i);
        larger += y > x;
        equal += y == x;
      }
      const int border = __ffs(__ballot_sync(0xffffffffu, lane < count && larger < need && larger + equal >= need)) - 1;
      base = __shfl_sync(0xffffffffu, x, border);
      need -= __shfl_sync(0xffffffffu, larger, border);
      top = base + 1;
      __syncwarp();
    }
  }
  int at = 0;
  each([&](int i0, uint32_t x) {
    const int i = i0 + lane;
    bool take = x >= top || (i < n && (i < lo || i >= hi));
    if (need > 0) {
      const unsigned equals = __ballot_sync(0xffffffffu, x < top && x == base);
      take = take || (x < top && x == base && __popc(equals & before) < need);
      need = max(0, need - __popc(equals));
    }
    const unsigned taken = __ballot_sync(0xffffffffu, take);
    if (take) out[at + __popc(taken & before)] = i;
    at += __popc(taken);
  });
}

template <int D, int kWarps>
struct TilesShared {
  __align__(16) int8_t codes[kTileRows][2 * D + 64];  // (rows 64 bytes apart in the banks)
  __align__(16) int bins[kWarps][kWarpBins];
};

// One tile of a request's tokens and one kv head.  kept: keys, [token][row].
template <typename T, int D, bool kGlobal, int kWarps>
__device__ __forceinline__ void select_tile(const BlockParams& p, int work, uint32_t* kept, int row,
                                            TilesShared<D, kWarps>& sh) {
  constexpr int STEPS = 2 * D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int tile = work / p.g.Hkv, h = work % p.g.Hkv;
  const int b = last_below(p.tile_indptr, p.batch + 1, tile);
  const Span r = load_span(p, b, false);
  const int q0 = (tile - p.tile_indptr[b]) * p.tile_tokens;
  const int tokens = min(p.tile_tokens, r.qo_len - q0), token = r.qo_start + q0;
  const int pos0 = r.kv_len - r.qo_len + q0;
  // pages that the last token sees (of tokens that see more than there is room for none is selected)
  const int end = pos0 + tokens - 1;
  const int pages = end < 0 ? 0 : min((end >> p.g.ps_shift) + 1, p.max_pages);
  if (pages > p.num_blocks) {
    for (int i = warp; i < kTileRows; i += kWarps) {
      if (i < tokens) {
        query_codes<T, D>(static_cast<const T*>(p.q) + (token + i) * p.q_stride + static_cast<int64_t>(h) * p.G * D, p.G, sh.codes[i]);
      } else {
        for (int c = lane; c < D / 2; c += 32) reinterpret_cast<uint32_t*>(sh.codes[i])[c] = 0;
      }
    }
    __syncthreads();
    // a lane takes every fourth piece of 16 bytes of a row, half a piece a k-step:
    // the order of the sum is free
    uint4 a[2][STEPS / 2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int s = 0; s < STEPS / 2; ++s) a[i][s] = *reinterpret_cast<const uint4*>(sh.codes[g + 8 * i] + (s * 4 + t4) * 16);
    // four steps of 8 pages at a time: their ids in one load
    for (int c0 = warp; c0 * 8 < pages; c0 += 4 * kWarps) {
      const int mine = (c0 + (lane >> 3) * kWarps) * 8 + (lane & 7);
      const int id = page_of(p, r.page_start + min(mine, pages - 1));
      for (int k = 0; k < 4; ++k) {
        const int b0 = (c0 + k * kWarps) * 8;
        if (b0 >= pages) break;
        const int64_t at = static_cast<int64_t>(__shfl_sync(0xffffffffu, id, k * 8 + g)) * p.g.Hkv + h;
        const uint4* src = reinterpret_cast<const uint4*>(p.bounds + at * (2 * D)) + t4;
        uint4 v[STEPS / 2];
#pragma unroll
        for (int i = 0; i < STEPS / 2; ++i) v[i] = __ldg(src + 4 * i);
        const float scale = __ldg(p.bound_scales + at);
        int c[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < STEPS / 2; ++i) {
          mma_s8(c, a[0][i].x, a[1][i].x, a[0][i].y, a[1][i].y, v[i].x, v[i].y);
          mma_s8(c, a[0][i].z, a[1][i].z, a[0][i].w, a[1][i].w, v[i].z, v[i].w);
        }
        // c: tokens g and g + 8, pages 2 t4 and the next
        const float s0 = __shfl_sync(0xffffffffu, scale, 8 * t4), s1 = __shfl_sync(0xffffffffu, scale, 8 * t4 + 4);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (g + 8 * i < tokens)
            *reinterpret_cast<uint2*>(kept + (g + 8 * i) * row + b0 + 2 * t4) =
                make_uint2(order_key(__fmul_rn(static_cast<float>(c[2 * i]), s0)),
                           order_key(__fmul_rn(static_cast<float>(c[2 * i + 1]), s1)));
      }
    }
  }
  __syncthreads();
  if constexpr (!kGlobal) pdl_launch();
  for (int i = warp; i < tokens; i += kWarps) {
    const int pos = pos0 + i, n = pos < 0 ? 0 : (pos >> p.g.ps_shift) + 1;
    int32_t* out = p.blocks + (static_cast<int64_t>(token + i) * p.g.Hkv + h) * p.num_blocks;
    if (n <= p.num_blocks || n > p.max_pages) {
      for (int c = lane; c < p.num_blocks; c += 32) out[c] = c < n && n <= p.max_pages ? c : -1;
      if (n > p.max_pages && lane == 0) atomicOr(p.status, PA_DEV_NO_ROOM);
    } else {
      // (a strip of 32 keys past n costs little, so few sizes do)
      if (n <= 256) warp_select<8>(kept + i * row, n, p.num_blocks, p.first, p.last, out, sh.bins[warp]);
      else if (n <= 512) warp_select<16>(kept + i * row, n, p.num_blocks, p.first, p.last, out, sh.bins[warp]);
      else warp_select<0>(kept + i * row, n, p.num_blocks, p.first, p.last, out, sh.bins[warp]);
    }
    __syncwarp();
  }
}

// kGlobal: the keys in global memory, a piece for each of the CTAs, which take
// tile after tile; otherwise the grid has a CTA for each tile.
template <typename T, int D, bool kGlobal>
__global__ void __launch_bounds__(kGlobal ? 512 : kThreads, D == 256 ? (kGlobal ? 1 : 2) : (kGlobal ? 2 : 4))
    select_tiles_kernel(const BlockParams p, const int row) {
  constexpr int kWarps = kGlobal ? 16 : kThreads / 32;
  extern __shared__ __align__(16) uint32_t kept[];
  __shared__ TilesShared<D, kWarps> shared;
  pdl_wait();
  const int works = p.tile_indptr[p.batch] * p.g.Hkv;
  if constexpr (kGlobal) {
    uint32_t* piece = p.keys + static_cast<int64_t>(blockIdx.x) * kTileRows * row;
    for (int work = blockIdx.x; work < works; work += gridDim.x) {
      select_tile<T, D, true, kWarps>(p, work, piece, row, shared);
      __syncthreads();
    }
  } else if (static_cast<int>(blockIdx.x) < works) {
    select_tile<T, D, false, kWarps>(p, blockIdx.x, kept, row, shared);
  }
}

template <typename T>
cudaError_t launch_t(const BlockParams& p, int D, unsigned grid, size_t smem, cudaStream_t stream) {
  switch (D) {
    case 64: return launch_pdl(select_kernel<T, 64>, grid, kThreads, smem, stream, p);
    case 128: return launch_pdl(select_kernel<T, 128>, grid, kThreads, smem, stream, p);
    default: return launch_pdl(select_kernel<T, 256>, grid, kThreads, smem, stream, p);
  }
}

template <typename T, int D>
cudaError_t launch_tiles_d(const BlockParams& p, const SelectShape& t, unsigned grid, cudaStream_t stream) {
  if (t.ctas) return launch_pdl(select_tiles_kernel<T, D, true>, grid < unsigned(t.ctas) ? grid : unsigned(t.ctas), 512u, size_t(0), stream, p, t.row);
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = set_smem_once(done, reinterpret_cast<const void*>(select_tiles_kernel<T, D, false>), kTileSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(select_tiles_kernel<T, D, false>, grid, kThreads, size_t(kTileRows) * t.row * 4, stream, p, t.row);
}
template <typename T>
cudaError_t launch_tiles(const BlockParams& p, const SelectShape& t, int D, unsigned grid, cudaStream_t stream) {
  switch (D) {
    case 64: return launch_tiles_d<T, 64>(p, t, grid, stream);
    case 128: return launch_tiles_d<T, 128>(p, t, grid, stream);
    default: return launch_tiles_d<T, 256>(p, t, grid, stream);
  }
}

}  // namespace

SelectShape select_shape(const BlockShape& s) {
  SelectShape t;
  t.row = (s.max_pages + 31) / 32 * 32 + 8;  // (rows 8 banks apart)
  t.tokens = kTileRows;
  // More keys than two CTAs an SM keep go to global memory, that is, to L2: 2000 tokens
  // at 8 kv heads take 199 us for 1500 pages with keys in shared memory and 210 so,
  // for 2000 pages (one CTA an SM) 396 and 275.  Beyond kKeptKeys pages tokens select by
  // themselves: the CTAs' keys would pass 160 MB (2000 tokens over all of 8192 pages 1876 us, with
  // room for one page more 2906; over 2000 of them 284 and 869).
  t.ctas = int64_t(kTileRows) * t.row * 4 > kTileSmem ? s.num_sms * (s.D == 256 ? 1 : 2) : 0;
  t.long_tokens = 4;
  // Fewer than the single tokens' CTAs of a full card are quicker there: of 500 pages
  // at 8 kv heads 32 tokens take 24 us in tiles and 11 by themselves, 64 24 and
  // 21, 128 24 and 30.
  t.least_long = 4 * s.num_sms / s.Hkv;
  if (s.max_qo_len < t.long_tokens || s.num_tokens < t.least_long || s.max_pages <= s.num_blocks ||
      s.max_pages > kKeptKeys)
    t.tokens = 0;
  const int64_t longs = s.num_tokens / t.long_tokens < s.batch ? s.num_tokens / t.long_tokens : s.batch;
  t.max_tiles = t.tokens ? int32_t(s.num_tokens / t.tokens + longs) : 0;
  return t;
}

cudaError_t launch_order_requests(const BlockParams& p, cudaStream_t stream) {
  return launch_pdl(order_requests_kernel, 1u, 1024u, size_t(0), stream, p);
}

cudaError_t launch_select(BlockParams p, const BlockShape& s, int select_tokens, int dtype, cudaStream_t stream) {
  const int tokens = select_tokens;
  const SelectShape chunk = select_shape(s);
  p.num_sms = s.num_sms;
  if (chunk.tokens) {
    p.tile_tokens = chunk.tokens;
    p.long_tokens = chunk.long_tokens;
    p.max_tiles = chunk.max_tiles;
    p.least_long = chunk.least_long;
    cudaError_t e = launch_order_requests(p, stream);
    if (e != cudaSuccess) return e;
    const unsigned grid = unsigned(chunk.max_tiles) * unsigned(s.Hkv);
    if (grid > 0) {
      e = dtype == PA_BF16 ? launch_tiles<__nv_bfloat16>(p, chunk, s.D, grid, stream)
                           : launch_tiles<__half>(p, chunk, s.D, grid, stream);
      if (e != cudaSuccess) return e;
    }
    p.listed = 1;
  }
  const size_t smem = sizeof(uint32_t) * (s.max_pages < kKept ? s.max_pages : kKept);
  // slices of 256 pages or more
  int most = 1;
  while (most < 64 && s.max_pages > 512 * most) most *= 2;
  if (p.listed) {
    // how many tokens are listed the host does not know: CTAs for a full card, slice after slice
    const int64_t works = int64_t(s.num_tokens) * s.Hkv * most, full = int64_t(s.num_sms) * 4;
    const unsigned grid = unsigned(works < full ? works : full);
    p.token0 = 0;
    p.slices = most;
    return dtype == PA_BF16 ? launch_t<__nv_bfloat16>(p, s.D, grid, smem, stream)
                            : launch_t<__half>(p, s.D, grid, smem, stream);
  }
  for (int t = 0; t < s.num_tokens; t += tokens) {
    const int n = s.num_tokens - t < tokens ? s.num_tokens - t : tokens;
    const int items = n * s.Hkv;
    // until the card has two CTAs an SM
    int slices = 1;
    while (slices < most && items * slices < 2 * s.num_sms) slices *= 2;
    p.token0 = t;
    p.slices = slices;
    const cudaError_t e = dtype == PA_BF16 ? launch_t<__nv_bfloat16>(p, s.D, unsigned(items * slices), smem, stream)
                                           : launch_t<__half>(p, s.D, unsigned(items * slices), smem, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace pa
