// Attention over a paged cache held in 4 bits, through device tables
// (pagedattn_kv4_run): the small-query kernel (decode, drafted tokens).
//
// Number formats.  K and V are e2m1 codes with an e4m3 scale per 16 values
// along head_dim.  code * scale has at most 6 significant bits and lies in
// [2^-10, 2688], so it is exact in fp16: every product below is an fp16 MMA
// over the exact cache values, for fp16 and bf16 queries alike.  A bf16 query
// row is multiplied by the power of two that brings its largest value to
// [2^13, 2^14) first (bf16's 8 significant bits fit fp16's 11; what falls
// below fp16's range is 2^-38 of the row's largest value) and the logits by
// its inverse.  The cache's own fp32 scales go into the logit factor (K) and
// the epilogue (V).  P is rounded to fp16 (2^-11 relative; small ones see
// kPHead) for the P V product, whatever the type of q: a bf16 P would cost 2^-8.
//
// Work.  A unit is 64 keys of one row tile (8 * NT packed rows: token major,
// the G query heads of the kv head minor) of one request.  The units of the
// batch, in request order, are cut into equal slices whatever the requests'
// boundaries, so that one request of 10^5 keys and 10^3 requests of 100 keys
// load the SMs alike with no plan from the host: every CTA sums the units of
// all requests itself (one block scan) and so finds where its slice begins.
// A row tile that a slice boundary cuts leaves fp32 partial states, which the
// last of its slices to finish joins.  (Batches that leave a slice for every
// row tile: see the kernel.)
// A CTA has up to 8 kv heads, a warp or a team of warps each: the heads of a
// page are read at the same time (in the NHD layout 4 heads share a 32-byte
// sector of scales), and where a warp has a head alone its state is the
// result, with nothing to join.  With fewer requests than slices it has one
// head, whose keys the 8 warps share, so that no warp joins many parts alone.
//
// A warp takes 32 keys at a time.  It copies its own steps two or more ahead
// (cp.async into a ring of its own: no warp waits for another) and computes
// S^T = K q^T and O^T = V^T P^T with m16n8k16, so that keys (or dims) fill the
// 16-row side and 8 packed rows the other.  Both contractions are free in the
// order of their index:
//   S^T  lane (g, t) takes dims [t D/4, (t+1) D/4) of its keys: 16 bytes each
//        (head_dim 128), converted in the order they lie in memory; q's
//        fragments are loaded in the same order.
//   O^T  lane (g, t) takes dims [g D/8, (g+1) D/8) of 4 keys of each 16: the
//        codes of two keys are merged nibble by nibble (two bitfield selects
//        for 16 values) so that one conversion gives the fragment's
//        (key, key + 1) pair.
//
// What bounds it: bytes and instructions alike.  256 decodes of 512 to 8192
// keys at 64 / 8 heads (1.27 GB) take 250 us, 5.1 TB/s; the copies alone take
// 214 to 220, the arithmetic alone 213 (635 warp instructions for 32 keys and a
// head, of them 140 conversions, 128 scalings and 32 MMAs).  Steps on the way:
// fragments straight from global memory 340 us; rings of cp.async 299; a CTA
// for all heads of its keys 263; constant shared offsets and q's loads under
// the page ids' 250.  Measured without gain: wider steps in registers (426
// us), the conversions replaced by bit operations (2.4 times their time).
#include <climits>
#include <cstring>
#include <type_traits>
#include <utility>

#include "internal.h"
#include "kv4_common.cuh"

namespace pa {
namespace {

constexpr int kUnitKeys = 64;
constexpr int kMinUnits = 4;  // of a slice: below 256 keys a split costs more than it spreads
constexpr int kStepKeys = 32;
constexpr int kTries = 8;       // part sizes that are weighed
constexpr int kKeptReqs = 128;  // requests of a slice kept in shared memory
constexpr float kLn2f = 0.6931471805599453f;
// A running maximum before any key: finite, so that it can be subtracted.
constexpr float kNone = -3.0e38f;

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// a / b for a >= 0, b > 0; in 32 bits where they do (a division in 64 takes a
// hundred instructions).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
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

// The same with a zero sum to start from.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// BYTES of shared memory in registers.  (Plain loads: a constant part of the
// address is the instruction's, where inline assembly had an addition for
// each of a step's 24 loads.)
template <int BYTES>
__device__ __forceinline__ void lds(uint32_t (&r)[BYTES / 4], const uint8_t* at) {
  if constexpr (BYTES == 4) {
    r[0] = *reinterpret_cast<const uint32_t*>(at);
  } else if constexpr (BYTES == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(at);
    r[0] = v.x;
    r[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(at);
    r[0] = v.x;
    r[1] = v.y;
    r[2] = v.z;
    r[3] = v.w;
  }
}
// 1, 2 or 4 bytes of shared memory.
template <int BYTES>
__device__ __forceinline__ uint32_t lds_scales(const uint8_t* at) {
  if constexpr (BYTES == 4) return *reinterpret_cast<const uint32_t*>(at);
  if constexpr (BYTES == 2) return *reinterpret_cast<const uint16_t*>(at);
  return *at;
}
// f(0), f(1), ... f(N - 1) with constants.
template <int... I, typename F>
__device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, F&& f) {
  (f(std::integral_constant<int, I>{}), ...);
}
// cp.async of N bytes (through L2 alone where N = 16), and one that writes
// zeros where !live.
template <int N, int OFF>
__device__ __forceinline__ void cp_async(uint32_t dst, const uint8_t* src) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0 + %2], [%1], 16;" ::"r"(dst), "l"(src), "n"(OFF) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0 + %3], [%1], %2;" ::"r"(dst), "l"(src), "n"(N), "n"(OFF) : "memory");
}
template <int N, int OFF>
__device__ __forceinline__ void cp_async_or_zero(uint32_t dst, const uint8_t* src, bool live) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0 + %3], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0), "n"(OFF)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0 + %4], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(live ? N : 0), "n"(N),
                 "n"(OFF)
                 : "memory");
}
template <int N> __device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A stage: 32 keys of one kv head in shared memory, K codes, V codes, K
// scales, V scales.  The rows of codes are 16-byte chunks whose place in the
// row is exclusive-ored with swizzle(row), and row r of each 8-row group of an
// MMA is the group's key order(r); both are chosen so that neither K's
// reads (rows r, r + 1, ... whole) nor V's (the even or the odd rows, one
// chunk of each) meet in a bank.
template <int D>
struct Stage {
  static constexpr int ROW = D / 2, SROW = D / 16;
  static constexpr int OFF_V = kStepKeys * ROW, OFF_KS = 2 * OFF_V, OFF_VS = OFF_KS + kStepKeys * SROW;
  static constexpr int BYTES = OFF_VS + kStepKeys * SROW;
  static constexpr int KB = D / 8;   // bytes of a K row that a lane reads: D/4 dims
  static constexpr int VB = D / 16;  // of a V row: D/8 dims
  static constexpr int KS = D / 64;  // their scales
  static constexpr int VS = D >= 128 ? D / 128 : 1;
  static constexpr int LANES = ROW / 16;  // lanes that copy a row
  static __device__ __forceinline__ int swizzle(int row) {
    if constexpr (D == 64) return 0;
    if constexpr (D == 128) return row & 2;
    return ((row & 3) << 1) | ((row >> 2) & 1);
  }
  static __device__ __forceinline__ int order(int r) {  // r in [0, 8)
    const int t = r >> 1;
    return r & 1 ? 4 + (t ^ (D == 64 ? 2 : 1)) : t;
  }
};

// Warps of a CTA and CTAs of an SM by head_dim and 8-row groups of a tile:
// O^T takes D / 4 registers a lane for each group, q's fragments D / 8 (kept
// in shared memory where that passes 64).
constexpr int small_ctas(int D, int nt) { return D < 256 && D * nt <= 256 && nt < 4 ? 2 : 1; }
constexpr int small_warps(int D, int nt) { return small_ctas(D, nt) == 2 && D * nt == 256 ? 6 : 8; }

template <int D, int NT>
struct SmallCfg {
  static constexpr int ROWS = 8 * NT;
  static constexpr int WARPS = small_warps(D, NT);
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int CTAS = small_ctas(D, NT);
  static constexpr bool Q_SMEM = NT * D >= 512;
  static constexpr int STAGES = D == 256 ? 3 : (CTAS == 1 ? 5 : (D == 64 ? 5 : (WARPS == 6 ? 4 : 3)));
  static constexpr int RING = STAGES * Stage<D>::BYTES;  // of a warp
  // after its loop a warp's state takes its ring's place (floats)
  static constexpr int O_STRIDE = D + 4;
  static_assert(ROWS * (O_STRIDE + 2) * 4 <= RING, "a warp's state fits its ring");
  static constexpr int SMEM = WARPS * RING + (Q_SMEM ? NT * (D / 16) * 256 + ROWS * 4 : 0);
  static_assert(CTAS * (SMEM + kKeptReqs * 16 + 768 + 1024) <= 233472, "shared memory per SM");
};

// kScrub: rows of a tile may see different keys (several tokens under a causal
// mask), so that a masked key's NaN has to be kept from the others.
template <typename T, int D, int NT, bool kScrub>
__global__ void __launch_bounds__(SmallCfg<D, NT>::THREADS, SmallCfg<D, NT>::CTAS) kv4_small_kernel(const Kv4Params p) {
  using C = SmallCfg<D, NT>;
  using St = Stage<D>;
  constexpr int kThreads = C::THREADS, kWarps = C::WARPS;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long scratch[kWarps];
  __shared__ int tiles_s[kWarps], longest_s[kWarps], sums_s[kWarps][kTries];
  __shared__ Req req_s[kKeptReqs];  // the slice's first requests, where its scan met them
  __shared__ long long found_u;
  __shared__ int found_b, last_s[8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  // the CTA's kv heads, and the warp's: `team` warps share one and take every
  // team-th step each
  const int cta_heads = C::Q_SMEM ? 1 : p.cta_heads;
  const int groups = p.g.Hkv / cta_heads;
  const int slice = blockIdx.x / groups, cta_head = warp % cta_heads;
  const int h = (blockIdx.x % groups) * cta_heads + cta_head;
  const int team = kWarps / cta_heads, member = warp / cta_heads;
  const int rank = member * 32 + lane;  // of the team's threads
  auto team_sync = [&]() {
    if (team == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + cta_head), "r"(team * 32) : "memory");
  };
  pdl_wait();

  // ---- the slice's units [u, u_end) and the request that they begin in
  auto units_of = [&](const Req& r) -> long long {
    return static_cast<long long>(row_tiles(p, r, C::ROWS)) * key_units(r);
  };
  Req mine{0, 0, 0, 0};
  long long units = 0;
  int tiles = 0, longest = 0;
  for (int b = tid; b < p.batch; b += kThreads) {
    mine = load_req(p, b);
    const int n = row_tiles(p, mine, C::ROWS), k = key_units(mine);
    units += static_cast<long long>(n) * k;
    tiles = min(tiles + n, 1 << 20);
    if (n > 0) longest = max(longest, k);
  }
  const int my_tiles = tiles;
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    tiles += __shfl_xor_sync(0xffffffffu, tiles, d);
    longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, d));
  }
  if (lane == 0) {
    tiles_s[warp] = tiles;
    longest_s[warp] = longest;
  }
  auto sum_before = [&](long long v, long long* all) -> long long {  // exclusive sum over the block
    long long x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    long long before = x - v, sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += scratch[w];
      sum += scratch[w];
    }
    __syncthreads();
    *all = sum;
    return before;
  };
  long long total;
  long long before = sum_before(units, &total);
  const long long per_slice = max(static_cast<long long>(kMinUnits), quotient(total + p.slices - 1, p.slices));

  // ---- Slices of one size take a share of the next request with them and leave
  // a share of their last one to the next slice.  Where there are slices enough
  // for every row tile, a slice may be one tile instead, or one of equal parts
  // of at most `part_units`: no second start in a slice, and no join where the
  // tiles stay whole.  Weighed in us: a unit's bytes at the 20 GB/s that a CTA
  // gets when all run, 8 for the second start and the joins of equal slices,
  // 4.5 for a join (128 requests of 1024 keys: 16.6 us in equal slices, 13.8
  // whole).
  int part_units = 0;  // 0: slices of equal size
  if (p.slices > 1 && p.batch <= kThreads) {
    tiles = longest = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      tiles += tiles_s[w];
      longest = max(longest, longest_s[w]);
    }
    const float unit_us = static_cast<float>(cta_heads) * D * 0.0036f;
    const int least = static_cast<int>(min(per_slice, static_cast<long long>(longest)));
    if (tiles > 0 && tiles <= p.slices) {
      float best = least * unit_us + 8.f;
      if (longest * unit_us < best) {
        best = longest * unit_us;
        part_units = longest;
      }
      if (least * unit_us + 4.5f < best) {
        int n[kTries];
#pragma unroll
        for (int k = 0; k < kTries; ++k) {
          const int size = least + (longest - least) * k / kTries;
          n[k] = my_tiles * ((key_units(mine) + size - 1) / max(1, size));
#pragma unroll
          for (int d = 16; d; d >>= 1) n[k] += __shfl_xor_sync(0xffffffffu, n[k], d);
          if (lane == 0) sums_s[warp][k] = n[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = kTries - 1; k >= 0; --k) {
          const int size = least + (longest - least) * k / kTries;
          int all = 0;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) all += sums_s[w][k];
          if (all <= p.slices && size * unit_us + 4.5f < best) {
            best = size * unit_us + 4.5f;
            part_units = size;
          }
        }
      }
    }
  }
  const bool by_parts = part_units > 0;
  auto parts_of = [&](const Req& r) { return (key_units(r) + part_units - 1) / part_units; };
  long long u = slice * per_slice;
  long long u_end = min(total, u + per_slice);
  if (by_parts) {  // u counts parts here
    units = static_cast<long long>(my_tiles) * parts_of(mine);
    before = sum_before(units, &total);
    u = slice;
    u_end = min(total, u + 1);
  }
  if (u >= u_end) return;
  int chunk = 0;  // first request of the threads' `mine`
  for (long long base = 0; chunk < p.batch; chunk += kThreads) {
    long long v = units, all = total;
    if (p.batch > kThreads) {
      mine = Req{0, 0, 0, 0};
      if (chunk + tid < p.batch) mine = load_req(p, chunk + tid);
      v = units_of(mine);
      before = base + sum_before(v, &all);
    }
    base += all;
    if (u >= base) continue;
    if (v > 0 && before <= u && u < before + v) {
      found_b = chunk + tid;
      found_u = before;
    }
    break;
  }
  __syncthreads();
  const int first_b = found_b;  // always found: u < total
  if (chunk + tid >= first_b && chunk + tid - first_b < kKeptReqs) req_s[chunk + tid - first_b] = mine;
  __syncthreads();
  const int kept_b = min(first_b + kKeptReqs, chunk + kThreads);
  int b = first_b;
  long long req_u = found_u;  // the request's first unit
  Req rq = req_s[0];

  const DivG div_g(p.G);

  // ---- where a lane copies to and reads from in a stage
  const uint32_t page_bytes = static_cast<uint32_t>(p.g.ps) * p.g.Hkv * D;  // K and V codes of a page, at most 2^31
  const uint32_t slot_bytes = static_cast<uint32_t>(p.g.slot_rows) * (D / 2);
  const int copy_row = lane / St::LANES, copy_chunk = lane % St::LANES;
  const uint8_t* codes_h = p.codes + static_cast<int64_t>(h) * p.g.head_rows * (D / 2) + copy_chunk * 16;
  const uint8_t* scales_h = p.scales + static_cast<int64_t>(h) * p.g.head_rows * (D / 16);
  const uint32_t smem_base = smem_u32(smem);
  const uint32_t ring = smem_base + warp * C::RING;
  // states: of member w of the team at w * team_step
  float* o_s = reinterpret_cast<float*>(smem + cta_head * C::RING);  // [rows][O_STRIDE], then m and l of each row
  const int team_step = cta_heads * C::RING / 4;
  constexpr int OFF_ML = C::ROWS * C::O_STRIDE;
  uint2* q_s = reinterpret_cast<uint2*>(smem + kWarps * C::RING);  // Q_SMEM: [NT][D / 16][lane], then the rows' factors
  float* fac_s = reinterpret_cast<float*>(q_s + NT * (D / 16) * 32);
  const uint32_t copy_to = copy_row * St::ROW + ((copy_chunk ^ St::swizzle(copy_row & 7)) << 4);
  const int k_row = St::order(g);  // + 8 i
  const uint32_t k_at = k_row * St::ROW + ((((t * St::KB) >> 4) ^ St::swizzle(k_row)) << 4) + ((t * St::KB) & 15);
  uint32_t v_at[2];  // rows 2t and 2t + 1, + 8 i
  int v_row[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    v_row[e] = St::order(2 * t + e);
    v_at[e] = St::OFF_V + v_row[e] * St::ROW + ((((g * St::VB) >> 4) ^ St::swizzle(v_row[e])) << 4) +
              ((g * St::VB) & 15);
  }

  // ---- row tiles, one after the other
  bool first_segment = true;
  while (u < u_end) {
    const int kts = key_units(rq);
    const int n_parts = by_parts ? parts_of(rq) : kts;  // of a row tile, in what u counts
    const int rt = static_cast<int>(quotient(u - req_u, n_parts));
    const long long tile_u = req_u + static_cast<long long>(rt) * n_parts;
    const long long seg_end = min(u_end, tile_u + n_parts);
    const int at0 = static_cast<int>(u - tile_u), at1 = static_cast<int>(seg_end - tile_u);
    const int unit0 = by_parts ? static_cast<int>(quotient(static_cast<long long>(kts) * at0, n_parts)) : at0;
    const int unit1 = by_parts ? static_cast<int>(quotient(static_cast<long long>(kts) * at1, n_parts)) : at1;
    const bool whole = unit0 == 0 && unit1 == kts;
    const int row0 = rt * C::ROWS;
    const int rows = min(C::ROWS, rq.qo_len * p.G - row0);
    // packed row n of the tile: token tok0 + token_of(n), head (head0 + n) % G
    const int tok0 = row0 / p.G, head0 = row0 - tok0 * p.G;
    auto token_of = [&](int n) { return div_g.div(head0 + n); };
    // keys that some row of the tile sees, and those that every row sees
    const int shift = rq.kv_len - rq.qo_len + 1;
    const int seen_end = p.causal ? max(0, shift + tok0 + token_of(rows - 1)) : rq.kv_len;
    const int all_end = p.causal ? shift + tok0 : rq.kv_len;
    const int key_a = unit0 * kUnitKeys;
    const int key_b = min(unit1 * kUnitKeys, seen_end);
    const int steps = key_b > key_a ? (key_b - key_a + kStepKeys - 1) / kStepKeys : 0;

    // page of key `lane` of a step; keys that no row sees have none
    const int32_t* page_ids = p.pages + rq.page_start;
    auto step_page = [&](int s) -> int {
      const int key = key_a + s * kStepKeys + lane;
      return s < steps && key < key_b ? __ldg(page_ids + (key >> p.g.ps_shift)) : 0;
    };
    // copies step s into the stage at `st`; `pids` from step_page(s)
    auto copy_rows = [&](int key, uint32_t st, int pids, auto tail) {
      constexpr bool kTail = decltype(tail)::value;  // rows of keys that no row sees are zeros
      const uint32_t dst0 = st + copy_to;
      each_of(std::make_integer_sequence<int, St::LANES>{}, [&](auto which) {
        constexpr int i = decltype(which)::value;
        constexpr int RPP = 32 / St::LANES;
        const int r = i * RPP + copy_row;
        const uint32_t pid = __shfl_sync(0xffffffffu, pids, r);
        const uint32_t slot = (key + r) & (p.g.ps - 1);
        const uint8_t* src = offset_by(offset_by(codes_h, slot, slot_bytes), pid, page_bytes);
        // (the swizzle of a 4-row pass changes with bit 2 of its first row)
        const uint32_t dst = D == 256 && (i & 1) ? dst0 ^ 16 : dst0;
        constexpr int OFF = i * RPP * St::ROW;
        if constexpr (kTail) {
          const bool live = key + r < key_b;
          cp_async_or_zero<16, OFF>(dst, src, live);
          cp_async_or_zero<16, OFF + St::OFF_V>(dst, src + (page_bytes >> 1), live);
        } else {
          cp_async<16, OFF>(dst, src);
          cp_async<16, OFF + St::OFF_V>(dst, src + (page_bytes >> 1));
        }
      });
      const uint32_t slot = (key + lane) & (p.g.ps - 1);
      const uint8_t* src =
          offset_by(offset_by(scales_h, slot, slot_bytes >> 3), static_cast<uint32_t>(pids), page_bytes >> 3);
      const uint32_t dst = st + lane * St::SROW;
      if constexpr (kTail) {
        const bool live = key + lane < key_b;
        cp_async_or_zero<St::SROW, St::OFF_KS>(dst, src, live);
        cp_async_or_zero<St::SROW, St::OFF_VS>(dst, src + (page_bytes >> 4), live);
      } else {
        cp_async<St::SROW, St::OFF_KS>(dst, src);
        cp_async<St::SROW, St::OFF_VS>(dst, src + (page_bytes >> 4));
      }
    };
    auto copy_step = [&](int s, uint32_t st, int pids) {
      if (s < steps) {
        if (static_cast<unsigned>(pids) >= static_cast<unsigned>(p.g.num_pages)) {
          atomicOr(p.status, PA_DEV_BAD_INDEX);
          pids = 0;
        }
        const int key = key_a + s * kStepKeys;
        if (key + kStepKeys <= key_b) copy_rows(key, st, pids, std::false_type{});
        else copy_rows(key, st, pids, std::true_type{});
      }
      cp_async_commit();
    };
    int pids[C::STAGES];
#pragma unroll
    for (int i = 0; i < C::STAGES; ++i) pids[i] = step_page(member + i * team);

    // q fragments (row n = g of each 8-row group, dims [t D/4, (t+1) D/4)) and
    // the logit factors of rows 2t, 2t + 1
    uint32_t qf[C::Q_SMEM ? 1 : NT][D / 16][2];
    float fac[NT][2];
    int lim[NT][2];
    auto load_q = [&](int nt, uint32_t (&f)[D / 16][2]) {
      const int n = nt * 8 + g, tok = token_of(n);
      if (n < rows) {
        const T* src = static_cast<const T*>(p.q) + static_cast<int64_t>(rq.qo_start + tok0 + tok) * p.q_stride +
                       static_cast<int64_t>(h * p.G + head0 + n - tok * p.G) * D + t * (D / 4);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          const uint4 w = *(reinterpret_cast<const uint4*>(src) + c);
          f[2 * c][0] = w.x;
          f[2 * c][1] = w.y;
          f[2 * c + 1][0] = w.z;
          f[2 * c + 1][1] = w.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < D / 16; ++j) f[j][0] = f[j][1] = 0;
      }
    };
    auto scale_q = [&](uint32_t (&f)[D / 16][2]) -> float {  // to fp16; returns the row's factor
      float my = p.scale_log2;
      if constexpr (Elt<T>::kBf16) {
        uint32_t top = 0;  // the largest magnitude's bf16 bits
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) top = max(top, max(f[j][i] & 0x7FFFu, (f[j][i] >> 16) & 0x7FFFu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int up = bf16_row_shift(top);
        const float mul = pow2(up);
        my = row_factor(my, pow2(-up));
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 x = Elt<T>::to_f2(f[j][i]);
            f[j][i] = pack_f16x2(x.x * mul, x.y * mul);
          }
      }
      return my;
    };
    if constexpr (C::Q_SMEM) {
      // warp nt makes row group nt's fragments for all (the CTA has one head)
      if (warp < NT) {
        load_q(warp, qf[0]);
        const float my = scale_q(qf[0]);
#pragma unroll
        for (int j = 0; j < D / 16; ++j) q_s[(warp * (D / 16) + j) * 32 + lane] = make_uint2(qf[0][j][0], qf[0][j][1]);
        if (t == 0) fac_s[warp * 8 + g] = my;
      }
      team_sync();
    } else {
      // q's loads fly while the copies wait for their page ids
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) load_q(nt, qf[nt]);
    }
#pragma unroll
    for (int i = 0; i < C::STAGES - 1; ++i) copy_step(member + i * team, ring + i * St::BYTES, pids[i]);
    int next_pids = pids[C::STAGES - 1];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float my = 0.f;
      if constexpr (!C::Q_SMEM) my = scale_q(qf[nt]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if constexpr (C::Q_SMEM) fac[nt][i] = fac_s[nt * 8 + 2 * t + i];
        else fac[nt][i] = __shfl_sync(0xffffffffu, my, (2 * t + i) * 4);
        lim[nt][i] = p.causal ? min(shift + tok0 + token_of(nt * 8 + 2 * t + i), rq.kv_len) : rq.kv_len;
      }
    }

    float o[NT][D / 16][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
      m[nt][0] = m[nt][1] = kNone;
      l[nt][0] = l[nt][1] = 0.f;
    }

    // One step; kEdge: some row does not see every key of it.
    uint32_t st_read = ring, st_write = ring + (C::STAGES - 1) * St::BYTES;
    const uint32_t ring_end = ring + C::STAGES * St::BYTES;
    auto step = [&](int s, auto edge) {
      constexpr bool kEdge = decltype(edge)::value;
      const int key = key_a + s * kStepKeys;
      // the step's stage has landed, and every lane is done with the one
      // that the copies below overwrite
      cp_async_wait<C::STAGES - 2>();
      __syncwarp();
      copy_step(s + (C::STAGES - 1) * team, st_write, next_pids);
      next_pids = step_page(s + C::STAGES * team);
      const uint8_t* st = smem + (st_read - smem_base);
      st_write = st_read;
      st_read = st_read + St::BYTES == ring_end ? ring : st_read + St::BYTES;
      // ---- S^T = K q^T
      float sc[NT][2][4];
      uint32_t ks[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) ks[i] = lds_scales<St::KS>(st + St::OFF_KS + (k_row + 8 * i) * St::SROW + t * St::KS);
#pragma unroll
      for (int w16 = 0; w16 < (St::KB + 15) / 16; ++w16) {  // 16 bytes (or all 8) of each key
      constexpr int LB = St::KB < 16 ? St::KB : 16;
      uint32_t kw[4][LB / 4];
#pragma unroll
      for (int i = 0; i < 4; ++i) lds<LB>(kw[i], st + ((k_at + i * 8 * St::ROW) ^ (w16 << 4)));
#pragma unroll
      for (int wi = 0; wi < LB / 4; ++wi) {  // 8 dims of each key
        const int w = w16 * 4 + wi;
        uint2 q0[NT], q1[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if constexpr (C::Q_SMEM) {
            q0[nt] = q_s[(nt * (D / 16) + 2 * w) * 32 + lane];
            q1[nt] = q_s[(nt * (D / 16) + 2 * w + 1) * 32 + lane];
          } else {
            q0[nt] = make_uint2(qf[nt][2 * w][0], qf[nt][2 * w][1]);
            q1[nt] = make_uint2(qf[nt][2 * w + 1][0], qf[nt][2 * w + 1][1]);
          }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          uint32_t a[4], c[4];
          e2m1x8(kw[2 * n][wi], a);
          e2m1x8(kw[2 * n + 1][wi], c);
          const uint32_t twice = (w >> 1) * 0x1111u;  // the scale's byte, twice
          const uint32_t s0 = e4m3x2_f16(__byte_perm(ks[2 * n], 0, twice));
          const uint32_t s1 = e4m3x2_f16(__byte_perm(ks[2 * n + 1], 0, twice));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a[i] = mul_f16x2(a[i], s0);
            c[i] = mul_f16x2(c[i], s1);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (w == 0) mma_f16_first(sc[nt][n], a[0], c[0], a[1], c[1], q0[nt].x, q0[nt].y);
            else mma_f16(sc[nt][n], a[0], c[0], a[1], c[1], q0[nt].x, q0[nt].y);
            mma_f16(sc[nt][n], a[2], c[2], a[3], c[3], q1[nt].x, q1[nt].y);
          }
        }
      }
      }
      // ---- softmax
      uint32_t pb[NT][2][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[n][e] = fmaf(sc[nt][n][e], fac[nt][e & 1], -m[nt][e & 1]);
        if constexpr (kEdge) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (key + 16 * n + k_row + 8 * (e >> 1) >= lim[nt][e & 1]) x[n][e] = -INFINITY;
        }
        // the reference moves when a logit passes it by kPMost (log2 units)
        const float top = fmax3(fmax3(x[0][0], x[0][1], x[0][2]), fmax3(x[0][3], x[1][0], x[1][1]),
                                fmaxf(x[1][2], x[1][3]));
        if (__any_sync(0xffffffffu, top > kPMost)) {
          // from the logits again: subtracting kNone has lost their bits
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float y = kNone;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int e = i; e < 4; e += 2) {
                x[n][e] = x[n][e] == -INFINITY ? -INFINITY : sc[nt][n][e] * fac[nt][i];
                y = fmaxf(y, x[n][e]);
              }
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
            y = fmaxf(m[nt][i], y - kPHead);
            const float alpha = ex2f(m[nt][i] - y);
            m[nt][i] = y;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int e = i; e < 4; e += 2) x[n][e] -= y;
            l[nt][i] *= alpha;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              o[nt][j][i] *= alpha;
              o[nt][j][i + 2] *= alpha;
            }
          }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[n][e] = ex2f(x[n][e]);
            l[nt][e & 1] += x[n][e];
          }
          pb[nt][n][0] = movmatrix(pack_f16x2(x[n][0], x[n][1]));
          pb[nt][n][1] = movmatrix(pack_f16x2(x[n][2], x[n][3]));
        }
      }
      // ---- O^T += V^T P^T
      if constexpr (kEdge && kScrub) {
        // a NaN of V would pass through P = 0 to rows that do not see its key:
        // the rows that do get it now, and its scale becomes 0 in the stage
        int first_nan[St::VS];  // by block of 16 dims: the step's first key with a NaN
        bool some = false;
#pragma unroll
        for (int k = 0; k < St::VS; ++k) first_nan[k] = INT_MAX;
        auto scale_at = [&](int i) -> uint8_t* {
          const int row = 8 * (i >> 1) + (i & 1 ? v_row[1] : v_row[0]);
          return smem + (st - smem) + St::OFF_VS + row * St::SROW + g * St::VB / 8;
        };
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          const uint8_t* at = scale_at(i);
#pragma unroll
          for (int k = 0; k < St::VS; ++k)
            if ((at[k] & 0x7F) == 0x7F) {
              some = true;
              first_nan[k] = min(first_nan[k], key + 8 * (i >> 1) + (i & 1 ? v_row[1] : v_row[0]));
            }
        }
        // (at head_dim 64 lanes g and g ^ 1 have one byte: both read it before one clears it)
        __syncwarp();
        if (__any_sync(0xffffffffu, some)) {
#pragma unroll
          for (int k = 0; k < St::VS; ++k) {
            int at = first_nan[k];  // of the block's 4 lanes
            at = min(at, __shfl_xor_sync(0xffffffffu, at, 1));
            at = min(at, __shfl_xor_sync(0xffffffffu, at, 2));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                if (at < lim[nt][i]) {
#pragma unroll
                  for (int j = 8 * k; j < (St::VS == 1 ? D / 16 : 8 * k + 8); ++j)
                    o[nt][j][i] = o[nt][j][i + 2] = __int_as_float(0x7FFFFFFF);
                }
          }
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            uint8_t* at = scale_at(i);
#pragma unroll
            for (int k = 0; k < St::VS; ++k)
              if ((D > 64 || g % 2 == 0) && (at[k] & 0x7F) == 0x7F) at[k] = 0;
          }
          __syncwarp();
        }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        uint32_t vw[4][St::VB / 4], vs[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int more = 16 * n + 8 * (i >> 1);
          lds<St::VB>(vw[i], st + v_at[i & 1] + more * St::ROW);
          vs[i] = lds_scales<St::VS>(st + St::OFF_VS + (v_row[i & 1] + more) * St::SROW + g * St::VB / 8);
        }
#pragma unroll
        for (int w = 0; w < St::VB / 4; ++w) {  // 8 dims of each key
          const uint32_t pair = (w >> 1) * 0x11u + 0x40u;  // byte w >> 1 of two keys' scales
          const uint32_t s01 = e4m3x2_f16(__byte_perm(vs[0], vs[1], pair));
          const uint32_t s89 = e4m3x2_f16(__byte_perm(vs[2], vs[3], pair));
          uint32_t a[4], b4[4], c[4], d[4];
          e2m1x8(select_nibbles(vw[0][w], vw[1][w] << 4), a);
          e2m1x8(select_nibbles(vw[0][w] >> 4, vw[1][w]), b4);
          e2m1x8(select_nibbles(vw[2][w], vw[3][w] << 4), c);
          e2m1x8(select_nibbles(vw[2][w] >> 4, vw[3][w]), d);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a[i] = mul_f16x2(a[i], s01);
            b4[i] = mul_f16x2(b4[i], s01);
            c[i] = mul_f16x2(c[i], s89);
            d[i] = mul_f16x2(d[i], s89);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16(o[nt][4 * w + i], a[i], b4[i], c[i], d[i], pb[nt][n][0], pb[nt][n][1]);
          }
        }
      }
    };
    int s = member;
    for (; s < steps && key_a + (s + 1) * kStepKeys <= all_end; s += team) step(s, std::false_type{});
    for (; s < steps; s += team) step(s, std::true_type{});

    // ---- the team's states are joined
    cp_async_wait<0>();
    __syncwarp();
    float* mine_s = o_s + member * team_step;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], d);
        const int n = nt * 8 + 2 * t + i;
        if (g == 0) *reinterpret_cast<float2*>(mine_s + OFF_ML + 2 * n) = make_float2(m[nt][i], l[nt][i]);
        float* dst = mine_s + n * C::O_STRIDE + g * (D / 8);
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
          *reinterpret_cast<float4*>(dst + 4 * j) = make_float4(o[nt][2 * j][i], o[nt][2 * j][i + 2],
                                                                o[nt][2 * j + 1][i], o[nt][2 * j + 1][i + 2]);
      }
    team_sync();
    auto out_row = [&](int n) -> int64_t {
      const int tok = token_of(n);
      return static_cast<int64_t>(rq.qo_start + tok0 + tok) * p.Hq + h * p.G + head0 + n - tok * p.G;
    };
    const int64_t part = ((static_cast<int64_t>(slice) * p.g.Hkv + h) * 2 + (first_segment ? 0 : 1)) * C::ROWS;
    for (int i = rank; i < rows * (D / 4); i += team * 32) {
      const int n = i / (D / 4), d = (i % (D / 4)) * 4;
      float top = kNone;
      for (int w = 0; w < team; ++w) top = fmaxf(top, o_s[w * team_step + OFF_ML + 2 * n]);
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < team; ++w) {
        const float2 ml = *reinterpret_cast<const float2*>(o_s + w * team_step + OFF_ML + 2 * n);
        const float a = ex2f(ml.x - top);
        const float4 v = *reinterpret_cast<const float4*>(o_s + w * team_step + n * C::O_STRIDE + d);
        sum += a * ml.y;
        acc.x += a * v.x;
        acc.y += a * v.y;
        acc.z += a * v.z;
        acc.w += a * v.w;
      }
      // a row that sees no key: zeros, and -inf as its lse
      const float inv = sum == 0.f ? 0.f : (whole ? p.v_scale : 1.f) / sum;
      const float lse2 = sum == 0.f ? -INFINITY : top + kPHead + log2f(sum * 0x1p-7f);  // (a logarithm near 0)
      acc.x *= inv;
      acc.y *= inv;
      acc.z *= inv;
      acc.w *= inv;
      if (whole) {
        const int64_t row = out_row(n);
        *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + row * D + d) =
            make_uint2(Elt<T>::from_f2(acc.x, acc.y), Elt<T>::from_f2(acc.z, acc.w));
        if (d == 0 && p.lse) p.lse[row] = lse2 * kLn2f;
      } else {
        *reinterpret_cast<float4*>(p.part_o + (part + n) * D + d) = acc;
        if (d == 0) p.part_lse[part + n] = lse2;
      }
    }
    if (!whole) {
      // ---- the last slice of a cut row tile joins its parts:
      // o = sum_s 2^(lse_s - lse) o_s.  The sum's order is the slices', so
      // the result does not depend on which one comes last.
      const long long step = by_parts ? 1 : per_slice;
      const int sa = static_cast<int>(quotient(tile_u, step)), sb = static_cast<int>(quotient(tile_u + n_parts - 1, step));
      const bool sa_first = tile_u == sa * step;
      team_sync();
      if (rank == 0) {
        __threadfence();
        int32_t* count = p.counters + (sa + 1) * p.g.Hkv + h;
        const int last = atomicAdd(count, 1) == sb - sa;
        if (last) *count = 0;  // for the next run
        last_s[cta_head] = last;
      }
      team_sync();
      if (last_s[cta_head]) {
        __threadfence();
        auto part_row = [&](int sl) -> int64_t {
          const int which = (sl == sa && !sa_first) ? 1 : 0;
          return ((static_cast<int64_t>(sl) * p.g.Hkv + h) * 2 + which) * C::ROWS;
        };
        auto from = [&](int k) { return part_row(sa + k); };
        if (rows * (D / 4) <= team * 32) join_parts<T, D, 1, 8>(p, rank, team * 32, rows, sb - sa + 1, from, out_row);
        else join_parts<T, D, 4, 2>(p, rank, team * 32, rows, sb - sa + 1, from, out_row);
      }
    }
    team_sync();  // the rings are the next row tile's
    first_segment = false;
    u = seg_end;
    if (u < u_end && rt + 1 == row_tiles(p, rq, C::ROWS)) {  // on to the next request with units
      req_u += static_cast<long long>(row_tiles(p, rq, C::ROWS)) * kts;  // (never by parts)
      do {
        if (++b >= p.batch) return;
        rq = b < kept_b ? req_s[b - first_b] : load_req(p, b);
      } while (row_tiles(p, rq, C::ROWS) == 0);
    }
  }
}

// 8-row groups of a tile: as many as the longest request needs, of 1, 2 or 4
// (the registers of head_dim 256 allow one).
int row_groups(const Kv4Shape& s) {
  if (s.D == 256 || s.max_rows <= 8) return 1;
  return s.max_rows <= 16 ? 2 : 4;
}

template <typename T, int D, int NT, bool kScrub>
cudaError_t launch_small(const Kv4Params& p, cudaStream_t stream) {
  using C = SmallCfg<D, NT>;
  const unsigned grid = static_cast<unsigned>(p.slices) * (p.g.Hkv / p.cta_heads);
  static std::atomic<uint64_t> set{0};
  auto* k = kv4_small_kernel<T, D, NT, kScrub>;
  cudaError_t e = set_smem_once(set, reinterpret_cast<const void*>(k), C::SMEM);
  return e != cudaSuccess ? e : launch_pdl(k, grid, unsigned(C::THREADS), size_t(C::SMEM), stream, p);
}

// One token a request, the commonest batch by far, does without the scrubbing
// (256 decodes 250 us, with it 253; 64 x 4 drafts 149 without, 152 with).
template <typename T, int D, int NT>
cudaError_t launch_nt(const Kv4Params& p, const Kv4Shape& s, cudaStream_t stream) {
  return p.causal && s.max_rows > s.G ? launch_small<T, D, NT, true>(p, stream)
                                      : launch_small<T, D, NT, false>(p, stream);
}

template <typename T, int D>
cudaError_t launch_d(const Kv4Params& p, const Kv4Shape& s, cudaStream_t stream) {
  if constexpr (D == 256) {
    return launch_nt<T, 256, 1>(p, s, stream);
  } else {
    switch (row_groups(s)) {
      case 1: return launch_nt<T, D, 1>(p, s, stream);
      case 2: return launch_nt<T, D, 2>(p, s, stream);
      default: return launch_nt<T, D, 4>(p, s, stream);
    }
  }
}

template <typename T>
cudaError_t launch_t(const Kv4Params& p, const Kv4Shape& s, cudaStream_t stream) {
  switch (s.D) {
    case 64: return launch_d<T, 64>(p, s, stream);
    case 128: return launch_d<T, 128>(p, s, stream);
    default: return launch_d<T, 256>(p, s, stream);
  }
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

Kv4Layout kv4_layout(const Kv4Shape& s) {
  Kv4Layout l;
  const int nt = row_groups(s);
  const int per_sm = small_ctas(s.D, nt), warps = small_warps(s.D, nt);
  l.cta_heads = 1;
  // (tiles of 4 row groups keep q in shared memory, one head a CTA)
  for (int n = 2; n <= 8 && warps % n == 0 && s.Hkv % n == 0 && s.D * nt < 512; n *= 2)
    if (int64_t(per_sm) * s.num_sms * n <= int64_t(3) * s.batch * s.Hkv / 2) l.cta_heads = n;
  const int slices = per_sm * s.num_sms * l.cta_heads / s.Hkv;
  l.slices = slices > 0 ? slices : 1;
  // partial rows of the most slices that any batch size gives (cta_heads 8),
  // so that the size depends on the shape alone
  const size_t most = size_t(per_sm) * s.num_sms * 8 > size_t(s.Hkv) ? size_t(per_sm) * s.num_sms * 8 : size_t(s.Hkv);
  const size_t pre = s.max_rows > kKv4SmallRows ? size_t(kv4_prefill_part_rows(s)) : 0;  // the two kernels take turns
  const size_t rows = most * 2 * 8 * nt > pre ? most * 2 * 8 * nt : pre;
  l.off_counters = 256;  // after the status word
  // the counters' place is the same for every shape: they have to stay zero
  // between runs (slices * Hkv, where there is more than one slice, is at most 8
  // for each CTA of the card)
  l.off_part_o = up256(l.off_counters + size_t(2) * s.num_sms * 8 * sizeof(int32_t));
  l.off_part_lse = up256(l.off_part_o + rows * s.D * sizeof(float));
  l.total = up256(l.off_part_lse + rows * sizeof(float));
  return l;
}

cudaError_t launch_kv4_attention(const Kv4Params& p, const Kv4Shape& s, int dtype, cudaStream_t stream) {
  return dtype == PA_BF16 ? launch_t<__nv_bfloat16>(p, s, stream) : launch_t<__half>(p, s, stream);
}

}  // namespace pa
