// Tensor-core attention of long query chunks over the 4-bit paged cache
// (sm_103a: tcgen05 + TMEM).
//
// One CTA takes NT tiles of 128 packed query rows (token major, the G heads
// of a kv head minor; any G) of one request and one kv head, against all keys
// that its last row sees, or a part of them where the items would leave most
// of the card's last wave idle.  The work is found on the device: every CTA
// sums the requests' tiles and looks its own up; the grid is the host's upper
// bound, and the CTAs behind the last item leave at once.  Tiles are taken
// from the last one down: under a causal mask the last are the longest.
//
// Warp roles (4 warps each; register shares after setmaxnreg):
//   warpgroup x < NT  softmax, correction and epilogue of tile x: thread i
//                     owns row i = TMEM lane i.  It also loads its q row,
//                     brings it to fp16 (bf16 rows by an exact power of two,
//                     see kv4_attn.cu) and stores it as the MMA's operand.
//   warpgroup NT      dequantisation: thread i owns key i of every 128-key
//                     tile; it loads the key's codes and scales a tile ahead,
//                     straight from its page, and writes the fp16 rows of K
//                     and V (exact values: code * scale has 6 bits) into the
//                     128-byte swizzled layout that the MMAs read.  Rows past
//                     the last key are written as zeros, so that whatever
//                     their memory holds cannot pass through P = 0.
//   warpgroup NT + 1  one thread issues the MMAs: S_x = Q_x K^T, O_x += P_x V,
//                     all fp16 with fp32 sums in TMEM.  P is fp16 whatever q's
//                     type (2^-11 relative; small ones see kPHead), so no row needs
//                     P in two parts.
// Per key tile j it issues PV_A(j), S_A(j+1), PV_B(j), S_B(j+1): one tile's
// MMAs run while the other tile's rows are in their softmax.
//
// What bounds it: 2000 tokens behind 6000 at 64 / 8 heads take 360 to 367 us,
// 1250 to 1275 TFLOP/s; the tensor pipe is busy 54 % of the time and a pair of row
// tiles takes 1.68 us a key tile, softmax and MMAs waiting for one another.  32
// prompts of up to 200 tokens at 32 / 8 heads take 38 us, most of it the set-up,
// first loads and epilogue of items with one or two key tiles.  At head_dim 256,
// with one K and one V stage and one row tile, the same chunk (at 32 / 4 heads)
// takes 608 us, 755 TFLOP/s.
//
// TMEM: S_x (fp32 128 x 128) at 128 x, O_x (fp32 128 x D) after them; P_x
// overwrites the first 64 columns of S_x.
#include <cstring>
#include <type_traits>

#include "internal.h"
#include "kv4_common.cuh"

namespace pa {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

// Bounded wait, made uniform across the warp (all lanes leave together).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int32_t* abort_flag,
                                          int32_t* status, long long limit) {
  bool ok = mbar_wait(bar, parity, abort_flag, status, limit);
  return __all_sync(0xffffffffu, ok);
}

// Bounded wait of the MMA thread, which polls and never suspends (as in the
// 16-bit prefill kernel, where waking it cost 1.8 %).
__device__ __forceinline__ bool spin_wait(uint64_t* bar, uint32_t parity, volatile int32_t* abort_flag,
                                          int32_t* status, long long limit) {
  const uint32_t a = smem_u32(bar);
  if (mbar_test_wait(a, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (mbar_test_wait(a, parity)) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > limit) {
      *abort_flag = 1;
      atomicOr(status, PA_DEV_TIMEOUT);
      return false;
    }
  }
}
// Wait that ignores the abort flag (used to drain in-flight async work).
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  const long long t0 = clock64();
  while (!mbar_try_wait(a, parity)) {
    if (clock64() - t0 > PA_WAIT_LIMIT_CYCLES) break;
  }
}

template <int D, int NT>
struct PreCfg {
  static_assert(NT == 1 || (NT == 2 && D <= 128), "two tiles need 2 x (128 + D) <= 512 TMEM columns");
  static constexpr int THREADS = 128 * (NT + 2);
  static constexpr int WARP_DQ = 4 * NT, WARP_MMA = 4 * NT + 4;
  static constexpr int NKB = D / 64;      // 128-byte column blocks of a row
  static constexpr int BLK = 128 * 128;   // one 128-row x 128-byte block
  static constexpr int TILE = NKB * BLK;  // 128 rows of Q, K or V
  static constexpr int NST = NT == 1 ? 1 : 2;
  static constexpr int OFF_K = NT * TILE;
  static constexpr int OFF_V = OFF_K + NST * TILE;
  static constexpr int OFF_BAR = OFF_V + NST * TILE;
  static constexpr int SMEM = OFF_BAR + 256 + 1024;  // barriers + alignment slack
  static_assert(SMEM <= 232448, "shared memory per CTA");
  static constexpr int O_COL = NT * 128;
  static constexpr uint32_t TMEM_COLS = (NT * (128 + D) <= 256) ? 256u : 512u;
  // Registers: the launch's share of every thread is handed over to the
  // warpgroups as they need it, 2 x 176 (softmax) + 72 (dequantisation) + 88
  // (MMA) = 4 x 128 with two tiles, 160 + 48 + 32 = 3 x 80 with one, two CTAs an
  // SM.  (At head_dim 256 the launch's own 168 do for all.)
  static constexpr bool HANDOVER = D < 256;
  static constexpr int CTAS = D < 256 && NT == 1 ? 2 : 1;
  static constexpr int REGS_SOFTMAX = NT == 2 ? 176 : 160, REGS_DQ = NT == 2 ? 72 : 48, REGS_MMA = NT == 2 ? 88 : 32;
  static constexpr int LAUNCH_REGS = NT == 2 ? 128 : 80;
};

template <int N> __device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A key's codes and scales of K or V.  The 32 rows of a warp are 32 lines, and
// the L1 cache looks up one a cycle, so a row is read in as few and as wide
// accesses as there are (with 16 bytes an access the look-ups took 2000 cycles
// a tile, more than the conversion).  (Whole rows to an access, a lane with 16
// bytes of every 8th key, needs fewer still but finds four addresses where
// this finds one: 64 drafting requests of 64 rows 247 -> 277 us.)
template <int D>
struct Row4 {
  uint32_t codes[D / 8];
  uint32_t scales[D / 64];
};

template <int D>
__device__ __forceinline__ void load_row4(Row4<D>& r, const Kv4Params& p, int64_t row, bool live) {
  if (live) {
    const uint8_t* c = p.codes + row * (D / 2);
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
      asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
          : "=r"(r.codes[8 * i]), "=r"(r.codes[8 * i + 1]), "=r"(r.codes[8 * i + 2]), "=r"(r.codes[8 * i + 3]),
            "=r"(r.codes[8 * i + 4]), "=r"(r.codes[8 * i + 5]), "=r"(r.codes[8 * i + 6]), "=r"(r.codes[8 * i + 7])
          : "l"(c + 32 * i));
    const uint8_t* s = p.scales + row * (D / 16);
    if constexpr (D == 64) {
      r.scales[0] = __ldg(reinterpret_cast<const uint32_t*>(s));
    } else if constexpr (D == 128) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(s));
      r.scales[0] = v.x;
      r.scales[1] = v.y;
    } else {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(s));
      r.scales[0] = v.x;
      r.scales[1] = v.y;
      r.scales[2] = v.z;
      r.scales[3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < D / 8; ++i) r.codes[i] = 0;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) r.scales[i] = 0;
  }
}

// Takes the NaN of a row of V out (its scale becomes 0) and notes its key by
// block of 16 dims: through P = 0 it would reach rows that do not see the key.
template <int D>
__device__ __forceinline__ void note_nans(Row4<D>& r, int key, int* first_nan, int* any_nan) {
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    if (__vcmpeq4(r.scales[i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) == 0) continue;
    for (int k = 0; k < 4; ++k)
      if (((r.scales[i] >> (8 * k)) & 0x7Fu) == 0x7Fu) {
        *any_nan = 1;
        atomicMin(first_nan + 4 * i + k, key);
        r.scales[i] &= ~(0xFFu << (8 * k));
      }
  }
}

// Row `key` of a tile at `dst` in fp16, 128-byte swizzled.
template <int D>
__device__ __forceinline__ void store_row4(uint8_t* dst, const Row4<D>& r, int key) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {  // 32 dims: two scales, four 16-byte chunks
    const uint32_t two = r.scales[i >> 1] >> (16 * (i & 1));
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t s = e4m3x2_f16(__byte_perm(two, 0, (w >> 1) * 0x1111u));
      uint32_t h[4];
      e2m1x8(r.codes[4 * i + w], h);
      const int c = (i & 1) * 4 + w;  // 16-byte chunk of the 128-byte block
      *reinterpret_cast<uint4*>(dst + (i >> 1) * (128 * 128) + key * 128 + ((c ^ (key & 7)) << 4)) =
          make_uint4(mul_f16x2(h[0], s), mul_f16x2(h[1], s), mul_f16x2(h[2], s), mul_f16x2(h[3], s));
    }
  }
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(PreCfg<D, NT>::THREADS, PreCfg<D, NT>::CTAS) kv4_prefill_kernel(const Kv4Params p) {
  using C = PreCfg<D, NT>;
  constexpr int NST = C::NST;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ int warp_sums[32], found_tile, last_s;
  __shared__ long long work_s;
  __shared__ Req found_rq;
  __shared__ int any_nan, first_nan[D / 16];     // first key whose V has a NaN there, of the tiles that some row sees in part
  __shared__ float fac_s[NT * kQRows];  // bf16: the rows' powers of two, inverted

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* full_k = bars;             // [NST] K tile written
  uint64_t* full_v = bars + NST;       // [NST] V tile written
  uint64_t* empty_k = bars + 2 * NST;  // [NST] every S MMA done with the slot
  uint64_t* empty_v = bars + 3 * NST;  // [NST] every PV MMA done with the slot
  uint64_t* q_full = bars + 4 * NST;   // the Q tiles written
  uint64_t* s_full = q_full + 1;       // [2] S_x done
  uint64_t* p_full = s_full + 2;       // [2] P_x (and O_x's correction) written
  uint64_t* o_done = p_full + 2;       // [2] the last PV_x done
  uint64_t* fin = o_done + 2;          // every MMA retired
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 24);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(tmem_slot + 1);
  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full_k[i], 4);
      mbar_init(&full_v[i], 4);
      mbar_init(&empty_k[i], 1);
      mbar_init(&empty_v[i], 1);
    }
    mbar_init(q_full, 4 * NT);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_done[i], 1);
    }
    mbar_init(fin, 1);
    *abort_flag = 0;
    work_s = 0;
    mbar_init_fence();
  }
  if (tid < D / 16) first_nan[tid] = INT_MAX;
  if (tid == 0) {
    any_nan = 0;
    found_rq = Req{0, 0, 0, 0};  // of an item that bad tables leave without a request
    found_tile = 0;
  }
  if (warp == C::WARP_MMA) tmem_alloc(tmem_slot, C::TMEM_COLS);
  pdl_wait();  // q, the cache and the tables may come from the kernel before

  // ---- the items: row tiles from the last one down, their kv heads adjacent
  auto tiles_of = [&](const Req& r) -> int {
    const int rows = r.qo_len * p.G;
    return rows > p.small_rows ? (rows + NT * kQRows - 1) / (NT * kQRows) : 0;
  };
  auto sum_before = [&](int v, int* total) -> int {  // exclusive sum over the block
    int x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int before = x - v, all = 0;
#pragma unroll
    for (int w = 0; w < C::THREADS / 32; ++w) {
      if (w < warp) before += warp_sums[w];
      all += warp_sums[w];
    }
    __syncthreads();
    *total = all;
    return before;
  };
  Req my_rq{0, 0, 0, 0};
  int mine = 0;
  long long work = 0;  // key tiles of all row tiles (as if no mask cut them)
  for (int b = tid; b < p.batch; b += C::THREADS) {
    my_rq = load_req(p, b);
    const int n = tiles_of(my_rq);
    mine += n;
    work += static_cast<long long>(n) * ((my_rq.kv_len + kKvTile - 1) / kKvTile);
  }
  int total;
  int before = sum_before(mine, &total);
  if (p.split_ctas > 0 && work > 0) atomicAdd(reinterpret_cast<unsigned long long*>(&work_s), static_cast<unsigned long long>(work));
  // Items are whole but for those that would not fill the last wave of one
  // CTA an SM: they are cut along the keys into `parts` each, as many as make
  // that wave shortest (8 key tiles stand for a part's start and join).
  const int items = total * p.g.Hkv;
  int whole_items = items, parts = 1;
  if (p.split_ctas > 0) {
    __syncthreads();
    const int rem = items % p.num_sms;
    // (requests that overlap, as bad tables may have them, can make more items
    // than the grid has CTAs: a part that never runs would leave its count)
    if (rem > 0 && items <= static_cast<int>(gridDim.x) - p.split_ctas) {
      const float kts = static_cast<float>(work_s) / static_cast<float>(total);
      // lane n - 1 weighs n parts; the cheapest, the fewest among equals
      const int n = lane + 1;
      float cost = static_cast<float>((rem * n + p.num_sms - 1) / p.num_sms) * (kts / n + (n > 1 ? 8.f : 0.f));
      if (n > 1 && rem * (n - 1) > p.split_ctas) cost = INFINITY;
      float best = cost;
#pragma unroll
      for (int d = 16; d; d >>= 1) best = fminf(best, __shfl_xor_sync(0xffffffffu, best, d));
      parts = __ffs(__ballot_sync(0xffffffffu, cost == best));
      if (parts > 1) whole_items = items - rem;
    }
  }
  const int cut_item = static_cast<int>(blockIdx.x) - whole_items;  // in the cut part of the grid
  const int item = cut_item < 0 ? static_cast<int>(blockIdx.x) : whole_items + cut_item / parts;
  if (item >= items) {
    __syncthreads();
    if (warp == C::WARP_MMA) tmem_dealloc(*tmem_slot, C::TMEM_COLS);
    return;
  }
  const int h = item % p.g.Hkv, tile_index = total - 1 - item / p.g.Hkv;
  for (int b0 = 0, base = 0; b0 < p.batch; b0 += C::THREADS) {
    int v = mine, all = total;
    if (p.batch > C::THREADS) {
      my_rq = Req{0, 0, 0, 0};
      if (b0 + tid < p.batch) my_rq = load_req(p, b0 + tid);
      v = tiles_of(my_rq);
      before = base + sum_before(v, &all);
    }
    if (v > 0 && before <= tile_index && tile_index < before + v) {
      found_rq = my_rq;
      found_tile = tile_index - before;
    }
    base += all;
    if (tile_index < base) break;
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const Req rq = found_rq;
  const int row0 = found_tile * NT * kQRows;  // first packed row of the item
  const int rows = min(NT * kQRows, rq.qo_len * p.G - row0);
  const int tok0 = row0 / p.G, head0 = row0 - tok0 * p.G;
  const DivG div_g(p.G);
  // packed row n of the item: token qo_start + tok0 + token_of(n), and its row of out
  auto token_of = [&](int n) { return div_g.div(head0 + n); };
  auto out_row = [&](int n) -> int64_t {
    const int tok = token_of(n);
    return (static_cast<int64_t>(rq.qo_start) + tok0 + tok) * p.Hq + h * p.G + head0 + n - tok * p.G;
  };
  const bool has_b = NT == 2 && rows > kQRows;
  const int shift = rq.kv_len - rq.qo_len + 1;
  const int seen_end = p.causal ? max(0, min(rq.kv_len, shift + tok0 + token_of(rows - 1))) : rq.kv_len;
  // the part's key tiles, from key 128 * kt0 on: keys below count from there
  const int all_kts = (seen_end + kKvTile - 1) / kKvTile;
  const int my_parts = cut_item < 0 ? 1 : max(1, min(parts, all_kts));
  const int part = cut_item < 0 ? 0 : cut_item % parts;
  const bool idle = part >= my_parts;
  const int kt0 = static_cast<int>(static_cast<long long>(all_kts) * part / my_parts);
  const int kt1 = idle ? kt0 : static_cast<int>(static_cast<long long>(all_kts) * (part + 1) / my_parts);
  const int nkt = kt1 - kt0;
  const int key_end = min(seen_end, kt1 * kKvTile);
  // one row tile alone: the two softmax warpgroups take its even and its odd
  // key tiles, as two states joined at the end
  const bool dual = NT == 2 && !has_b && nkt > 1;
  constexpr long long kLimit = PA_WAIT_LIMIT_CYCLES;

  if (warp >= C::WARP_DQ && warp < C::WARP_DQ + 4) {
    // ---------------------------------------------------------------- dequantisation
    if constexpr (C::HANDOVER) regs_down<C::REGS_DQ>();
    const int r = tid - 32 * C::WARP_DQ;  // key of the tile
    const int32_t* ids = p.pages + rq.page_start;
    const int all_end = p.causal ? shift + tok0 : rq.kv_len;  // keys that every row sees
    const int64_t half_rows = static_cast<int64_t>(p.g.ps) * p.g.Hkv;
    auto page_of = [&](int j) -> int {
      const int key = (kt0 + j) * kKvTile + r;
      return key < key_end ? __ldg(ids + (key >> p.g.ps_shift)) : 0;
    };
    auto row_of = [&](int j, int pid) -> int64_t {  // the K row; V's lies half_rows behind it
      const int key = (kt0 + j) * kKvTile + r;
      if (static_cast<unsigned>(pid) >= static_cast<unsigned>(p.g.num_pages)) {
        atomicOr(p.status, PA_DEV_BAD_INDEX);
        pid = 0;
      }
      return static_cast<int64_t>(pid) * 2 * half_rows + static_cast<int64_t>(key & (p.g.ps - 1)) * p.g.slot_rows +
             static_cast<int64_t>(h) * p.g.head_rows;
    };
    int64_t at = row_of(0, page_of(0));
    if constexpr (C::CTAS == 2) {
      // few registers: one row of codes at a time, its load's wait is the other
      // CTA's time
      int next_page = page_of(1);
      for (int j = 0; j < nkt; ++j) {
        const bool live = (kt0 + j) * kKvTile + r < key_end;
        const int st = j % NST;
        const uint32_t parity = ((j / NST) - 1) & 1;
        Row4<D> row;
        load_row4(row, p, at, live);
        if (j >= NST && !warp_wait(&empty_k[st], parity, abort_flag, p.status, kLimit)) break;
        store_row4<D>(smem + C::OFF_K + st * C::TILE, row, r);
        load_row4(row, p, at + half_rows, live);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full_k[st]);
        if (j >= NST && !warp_wait(&empty_v[st], parity, abort_flag, p.status, kLimit)) break;
        if ((kt0 + j + 1) * kKvTile > all_end) note_nans(row, (kt0 + j) * kKvTile + r, first_nan, &any_nan);
        store_row4<D>(smem + C::OFF_V + st * C::TILE, row, r);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full_v[st]);
        at = row_of(j + 1, next_page);
        next_page = page_of(j + 2);
      }
    } else {
      Row4<D> k4, v4;
      load_row4(k4, p, at, kt0 * kKvTile + r < key_end);
      load_row4(v4, p, at + half_rows, kt0 * kKvTile + r < key_end);
      int next_page = page_of(1);
      for (int j = 0; j < nkt; ++j) {
        const int st = j % NST;
        const uint32_t parity = ((j / NST) - 1) & 1;
        const bool more = (kt0 + j + 1) * kKvTile + r < key_end;
        at = row_of(j + 1, next_page);
        next_page = page_of(j + 2);
        if (j >= NST && !warp_wait(&empty_k[st], parity, abort_flag, p.status, kLimit)) break;
        store_row4<D>(smem + C::OFF_K + st * C::TILE, k4, r);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full_k[st]);
        load_row4(k4, p, at, more);
        if (j >= NST && !warp_wait(&empty_v[st], parity, abort_flag, p.status, kLimit)) break;
        if ((kt0 + j + 1) * kKvTile > all_end) note_nans(v4, (kt0 + j) * kKvTile + r, first_nan, &any_nan);
        store_row4<D>(smem + C::OFF_V + st * C::TILE, v4, r);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full_v[st]);
        load_row4(v4, p, at + half_rows, more);
      }
    }
  } else if (warp >= C::WARP_MMA) {
    // ---------------------------------------------------------------- MMA issuer
    if constexpr (C::HANDOVER) regs_down<C::REGS_MMA>();
    if (warp == C::WARP_MMA && lane == 0 && nkt > 0) {
      const uint32_t id_s = idesc_f16(0, 0, 0, 128, 128);
      const uint32_t id_o = idesc_f16(0, 0, 1, 128, D);
      const uint64_t dq0 = smem_desc_sw128(sbase, 16, 1024);
      const uint64_t dk0 = smem_desc_sw128(sbase + C::OFF_K, 16, 1024);
      const uint64_t dv0 = smem_desc_sw128(sbase + C::OFF_V, C::BLK, 1024);
      auto issue_s = [&](int x, int st) {
        const uint64_t qd = dq0 + uint64_t(dual ? 0 : x) * (C::TILE >> 4);
        const uint64_t kd = dk0 + uint64_t(st) * (C::TILE >> 4);
#pragma unroll(NT == 1 ? 1 : D / 16)  // one tile: few registers
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * C::BLK + (k & 3) * 32) >> 4;
          tc_mma_ss(tmem + x * 128, qd + off, kd + off, id_s, k > 0 ? 1u : 0u);
        }
        tc_commit(&s_full[x]);
      };
      auto issue_pv = [&](int x, bool first, bool last, int st) {
        const uint64_t vd = dv0 + uint64_t(st) * (C::TILE >> 4);
#pragma unroll(NT == 1 ? 1 : kKvTile / 16)
        for (int k = 0; k < kKvTile / 16; ++k)
          tc_mma_ts(tmem + C::O_COL + x * 128, tmem + x * 128 + k * 8, vd + (k * 2048 >> 4), id_o,
                    (!first || k > 0) ? 1u : 0u);
        if (last) tc_commit(&o_done[x]);
      };
      bool ok = spin_wait(q_full, 0, abort_flag, p.status, kLimit);
      if (ok) ok = spin_wait(&full_k[0], 0, abort_flag, p.status, kLimit);
      if (ok) {
        tc_fence_after();
        issue_s(0, 0);
        if (has_b) issue_s(1, 0);
        tc_commit(&empty_k[0]);
      }
      if (ok && dual) {
        ok = spin_wait(&full_k[1 % NST], 0, abort_flag, p.status, kLimit);
        if (ok) {
          tc_fence_after();
          issue_s(1, 1 % NST);
          tc_commit(&empty_k[1 % NST]);
        }
      }
      if (!dual) {
        for (int j = 0; ok && j < nkt; ++j) {  // key tile j of both row tiles
          const int st = j % NST, st1 = (j + 1) % NST;
          const bool more = j + 1 < nkt;
          ok = spin_wait(&p_full[0], j & 1, abort_flag, p.status, kLimit);
          if (ok) ok = spin_wait(&full_v[st], (j / NST) & 1, abort_flag, p.status, kLimit);
          if (!ok) break;
          tc_fence_after();
          issue_pv(0, j == 0, !more, st);
          if (more) {
            ok = spin_wait(&full_k[st1], ((j + 1) / NST) & 1, abort_flag, p.status, kLimit);
            if (!ok) break;
            tc_fence_after();
            issue_s(0, st1);
            if (!has_b) tc_commit(&empty_k[st1]);
          }
          if (has_b) {
            ok = spin_wait(&p_full[1], j & 1, abort_flag, p.status, kLimit);
            if (!ok) break;
            tc_fence_after();
            issue_pv(1, j == 0, !more, st);
          }
          tc_commit(&empty_v[st]);
          if (has_b && more) {
            issue_s(1, st1);
            tc_commit(&empty_k[st1]);
          }
        }
      } else {
        for (int j = 0; ok && j < nkt; ++j) {  // key tile j of warpgroup j & 1, whose next is j + 2
          const int st = j % NST, x = j & 1;
          ok = spin_wait(&p_full[x], (j >> 1) & 1, abort_flag, p.status, kLimit);
          if (ok) ok = spin_wait(&full_v[st], (j / NST) & 1, abort_flag, p.status, kLimit);
          if (!ok) break;
          tc_fence_after();
          issue_pv(x, j < 2, j + 2 >= nkt, st);
          tc_commit(&empty_v[st]);
          if (j + 2 < nkt) {
            const int st2 = (j + 2) % NST;
            ok = spin_wait(&full_k[st2], ((j + 2) / NST) & 1, abort_flag, p.status, kLimit);
            if (!ok) break;
            tc_fence_after();
            issue_s(x, st2);
            tc_commit(&empty_k[st2]);
          }
        }
      }
      tc_commit(fin);
      drain_wait(fin, 0);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax warps
    if constexpr (C::HANDOVER) regs_up<C::REGS_SOFTMAX>();
    const int x = warp >> 2;
    const int r = tid & 127;
    const int rx = dual ? 0 : x;            // the warpgroup's row tile
    const int pr = rx * kQRows + r;         // row of the item
    const bool row_valid = pr < rows;
    const bool active = x == 0 || has_b || dual;
    const bool warp_rows = rx * kQRows + (r & ~31) < rows;  // some row of the warp is one
    int row_end = p.causal ? shift + tok0 + token_of(pr) : rq.kv_len;
    row_end = row_valid ? min(row_end, key_end) - kt0 * kKvTile : 0;
    float sl2 = p.scale_log2;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lane_base + x * 128;
    const uint32_t o_col = tmem + lane_base + C::O_COL + x * 128;
    uint8_t* q_row = smem + x * C::TILE + r * 128;  // chunk c of block kb at kb * BLK + ((c ^ (r & 7)) << 4)

    if (active && warp_rows) {
      // the warp's 32 rows of q as fp16, whole rows at a time (a thread loading
      // its own row took 5 us: 32 rows an access); dual: warpgroup 1 needs the
      // factors alone
      constexpr int LPR = D / 8;                      // lanes of a row
      constexpr int RPI = 32 / LPR;                   // rows of an access
      constexpr int NQ = 32 / RPI < 16 ? 32 / RPI : 16;  // accesses in flight
#pragma unroll 1
      for (int i0 = 0; i0 < 32 / RPI; i0 += NQ) {
        uint4 w[NQ];
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
          const int n = rx * kQRows + (warp & 3) * 32 + (i0 + i) * RPI + lane / LPR;  // row of the item
          const int t = token_of(n);
          w[i] = make_uint4(0, 0, 0, 0);
          if (n < rows)
            w[i] = __ldg(reinterpret_cast<const uint4*>(
                static_cast<const T*>(p.q) + (static_cast<int64_t>(rq.qo_start) + tok0 + t) * p.q_stride +
                static_cast<int64_t>(h * p.G + head0 + n - t * p.G) * D + (lane % LPR) * 8));
        }
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
          const int rr = (warp & 3) * 32 + (i0 + i) * RPI + lane / LPR, c = lane % LPR;
          if constexpr (Elt<T>::kBf16) {
            uint32_t m = __vmaxu2(__vmaxu2(w[i].x & 0x7FFF7FFFu, w[i].y & 0x7FFF7FFFu),
                                  __vmaxu2(w[i].z & 0x7FFF7FFFu, w[i].w & 0x7FFF7FFFu));
#pragma unroll
            for (int d2 = 1; d2 < LPR; d2 <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, d2));
            const int up = bf16_row_shift(max(m & 0xFFFFu, m >> 16));
            const float mul = pow2(up);
            if (c == 0) fac_s[x * kQRows + rr] = pow2(-up);
            uint32_t ws[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = Elt<T>::to_f2(ws[e]);
              ws[e] = pack_f16x2(f.x * mul, f.y * mul);
            }
            w[i] = make_uint4(ws[0], ws[1], ws[2], ws[3]);
          }
          if (!dual || x == 0)
            *reinterpret_cast<uint4*>(smem + x * C::TILE + (c >> 3) * C::BLK + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) =
                w[i];
        }
      }
      if constexpr (Elt<T>::kBf16) {
        __syncwarp();
        sl2 = row_factor(sl2, fac_s[x * kQRows + r]);
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(q_full);

    float m_ref = -INFINITY, l_sum = 0.f;
    bool ok = active;
    // the warpgroup's key tiles, and the row's keys that remain at each
    const int mine_kts = dual ? (nkt + 1 - x) >> 1 : nkt;
    int lim = row_end - (dual ? x * kKvTile : 0);
    const int lim_step = dual ? 2 * kKvTile : kKvTile;
    for (int i = 0; ok && i < mine_kts; ++i, lim -= lim_step) {
      ok = warp_wait(&s_full[x], i & 1, abort_flag, p.status, kLimit);
      if (!ok) break;
      tc_fence_after();
      if (!warp_rows) {  // rows of none: whatever stands in P reaches their O alone
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
        continue;
      }
      // the whole S row in registers: four loads, one wait
      uint32_t s[128];
      tmem_ld32(s_col + 0, *reinterpret_cast<uint32_t(*)[32]>(s + 0));
      tmem_ld32(s_col + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
      tmem_ld32(s_col + 64, *reinterpret_cast<uint32_t(*)[32]>(s + 64));
      tmem_ld32(s_col + 96, *reinterpret_cast<uint32_t(*)[32]>(s + 96));
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 128; ++i) asm volatile("" : "+r"(s[i]));
      if (lim < kKvTile) {
#pragma unroll
        for (int i = 0; i < 128; ++i)
          if (i >= lim) s[i] = __float_as_uint(-INFINITY);
      }
      float m43[43];
#pragma unroll
      for (int u = 0; u < 42; ++u)
        m43[u] = fmax3(__uint_as_float(s[3 * u]), __uint_as_float(s[3 * u + 1]), __uint_as_float(s[3 * u + 2]));
      m43[42] = fmaxf(__uint_as_float(s[126]), __uint_as_float(s[127]));
      float m15[15];
#pragma unroll
      for (int u = 0; u < 14; ++u) m15[u] = fmax3(m43[3 * u], m43[3 * u + 1], m43[3 * u + 2]);
      m15[14] = m43[42];
      float m5[5];
#pragma unroll
      for (int u = 0; u < 5; ++u) m5[u] = fmax3(m15[3 * u], m15[3 * u + 1], m15[3 * u + 2]);
      const float mx2 = fmax3(fmax3(m5[0], m5[1], m5[2]), m5[3], m5[4]) * sl2;
      // the reference moves when a logit passes it by kPMost (log2 units)
      float alpha = 1.f;
      bool resc = false;
      if (mx2 > m_ref + kPMost) {
        const float lower = mx2 - kPHead;
        if (m_ref != -INFINITY) {
          alpha = ex2(m_ref - lower);
          resc = true;
        }
        m_ref = lower;
      }
      const float m_use = (m_ref == -INFINITY) ? 0.f : m_ref;
      const float2 sc2 = make_float2(sl2, sl2), nm2 = make_float2(-m_use, -m_use);
      float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t ph[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int k = 32 * c + 2 * i;
          const float2 t2 = __ffma2_rn(make_float2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), sc2, nm2);
          const float a = ex2(t2.x), b = ex2(t2.y);
          acc[(i >> 2) & 1] = __fadd2_rn(acc[(i >> 2) & 1], make_float2(a, b));
          ph[i] = pack_f16x2(a, b);
        }
        tmem_st16(s_col + c * 16, ph);
      }
      // PV_x(j-1) is complete: it was issued before S_x(j), whose commit
      // tracks every MMA issued before it, so O may be rescaled
      if (__any_sync(0xffffffffu, resc)) {
#pragma unroll
        for (int c4 = 0; c4 < D / 32; ++c4) {
          uint32_t o[32];
          tmem_ld32(o_col + c4 * 32, o);
          tmem_wait_ld(o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          tmem_st32(o_col + c4 * 32, o);
        }
      }
      const float2 sum = __fadd2_rn(acc[0], acc[1]);
      l_sum = l_sum * alpha + (sum.x + sum.y);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[x]);
    }

    // ---------------------------------------------------------------- epilogue
    const bool some = nkt > 0;  // the warpgroup had a key tile (dual: two or more)
    if (ok && some) ok = warp_wait(&o_done[x], 0, abort_flag, p.status, kLimit);
    float other_w = 0.f;  // dual: weight of warpgroup 1's state
    float* o_x = reinterpret_cast<float*>(smem + C::OFF_K);  // its O, [128][D + 4], where K and V were
    float2* ml_x = reinterpret_cast<float2*>(o_x + 128 * (D + 4));
    float scale = 1.f;
    if (dual) {
      if (x == 1) {
        if (ok) ok = warp_wait(&o_done[0], 0, abort_flag, p.status, kLimit);  // nothing reads K and V any more
        if (ok && warp_rows) {
          tc_fence_after();
          ml_x[r] = make_float2(m_ref, l_sum);
#pragma unroll
          for (int c4 = 0; c4 < D / 32; ++c4) {
            uint32_t o[32];
            tmem_ld32(o_col + c4 * 32, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int v = 0; v < 8; ++v)
              *reinterpret_cast<uint4*>(o_x + r * (D + 4) + c4 * 32 + 4 * v) =
                  make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
          }
        }
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (x == 0 && warp_rows) {
        const float2 ml = ml_x[r];
        const float top = fmaxf(m_ref, ml.x);
        const float ref = top == -INFINITY ? 0.f : top;
        scale = ex2(m_ref - ref);
        other_w = ex2(ml.x - ref);
        l_sum = l_sum * scale + ml.y * other_w;
        m_ref = top;
      }
    }
    const bool writes = ok && (x == 0 || has_b) && !idle;
    const bool split = my_parts > 1;
    // a cut item's states: part i of item n at (n * parts + i) row tiles
    const int64_t part_tile = split ? static_cast<int64_t>(cut_item / parts) * parts : 0;
    if (writes) {
      tc_fence_after();
      const float m_use = (m_ref == -INFINITY) ? 0.f : m_ref;
      // a row that sees no key: zeros, and -inf as its lse
      const float inv = l_sum == 0.f ? 0.f : (split ? 1.f : p.v_scale) / l_sum;
      const float lse2 = l_sum == 0.f ? -INFINITY : m_use + kPHead + __log2f(l_sum * 0x1p-7f);  // (a logarithm near 0)
      const int64_t part_row = (part_tile + part) * (NT * kQRows) + x * kQRows + r;
      if (row_valid) {
        if (split) p.part_lse[part_row] = lse2;
        else if (p.lse) p.lse[out_row(pr)] = lse2 * kLn2;
      }
      // O scaled: to the part's state, or rounded into the row of q's slot (free
      // since the last S MMA), from where each warp writes whole rows
      if (warp_rows) {
#pragma unroll
        for (int c4 = 0; c4 < D / 32; ++c4) {
          uint32_t o[32];
          float* f = reinterpret_cast<float*>(o);
          if (some) {
            tmem_ld32(o_col + c4 * 32, o);
            tmem_wait_ld(o);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0;
          }
          if (dual) {
#pragma unroll
            for (int v = 0; v < 8; ++v) {
              const float4 w = *reinterpret_cast<const float4*>(o_x + r * (D + 4) + c4 * 32 + 4 * v);
              f[4 * v] = f[4 * v] * scale + w.x * other_w;
              f[4 * v + 1] = f[4 * v + 1] * scale + w.y * other_w;
              f[4 * v + 2] = f[4 * v + 2] * scale + w.z * other_w;
              f[4 * v + 3] = f[4 * v + 3] * scale + w.w * other_w;
            }
          }
          if (split) {
            // through the warp's own rows of q's slot, so that a store covers
            // 128 bytes of 4 rows and not 16 of 32
            uint8_t* rows_s = smem + x * C::TILE + (warp & 3) * 32 * 128;
#pragma unroll
            for (int v = 0; v < 8; ++v)
              *reinterpret_cast<float4*>(rows_s + lane * 128 + ((v ^ (lane & 7)) << 4)) =
                  make_float4(f[4 * v] * inv, f[4 * v + 1] * inv, f[4 * v + 2] * inv, f[4 * v + 3] * inv);
            __syncwarp();
            const int64_t first = part_row - lane;
#pragma unroll
            for (int v = 0; v < 8; ++v) {
              const int rr = v * 4 + (lane >> 3), c = lane & 7;
              const float4 w = *reinterpret_cast<const float4*>(rows_s + rr * 128 + ((c ^ (rr & 7)) << 4));
              if ((r & ~31) + rr + x * kQRows < rows)
                *reinterpret_cast<float4*>(p.part_o + (first + rr) * D + c4 * 32 + c * 4) = w;
            }
            __syncwarp();
          } else {
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const int c = (c4 & 1) * 4 + v;
              const float* e = f + 8 * v;
              *reinterpret_cast<uint4*>(q_row + (c4 >> 1) * C::BLK + ((c ^ (r & 7)) << 4)) =
                  make_uint4(Elt<T>::from_f2(e[0] * inv, e[1] * inv), Elt<T>::from_f2(e[2] * inv, e[3] * inv),
                             Elt<T>::from_f2(e[4] * inv, e[5] * inv), Elt<T>::from_f2(e[6] * inv, e[7] * inv));
            }
          }
        }
      }
      if (!split) {
        __syncwarp();
        constexpr int LPR = D / 8;     // lanes of a row
        constexpr int RPI = 32 / LPR;  // rows of an access
        const int c = lane % LPR;
#pragma unroll 4
        for (int i = 0; i < 32 / RPI; ++i) {
          const int rr = (warp & 3) * 32 + i * RPI + lane / LPR;  // row of the tile
          if (x * kQRows + rr >= rows) break;
          const uint4 w = *reinterpret_cast<const uint4*>(smem + x * C::TILE + (c >> 3) * C::BLK + rr * 128 +
                                                          (((c & 7) ^ (rr & 7)) << 4));
          const int64_t row = out_row(x * kQRows + rr);
          *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + row * D + c * 8) = w;
        }
      }
    }
    if (any_nan && writes && warp_rows) {
      // the NaN that were taken out of V, for the rows that see them
      __syncwarp();
      for (int k = 0; k < D / 16; ++k) {
        if (!row_valid || first_nan[k] >= row_end + kt0 * kKvTile) continue;
        const float nan = __int_as_float(0x7FFFFFFF);
        const int64_t part_row = (part_tile + part) * (NT * kQRows) + x * kQRows + r;
        for (int e = 0; e < 16; ++e) {
          if (split) p.part_o[part_row * D + k * 16 + e] = nan;
          else static_cast<T*>(p.out)[out_row(pr) * D + k * 16 + e] = Elt<T>::from_f(nan);
        }
      }
    }
    if (split && !idle) {
      // ---- the last part of an item joins them all: o = sum_s 2^(lse_s - lse)
      // o_s, in the parts' order whichever comes last.  (A part that gave up
      // has raised its status; it is counted all the same.)
      asm volatile("bar.sync 1, %0;" ::"n"(NT * 128) : "memory");
      if (tid == 0) {
        __threadfence();
        int32_t* count = p.counters + cut_item / parts;
        const int last = atomicAdd(count, 1) == my_parts - 1;
        if (last) *count = 0;  // for the next run
        last_s = last;
      }
      asm volatile("bar.sync 1, %0;" ::"n"(NT * 128) : "memory");
      if (last_s) {
        __threadfence();
        join_parts<T, D, 8, 2>(p, tid, NT * 128, rows, my_parts,
                            [&](int k) -> int64_t { return (part_tile + k) * (NT * kQRows); }, out_row);
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  // a softmax warp that gave up between its P stores and their wait still
  // has TMEM stores in flight: they complete before TMEM is released
  if (warp < C::WARP_DQ) tmem_wait_st();
  tc_fence_before();
  __syncthreads();
  if (warp == C::WARP_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <typename T, int D, int NT>
cudaError_t launch_d(const Kv4Params& p, cudaStream_t stream) {
  using C = PreCfg<D, NT>;
  auto* kernel = kv4_prefill_kernel<T, D, NT>;
  static std::atomic<uint64_t> attr_set{0};
  cudaError_t e = set_smem_once(attr_set, reinterpret_cast<const void*>(kernel), C::SMEM);
  if (e != cudaSuccess) return e;
  if (C::HANDOVER) {
    // the register hand-over adds up to what the launch gives: a build that
    // gives less would wait forever
    static std::atomic<int> regs{0};
    int n = regs.load(std::memory_order_relaxed);
    if (n == 0) {
      cudaFuncAttributes at;
      e = cudaFuncGetAttributes(&at, kernel);
      if (e != cudaSuccess) return e;
      n = at.numRegs;
      regs.store(n, std::memory_order_relaxed);
    }
    if (n != C::LAUNCH_REGS) return cudaErrorLaunchOutOfResources;
  }
  // at most one tile more than its rows need for each request that has any
  const int64_t tile = int64_t(NT) * kQRows;
  const int64_t rows = int64_t(p.num_tokens) * p.G;
  const int64_t some = rows / (p.small_rows + 1);  // requests of more rows than the small kernel takes
  const int64_t tiles = rows / tile + (some < p.batch ? some : p.batch);
  if (tiles == 0) return cudaSuccess;
  if (tiles * p.g.Hkv + p.split_ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return launch_pdl(kernel, unsigned(tiles * p.g.Hkv + p.split_ctas), unsigned(C::THREADS), size_t(C::SMEM), stream, p);
}

template <typename T>
cudaError_t launch_t(const Kv4Params& p, int D, cudaStream_t stream) {
  switch (D) {
    case 64: return p.short_keys ? launch_d<T, 64, 1>(p, stream) : launch_d<T, 64, 2>(p, stream);
    case 128: return p.short_keys ? launch_d<T, 128, 1>(p, stream) : launch_d<T, 128, 2>(p, stream);
    default: return launch_d<T, 256, 1>(p, stream);
  }
}

}  // namespace

// (parts of the cut items: fewer than the items of a wave and split_ctas)
int64_t kv4_prefill_part_rows(const Kv4Shape& s) {
  return int64_t(3) * s.num_sms * (s.D == 256 ? 1 : 2) * kQRows;
}

cudaError_t launch_kv4_prefill(const Kv4Params& p, const Kv4Shape& s, int dtype, cudaStream_t stream) {
  return dtype == PA_BF16 ? launch_t<__nv_bfloat16>(p, s.D, stream) : launch_t<__half>(p, s.D, stream);
}

}  // namespace pa
