// Page tables, slot maps and positions of one step, built on the device from
// the requests' lengths (pagedattn_build_tables).
//
// With ps = page size, request b holds old_b = ceil(kv_b / ps) pages and
// needs new_b = ceil((kv_b + qo_b) / ps); the new_b - old_b missing ones come
// off the top of the free stack in request order.  Everything else follows
// from exclusive sums over the batch of qo_b, new_b and new_b - old_b:
//   one launch    (batches of up to kTablesShared requests) every CTA makes the
//                 sums itself and fills its share of the lists from shared
//                 memory; per-request outputs are the first CTA's.  Those that
//                 may be the input arrays (kv_lens, free_count) are written by
//                 the CTA that is the last to have read them (a ticket).
//   two launches  (larger batches) a scan by one CTA, then the fill, which
//                 reads only what the scan wrote, the held part of the block
//                 table and the free stack.
// The fill takes one thread per page-list entry and per token: a binary
// search in the sums names the request, so that one request of 10^5 tokens
// costs no more than 10^5 requests of one.  Nothing at all is changed when a
// check fails.
//
// Latency binds both: 64 requests of up to 8191 tokens move 135 KB in 3.8 to 4.3
// us, 2000 requests 2.2 MB in 7.6 (one launch; an eager call costs the host 6.4);
// decode steps of 2900 requests take 9.0 in one launch, of 3500 13.9 in two.
#include <climits>
#include <cstring>

#include "common.cuh"
#include "internal.h"
#include "kv4.h"

namespace pa {
namespace {

constexpr int kScanThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kScanWarps = kScanThreads / 32;

struct Sums {
  long long t, pages, fresh;  // tokens, pages, pages taken off the free stack
};

__device__ __forceinline__ Sums add(const Sums& a, const Sums& b) {
  return Sums{a.t + b.t, a.pages + b.pages, a.fresh + b.fresh};
}

// Lengths of request b and the flags they raise (a request that cannot be is
// counted as empty: its flag stops the whole build).
__device__ __forceinline__ Sums load_request(const TablesParams& p, int b, int* flags) {
  const int qo = p.qo_lens[b], kv = p.kv_lens[b];
  if (qo < 0 || kv < 0 || static_cast<long long>(qo) + kv > INT_MAX - p.ps) {
    *flags |= PA_DEV_BAD_INDEX;
    return Sums{0, 0, 0};
  }
  const int old = (kv + p.ps - 1) >> p.ps_shift, now = (kv + qo + p.ps - 1) >> p.ps_shift;
  if (now > p.table_width) *flags |= PA_DEV_NO_ROOM;
  return Sums{qo, now, now - old};
}

__device__ __forceinline__ Sums shfl_up(const Sums& v, int d) {
  return Sums{__shfl_up_sync(0xffffffffu, v.t, d), __shfl_up_sync(0xffffffffu, v.pages, d),
              __shfl_up_sync(0xffffffffu, v.fresh, d)};
}

// Exclusive sums over the block's threads; *total is the block's sum.
__device__ Sums block_scan(const Sums& v, Sums* warp_sums, Sums* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sums x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Sums y = shfl_up(x, d);
    if (lane >= d) x = add(x, y);
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    Sums w = lane < kScanWarps ? warp_sums[lane] : Sums{0, 0, 0};
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Sums y = shfl_up(w, d);
      if (lane >= d) w = add(w, y);
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  *total = warp_sums[kScanWarps - 1];
  Sums before = warp > 0 ? warp_sums[warp - 1] : Sums{0, 0, 0};
  before = add(before, Sums{x.t - v.t, x.pages - v.pages, x.fresh - v.fresh});
  __syncthreads();  // warp_sums may be used again
  return before;
}

// The request that entry `at` of a list with these sums belongs to: the last
// b with indptr[b] <= at (requests without entries are passed over).
__device__ __forceinline__ int request_of(const int32_t* indptr, int batch, int at) {
  int lo = 0, hi = batch;  // indptr[lo] <= at < indptr[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (indptr[mid] <= at) lo = mid; else hi = mid;
  }
  return lo;
}

// Page `nth` of request b: held already, or the next of the free stack.
__device__ __forceinline__ int page_id(const TablesParams& p, int b, int nth, int old, int first_fresh, int free_count) {
  return nth < old ? p.block_table[static_cast<int64_t>(b) * p.table_stride + nth]
                   : p.free_pages[free_count - 1 - (first_fresh + nth - old)];
}

// Entry i of the page list (i < max_pages) and of the token lists (i <
// max_tokens).  free_before is the count before this step's pages are taken.
__device__ __forceinline__ void fill_entry(const TablesParams& p, const int32_t* qo_indptr, const int32_t* page_indptr,
                                           const int32_t* fresh_indptr, const int32_t* kv_lens, int free_before,
                                           int i) {
  if (i < p.max_pages && i < page_indptr[p.batch]) {
    const int b = request_of(page_indptr, p.batch, i);
    const int nth = i - page_indptr[b], pages = page_indptr[b + 1] - page_indptr[b];
    const int first = fresh_indptr[b], old = pages - (fresh_indptr[b + 1] - first);
    const int id = page_id(p, b, nth, old, first, free_before);
    p.kv_page_indices[i] = id;
    if (nth >= old) p.block_table[static_cast<int64_t>(b) * p.table_stride + nth] = id;
    if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_pages)) atomicOr(p.status, PA_DEV_BAD_INDEX);
  }
  if (i < p.max_tokens) {
    int64_t slot = -1;
    int pos = 0;
    if (i < qo_indptr[p.batch]) {
      const int b = request_of(qo_indptr, p.batch, i);
      const int pages = page_indptr[b + 1] - page_indptr[b];
      const int first = fresh_indptr[b], old = pages - (fresh_indptr[b + 1] - first);
      // the request's tokens end at kv_len: position = kv_len - qo_len + nth
      pos = kv_lens[b] - (qo_indptr[b + 1] - i);
      const int id = page_id(p, b, pos >> p.ps_shift, old, first, free_before);
      if (static_cast<unsigned>(id) < static_cast<unsigned>(p.num_pages))
        slot = (static_cast<int64_t>(id) << p.ps_shift) + (pos & (p.ps - 1));
    }
    p.slot_mapping[i] = slot;
    p.positions[i] = pos;
  }
}

// kFill: the one launch, by any number of CTAs; else the scan, by one.
template <bool kFill, int kPerThread>
__global__ void __launch_bounds__(kScanThreads) tables_scan_kernel(const TablesParams p) {
  __shared__ Sums warp_sums[32];
  __shared__ int flags_s, last_s;
  extern __shared__ int32_t sums_s[];  // kFill: qo, page and fresh sums, batch + 1 of each, then the new kv_lens
  const bool writer = blockIdx.x == 0;
  const int tid = threadIdx.x;
  if (tid == 0) flags_s = 0;
  pdl_wait();  // the lengths may come from the kernel before
  __syncthreads();
  const int free_before = *p.free_count;

  // totals and checks; in the one launch a thread keeps its kPerThread
  // consecutive requests in registers
  constexpr int kKept = kFill ? kPerThread : 1;
  int flags = 0;
  Sums kept[kKept], all{0, 0, 0};
  if constexpr (kFill) {
#pragma unroll
    for (int i = 0; i < kKept; ++i) {
      const int b = tid * kKept + i;
      kept[i] = b < p.batch ? load_request(p, b, &flags) : Sums{0, 0, 0};
      all = add(all, kept[i]);
    }
  } else {
    for (int b = tid; b < p.batch; b += kScanThreads) all = add(all, load_request(p, b, &flags));
  }
  if (flags) atomicOr(&flags_s, flags);
  Sums total;
  Sums before = block_scan(all, warp_sums, &total);
  if (tid == 0) {
    int f = flags_s;
    if (free_before < 0 || free_before > p.free_capacity) f |= PA_DEV_BAD_INDEX;
    else if (total.fresh > free_before) f |= PA_DEV_NO_PAGES;
    if (total.t > p.max_tokens || total.pages > p.max_pages) f |= PA_DEV_NO_ROOM;
    if (f && writer) atomicOr(p.status, f);
    flags_s = f;
  }
  __syncthreads();
  const bool fail = flags_s != 0;

  // per-request outputs (of an empty batch when a check failed)
  Sums carry{0, 0, 0};
  const int rounds = kFill ? kKept : (p.batch + kScanThreads - 1) / kScanThreads;
#pragma unroll
  for (int i = 0; i < rounds; ++i) {
    const int b = kFill ? tid * kKept + i : i * kScanThreads + tid;
    Sums v{0, 0, 0};
    if constexpr (kFill) {
      if (i > 0) before = add(before, kept[i - 1]);
      v = kept[i];
    } else {
      int ignored = 0;
      if (b < p.batch) v = load_request(p, b, &ignored);
      Sums chunk;
      before = add(carry, block_scan(v, warp_sums, &chunk));
      carry = add(carry, chunk);
    }
    if (b < p.batch) {
      const int t = fail ? 0 : static_cast<int>(before.t), pages = fail ? 0 : static_cast<int>(before.pages);
      const int fresh = fail ? 0 : static_cast<int>(before.fresh);
      const int kv = p.kv_lens[b];
      const int n = static_cast<int>(v.pages);
      const int now = fail ? kv : kv + static_cast<int>(v.t);
      if (writer) {
        p.qo_indptr[b] = t;
        p.kv_page_indptr[b] = pages;
        p.new_page_indptr[b] = fresh;
        p.kv_last_page_len[b] = fail || n == 0 ? 0 : now - ((n - 1) << p.ps_shift);
        // (the one CTA of a scan has each element read and written by one thread)
        if constexpr (!kFill) p.kv_lens_out[b] = now;
      }
      if constexpr (kFill) {
        sums_s[b] = t;
        sums_s[p.batch + 1 + b] = pages;
        sums_s[2 * (p.batch + 1) + b] = fresh;
        sums_s[3 * (p.batch + 1) + b] = now;
      }
    }
  }
  if (tid == 0) {
    const int t = fail ? 0 : static_cast<int>(total.t), pages = fail ? 0 : static_cast<int>(total.pages);
    const int fresh = fail ? 0 : static_cast<int>(total.fresh);
    if (writer) {
      p.qo_indptr[p.batch] = t;
      p.kv_page_indptr[p.batch] = pages;
      p.new_page_indptr[p.batch] = fresh;
    }
    if constexpr (kFill) {
      sums_s[p.batch] = t;
      sums_s[2 * p.batch + 1] = pages;
      sums_s[3 * p.batch + 2] = fresh;
    } else {
      *p.free_count_out = free_before - fresh;
    }
  }
  if constexpr (kFill) {
    __syncthreads();  // the sums are there, and this CTA has read what it reads of kv_lens and free_count
    if (tid == 0) {
      __threadfence();
      last_s = atomicAdd(p.status + 1, 1) == static_cast<int>(gridDim.x) - 1;
    }
    const int n = max(p.max_tokens, sums_s[2 * p.batch + 1]);
    for (int i = blockIdx.x * kScanThreads + tid; i < n; i += gridDim.x * kScanThreads)
      fill_entry(p, sums_s, sums_s + p.batch + 1, sums_s + 2 * (p.batch + 1), sums_s + 3 * (p.batch + 1), free_before, i);
    __syncthreads();
    if (last_s) {
      for (int b = tid; b < p.batch; b += kScanThreads) p.kv_lens_out[b] = sums_s[3 * (p.batch + 1) + b];
      if (tid == 0) {
        *p.free_count_out = free_before - sums_s[3 * p.batch + 2];
        p.status[1] = 0;  // for the next build
      }
    }
  }
}

__global__ void __launch_bounds__(kFillThreads) tables_fill_kernel(const TablesParams p) {
  pdl_wait();
  // the count before this step: what is left plus what was taken
  const int free_before = *p.free_count_out + p.new_page_indptr[p.batch];
  const int n = max(p.max_tokens, p.kv_page_indptr[p.batch]);
  for (int i = blockIdx.x * kFillThreads + threadIdx.x; i < n; i += gridDim.x * kFillThreads)
    fill_entry(p, p.qo_indptr, p.kv_page_indptr, p.new_page_indptr, p.kv_lens_out, free_before, i);
}

}  // namespace

cudaError_t launch_tables(const TablesParams& p, int num_sms, cudaStream_t stream) {
  const int longest = p.max_tokens > p.max_pages ? p.max_tokens : p.max_pages;
  if (p.batch <= kTablesShared) {
    // one entry a thread, as far as the SMs go: the entries wait for loads (the
    // scan that every CTA repeats waits for them together)
    const int blocks = (longest + kScanThreads - 1) / kScanThreads;
    const unsigned grid = static_cast<unsigned>(blocks < 1 ? 1 : (blocks < num_sms ? blocks : num_sms));
    const size_t smem = size_t(16) * (p.batch + 1);
    if (p.batch <= kScanThreads)
      return launch_pdl(tables_scan_kernel<true, 1>, grid, unsigned(kScanThreads), smem, stream, p);
    return launch_pdl(tables_scan_kernel<true, 3>, grid, unsigned(kScanThreads), smem, stream, p);
  }
  cudaError_t e = launch_pdl(tables_scan_kernel<false, 1>, 1u, unsigned(kScanThreads), size_t(0), stream, p);
  if (e != cudaSuccess) return e;
  if (longest == 0) return cudaSuccess;  // nothing to fill
  const int blocks = (longest + kFillThreads - 1) / kFillThreads;
  const int most = num_sms * 8;
  return launch_pdl(tables_fill_kernel, unsigned(blocks < most ? blocks : most), unsigned(kFillThreads), size_t(0),
                    stream, p);
}

}  // namespace pa
