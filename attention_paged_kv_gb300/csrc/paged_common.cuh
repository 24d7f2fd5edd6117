// Device helpers that the selection and the attention over selected pages share.
#pragma once

#include <climits>

#include "common.cuh"
#include "paged.h"

namespace pa {

// What a query token knows of its request; pos < 0: it sees no key.
struct Query {
  int page_start, pages, pos;
  bool there;  // false: no request has this token (or its tables cannot be)
};

// A warp's search in 32 parts: the last index in [0, n) with indptr[index] <= x, 0 if there is none.
__device__ __forceinline__ int last_below(const int32_t* indptr, int n, int x) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const bool below = lane == 0 || (at < hi && indptr[at] <= x);
    const unsigned m = __ballot_sync(0xffffffffu, below);
    const int k = m == 0xffffffffu ? 31 : __ffs(~m) - 2;  // the last of the leading lanes below
    lo += k * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// The request of token t, found by a warp: first where the caller guesses it
// (request t, in a decode step), then by a search over qo_indptr.
__device__ __forceinline__ Query find_query(const BlockParams& p, int t, int guess) {
  const int lane = threadIdx.x & 31;
  int b = guess;
  int q0 = -1, q1 = -1, p0 = 0, p1 = 0, last = 0;
  if (b < p.batch) {  // all that is needed of it at once
    q0 = p.qo_indptr[b], q1 = p.qo_indptr[b + 1];
    p0 = p.page_indptr[b], p1 = p.page_indptr[b + 1], last = p.last_page_len[b];
  }
  if (!(q0 >= 0 && q0 <= t && t < q1)) {
    b = last_below(p.qo_indptr, p.batch + 1, t);
    if (b >= p.batch) return Query{0, 0, -1, false};
    q0 = p.qo_indptr[b], q1 = p.qo_indptr[b + 1];
    p0 = p.page_indptr[b], p1 = p.page_indptr[b + 1], last = p.last_page_len[b];
    if (q0 > t) return Query{0, 0, -1, false};
  }
  const long long kv = p1 > p0 ? static_cast<long long>(p1 - p0 - 1) * p.g.ps + last : 0;
  const bool ok = q0 >= 0 && q1 > t && q1 <= p.num_tokens && p0 >= 0 && p1 >= p0 && p1 <= p.num_page_indices &&
                  (p1 == p0 || (last >= 1 && last <= p.g.ps)) && kv <= INT_MAX - 256;
  if (!ok) {
    if (lane == 0) atomicOr(p.status, PA_DEV_BAD_INDEX);
    return Query{0, 0, -1, false};
  }
  return Query{p0, p1 - p0, static_cast<int>(kv) - (q1 - q0) + (t - q0), true};
}

struct Span {  // a request, checked; qo_len 0 where its tables cannot be
  int qo_start, qo_len, page_start, pages, kv_len;
};
__device__ __forceinline__ Span load_span(const BlockParams& p, int b, bool report) {
  const int q0 = p.qo_indptr[b], q1 = p.qo_indptr[b + 1];
  const int p0 = p.page_indptr[b], p1 = p.page_indptr[b + 1], last = p.last_page_len[b];
  const long long kv = p1 > p0 ? static_cast<long long>(p1 - p0 - 1) * p.g.ps + last : 0;
  const bool ok = q0 >= 0 && q1 >= q0 && q1 <= p.num_tokens && p0 >= 0 && p1 >= p0 && p1 <= p.num_page_indices &&
                  (p1 == p0 || (last >= 1 && last <= p.g.ps)) && kv <= INT_MAX - 256;
  if (!ok) {
    if (report) atomicOr(p.status, PA_DEV_BAD_INDEX);
    return Span{0, 0, 0, 0, 0};
  }
  return Span{q0, q1 - q0, p0, p1 - p0, static_cast<int>(kv)};
}

// A page id, checked.
__device__ __forceinline__ int checked_page(const BlockParams& p, int id) {
  if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.g.num_pages)) {
    atomicOr(p.status, PA_DEV_BAD_INDEX);
    id = 0;
  }
  return id;
}
__device__ __forceinline__ int page_of(const BlockParams& p, int at) { return checked_page(p, p.pages[at]); }

__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

}  // namespace pa
