// Host-side internals of the device-built tables and the 4-bit cache:
// kernel parameters and launchers.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/pagedattn.h"

namespace pa {

// ---------------------------------------------------------------------------
// tables.cu

struct TablesParams {
  const int32_t* qo_lens;     // [batch]
  const int32_t* kv_lens;     // [batch], before this step's tokens
  int32_t* block_table;       // [batch, table_width]
  const int32_t* free_pages;  // [free_capacity], the top of the stack at free_count - 1
  const int32_t* free_count;
  int32_t *qo_indptr, *kv_page_indptr, *new_page_indptr;      // [batch + 1]
  int32_t *kv_page_indices, *kv_last_page_len, *kv_lens_out;  // [max_pages], [batch], [batch]
  int64_t* slot_mapping;                                      // [max_tokens]
  int32_t* positions;                                         // [max_tokens]
  int32_t* free_count_out;
  int32_t* status;  // status word, then the ticket of the build's CTAs (0 between builds)
  int64_t table_stride;
  int32_t table_width, free_capacity, batch, ps, ps_shift, num_pages, max_tokens, max_pages;
};

// The largest batch whose sums are kept in shared memory (16 bytes each, 48 KB
// without asking for more).
constexpr int kTablesShared = 2900;

cudaError_t launch_tables(const TablesParams& p, int num_sms, cudaStream_t stream);

// ---------------------------------------------------------------------------
// kv4_append.cu

// Offsets of a 4-bit cache's rows.  A row is (page, half, slot, kv head):
// half 0 = K, 1 = V.  In units of rows:
//   ((page * 2 + half) * ps * Hkv) + slot * slot_rows + head * head_rows
struct Kv4Geom {
  int32_t Hkv, ps, ps_shift, num_pages;
  int32_t slot_rows, head_rows;  // NHD: Hkv, 1; HND: 1, ps
};

struct Kv4AppendParams {
  uint8_t *codes, *scales;
  const void *k, *v;
  void *k_values, *v_values;  // nullptr: not wanted
  const int64_t* slots;
  int32_t* status;
  int64_t k_stride, v_stride;  // elements between tokens
  Kv4Geom g;
  float k_scale, v_scale;
  int32_t n;  // tokens
};

cudaError_t launch_kv4_append(const Kv4AppendParams& p, int D, int dtype, int num_sms, cudaStream_t stream);

// ---------------------------------------------------------------------------
// kv4_attn.cu

struct Kv4Params {
  const void* q;
  void* out;
  float* lse;
  const uint8_t *codes, *scales;
  const int32_t *qo_indptr, *page_indptr, *pages, *last_page_len;
  int32_t* status;
  int32_t* counters;  // parts written of each cut row tile and kv head (prefill: of each cut item); 0 between runs
  float* part_o;      // partial states, normalised, v_scale not in them: [slices * Hkv * 2][rows of a tile][D]
                      // (prefill: [parts of the cut items][rows of an item][D])
  float* part_lse;    // their log-sums, base 2
  int64_t q_stride;  // elements between tokens
  Kv4Geom g;
  int32_t batch, num_tokens, num_page_indices, Hq, G, causal, slices, cta_heads;
  int32_t short_keys;  // prefill: requests of few keys, one row tile and two CTAs an SM
  int32_t num_sms, split_ctas;  // prefill: CTAs of the grid for cutting items along the keys (0: never)
  int32_t small_rows;  // requests of more packed rows are the prefill kernel's
  float scale_log2;    // log2(e) / sqrt(D) * k_scale
  float v_scale;
};

struct Kv4Shape {  // what the launch and its workspace depend on
  int32_t D, Hkv, G, num_sms;
  int32_t max_rows;  // packed rows of the longest request
  int32_t batch;     // requests (not for the workspace's size)
};

// Bytes of a run's workspace, and where its parts lie in it.
struct Kv4Layout {
  int32_t slices, cta_heads;
  size_t off_counters, off_part_o, off_part_lse, total;
};
Kv4Layout kv4_layout(const Kv4Shape& s);
// Rows of partial states that the prefill kernel may write.
int64_t kv4_prefill_part_rows(const Kv4Shape& s);

// Requests of more packed rows than this go to the tensor-core kernel.  us, the
// small-query kernel / that one, 64 requests of 512 to 8192 keys at 64 / 8 heads:
//   rows    head_dim 64   128         256
//   16       70 / 179     114 / 233   229 / 476
//   24      100 / 179     149 / 233   329 / 479
//   32      104 / 171     152 / 223   430 / 464
// and 64 requests of 128 to 512 keys with 32 rows at head_dim 128 48 / 37, with
// 16 rows 21 / 38: the one place where it would be the other way round.
constexpr int kKv4SmallRows = 32;

cudaError_t launch_kv4_prefill(const Kv4Params& p, const Kv4Shape& s, int dtype, cudaStream_t stream);
cudaError_t launch_kv4_attention(const Kv4Params& p, const Kv4Shape& s, int dtype, cudaStream_t stream);

}  // namespace pa
