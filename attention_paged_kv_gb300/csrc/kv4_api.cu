// C entry points of the device-built tables and the 4-bit cache (declared in
// include/pagedattn.h): argument checks and launches.
#include <cmath>
#include <cstring>
#include <string>

#include "common.cuh"
#include "checks.h"
#include "internal.h"
#include "kv4.h"

using pa::cuda_err;
using pa::set_err;

namespace {

using pa::aligned;
using pa::check_dtype;
using pa::check_heads;
using pa::device_sms;
using pa::page_shift;

pagedattn_status check_cache(const pagedattn_kv4_cache* c, pa::Kv4Geom* g) {
  if (!c) return set_err(PA_ERR_INVALID_ARG, "cache is NULL");
  if (!c->codes || !c->scales) return set_err(PA_ERR_INVALID_ARG, "the cache's codes and scales are required");
  if (!aligned(c->codes, 32) || !aligned(c->scales, 32))
    return set_err(PA_ERR_INVALID_ARG, "the cache's codes and scales must be 32-byte aligned");
  pagedattn_status s = check_heads(c->num_kv_heads, c->num_kv_heads, c->head_dim);
  if (s != PA_OK) return s;
  const int shift = page_shift(c->page_size);
  if (shift < 0) return set_err(PA_ERR_UNSUPPORTED, "page_size must be a power of two in [1, 128]");
  if (c->num_pages < 1) return set_err(PA_ERR_INVALID_ARG, "num_pages must be positive");
  if (c->kv_layout != PA_LAYOUT_NHD && c->kv_layout != PA_LAYOUT_HND)
    return set_err(PA_ERR_UNSUPPORTED, "kv_layout must be PA_LAYOUT_NHD or PA_LAYOUT_HND");
  for (float x : {c->k_scale, c->v_scale})
    if (!(x >= 1e-15f && x <= 1e15f))  // (the append's divisions are exact to the last bit in this range)
      return set_err(PA_ERR_INVALID_ARG, "k_scale and v_scale must lie in [1e-15, 1e15]");
  g->Hkv = c->num_kv_heads;
  g->ps = c->page_size;
  g->ps_shift = shift;
  g->num_pages = c->num_pages;
  const bool hnd = c->kv_layout == PA_LAYOUT_HND;
  g->slot_rows = hnd ? 1 : c->num_kv_heads;
  g->head_rows = hnd ? c->page_size : 1;
  return PA_OK;
}

}  // namespace

extern "C" {

pagedattn_status pagedattn_build_tables(const pagedattn_tables_in* in, const pagedattn_tables_out* out,
                                        pagedattn_stream_t stream) {
  if (!in || !out) return set_err(PA_ERR_INVALID_ARG, "in and out are required");
  if (in->batch_size < 0 || in->block_table_width < 0 || in->free_capacity < 0 || out->max_tokens < 0 ||
      out->max_pages < 0)
    return set_err(PA_ERR_INVALID_ARG, "a size is negative");
  if (in->batch_size > (1 << 30) || out->max_tokens > (1 << 30) || out->max_pages > (1 << 30))
    return set_err(PA_ERR_UNSUPPORTED, "batch_size, max_tokens and max_pages must be at most 2^30");
  if (in->block_table_stride < in->block_table_width)
    return set_err(PA_ERR_INVALID_ARG, "block_table_stride is below block_table_width");
  if (in->num_pages < 1) return set_err(PA_ERR_INVALID_ARG, "num_pages must be positive");
  const int shift = page_shift(in->page_size);
  if (shift < 0) return set_err(PA_ERR_UNSUPPORTED, "page_size must be a power of two in [1, 128]");
  const void* need[] = {in->qo_lens, in->kv_lens, out->kv_last_page_len, out->kv_lens};
  for (const void* p : need)
    if (in->batch_size > 0 && !p) return set_err(PA_ERR_INVALID_ARG, "a per-request array is NULL");
  if (!in->free_count || !out->free_count || !out->qo_indptr || !out->kv_page_indptr || !out->new_page_indptr ||
      !out->status || (in->batch_size > 0 && in->block_table_width > 0 && !in->block_table) ||
      (in->free_capacity > 0 && !in->free_pages) || (out->max_pages > 0 && !out->kv_page_indices) ||
      (out->max_tokens > 0 && (!out->slot_mapping || !out->positions)))
    return set_err(PA_ERR_INVALID_ARG, "a required array is NULL");
  if (!aligned(out->slot_mapping, 8)) return set_err(PA_ERR_INVALID_ARG, "slot_mapping must be 8-byte aligned");
  int sms = 0;
  pagedattn_status s = device_sms(&sms);
  if (s != PA_OK) return s;
  pa::TablesParams p;
  p.qo_lens = in->qo_lens;
  p.kv_lens = in->kv_lens;
  p.block_table = in->block_table;
  p.free_pages = in->free_pages;
  p.free_count = in->free_count;
  p.qo_indptr = out->qo_indptr;
  p.kv_page_indptr = out->kv_page_indptr;
  p.new_page_indptr = out->new_page_indptr;
  p.kv_page_indices = out->kv_page_indices;
  p.kv_last_page_len = out->kv_last_page_len;
  p.kv_lens_out = out->kv_lens;
  p.slot_mapping = out->slot_mapping;
  p.positions = out->positions;
  p.free_count_out = out->free_count;
  p.status = out->status;
  p.table_stride = in->block_table_stride;
  p.table_width = in->block_table_width;
  p.free_capacity = in->free_capacity;
  p.batch = in->batch_size;
  p.ps = in->page_size;
  p.ps_shift = shift;
  p.num_pages = in->num_pages;
  p.max_tokens = out->max_tokens;
  p.max_pages = out->max_pages;
  cudaError_t e = pa::launch_tables(p, sms, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_err(e, "tables launch");
  return PA_OK;
}

pagedattn_status pagedattn_kv4_append(const pagedattn_kv4_cache* cache, const pagedattn_kv4_rows* rows,
                                      pagedattn_stream_t stream) {
  pa::Kv4AppendParams p;
  std::memset(&p, 0, sizeof(p));
  pagedattn_status s = check_cache(cache, &p.g);
  if (s != PA_OK) return s;
  if (!rows) return set_err(PA_ERR_INVALID_ARG, "rows is NULL");
  s = check_dtype(rows->dtype);
  if (s != PA_OK) return s;
  if (rows->num_tokens < 0) return set_err(PA_ERR_INVALID_ARG, "num_tokens is negative");
  if (rows->num_tokens > (1 << 30)) return set_err(PA_ERR_UNSUPPORTED, "num_tokens must be at most 2^30");
  if (rows->num_tokens == 0) return PA_OK;
  const int64_t width = int64_t(cache->num_kv_heads) * cache->head_dim;
  if (!rows->k || !rows->v || !rows->slot_mapping || !rows->status)
    return set_err(PA_ERR_INVALID_ARG, "k, v, slot_mapping and status are required");
  if (!aligned(rows->k, 16) || !aligned(rows->v, 16) || !aligned(rows->k_values, 16) || !aligned(rows->v_values, 16))
    return set_err(PA_ERR_INVALID_ARG, "k, v, k_values and v_values must be 16-byte aligned");
  if (!aligned(rows->slot_mapping, 8)) return set_err(PA_ERR_INVALID_ARG, "slot_mapping must be 8-byte aligned");
  if (rows->num_tokens > 1)
    for (int64_t st : {rows->k_stride, rows->v_stride})
      if (st < width || st % 8)
        return set_err(PA_ERR_INVALID_ARG, "token strides must be multiples of 8 that hold num_kv_heads * head_dim");
  int sms = 0;
  s = device_sms(&sms);
  if (s != PA_OK) return s;
  p.codes = static_cast<uint8_t*>(cache->codes);
  p.scales = static_cast<uint8_t*>(cache->scales);
  p.k = rows->k;
  p.v = rows->v;
  p.k_values = rows->k_values;
  p.v_values = rows->v_values;
  p.slots = rows->slot_mapping;
  p.status = rows->status;
  p.k_stride = rows->k_stride;
  p.v_stride = rows->v_stride;
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.n = rows->num_tokens;
  cudaError_t e = pa::launch_kv4_append(p, cache->head_dim, rows->dtype, sms, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_err(e, "append launch");
  return PA_OK;
}

pagedattn_status pagedattn_kv4_workspace_size(int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
                                              int32_t max_qo_len, size_t* bytes) {
  if (!bytes) return set_err(PA_ERR_INVALID_ARG, "bytes is NULL");
  pagedattn_status s = check_heads(num_qo_heads, num_kv_heads, head_dim);
  if (s != PA_OK) return s;
  if (max_qo_len < 0) return set_err(PA_ERR_INVALID_ARG, "max_qo_len is negative");
  pa::Kv4Shape shape;
  s = device_sms(&shape.num_sms);
  if (s != PA_OK) return s;
  shape.D = head_dim;
  shape.Hkv = num_kv_heads;
  shape.G = num_qo_heads / num_kv_heads;
  const int64_t rows = int64_t(max_qo_len) * shape.G;
  shape.max_rows = rows < (1 << 30) ? int32_t(rows) : (1 << 30);
  shape.batch = 1;
  *bytes = pa::kv4_layout(shape).total;
  return PA_OK;
}

pagedattn_status pagedattn_kv4_run(const pagedattn_kv4_cache* cache, const pagedattn_kv4_batch* batch, const void* q,
                                   int64_t q_stride, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                   pagedattn_stream_t stream) {
  pa::Kv4Params p;
  std::memset(&p, 0, sizeof(p));
  pagedattn_status s = check_cache(cache, &p.g);
  if (s != PA_OK) return s;
  if (!batch) return set_err(PA_ERR_INVALID_ARG, "batch is NULL");
  s = check_heads(batch->num_qo_heads, cache->num_kv_heads, cache->head_dim);
  if (s != PA_OK) return s;
  s = check_dtype(batch->dtype);
  if (s != PA_OK) return s;
  if (batch->batch_size < 0 || batch->num_tokens < 0 || batch->num_page_indices < 0 || batch->max_qo_len < 0)
    return set_err(PA_ERR_INVALID_ARG, "a size is negative");
  if (int64_t(batch->num_tokens) * batch->num_qo_heads > 0x3FFFFFFF)
    return set_err(PA_ERR_UNSUPPORTED, "num_tokens * num_qo_heads must be below 2^30");
  if (!workspace || !aligned(workspace, 256))
    return set_err(PA_ERR_INVALID_ARG, "a 256-byte aligned workspace is required");
  pa::Kv4Shape shape;
  s = device_sms(&shape.num_sms);
  if (s != PA_OK) return s;
  shape.D = cache->head_dim;
  shape.Hkv = cache->num_kv_heads;
  shape.G = batch->num_qo_heads / cache->num_kv_heads;
  const int64_t rows = int64_t(batch->max_qo_len) * shape.G;
  shape.max_rows = rows < (1 << 30) ? int32_t(rows) : (1 << 30);
  shape.batch = batch->batch_size;
  const pa::Kv4Layout lay = pa::kv4_layout(shape);
  if (workspace_bytes < lay.total)
    return set_err(PA_ERR_WORKSPACE_TOO_SMALL, "workspace needs " + std::to_string(lay.total) + " bytes, got " +
                                                   std::to_string(workspace_bytes));
  if (batch->batch_size == 0 || batch->num_tokens == 0) return PA_OK;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16))
    return set_err(PA_ERR_INVALID_ARG, "q and out are required and must be 16-byte aligned");
  const int64_t width = int64_t(batch->num_qo_heads) * cache->head_dim;
  if (batch->num_tokens > 1 && (q_stride < width || q_stride % 8))
    return set_err(PA_ERR_INVALID_ARG, "q_stride must be a multiple of 8 that holds num_qo_heads * head_dim");
  if (!batch->qo_indptr || !batch->kv_page_indptr || !batch->kv_last_page_len ||
      (batch->num_page_indices > 0 && !batch->kv_page_indices))
    return set_err(PA_ERR_INVALID_ARG, "qo_indptr, kv_page_indptr, kv_page_indices and kv_last_page_len are required");
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.q = q;
  p.out = out;
  p.lse = lse;
  p.codes = static_cast<const uint8_t*>(cache->codes);
  p.scales = static_cast<const uint8_t*>(cache->scales);
  p.qo_indptr = batch->qo_indptr;
  p.page_indptr = batch->kv_page_indptr;
  p.pages = batch->kv_page_indices;
  p.last_page_len = batch->kv_last_page_len;
  p.status = reinterpret_cast<int32_t*>(ws);
  p.counters = reinterpret_cast<int32_t*>(ws + lay.off_counters);
  p.part_o = reinterpret_cast<float*>(ws + lay.off_part_o);
  p.part_lse = reinterpret_cast<float*>(ws + lay.off_part_lse);
  p.q_stride = q_stride;
  p.batch = batch->batch_size;
  p.num_tokens = batch->num_tokens;
  p.num_page_indices = batch->num_page_indices;
  p.Hq = batch->num_qo_heads;
  p.G = shape.G;
  p.causal = batch->causal ? 1 : 0;
  // no more slices than the tables can hold work for (the workspace's layout
  // stays): 64-key units of at most this many row tiles, 4 to a slice
  const int64_t tiles = int64_t(batch->num_tokens) * shape.G / 8 + 1;
  const int64_t key_units = int64_t(batch->num_page_indices) * cache->page_size / 64 + batch->batch_size;
  const int64_t most = (key_units * tiles + 3) / 4;
  p.slices = most < lay.slices ? int32_t(most) : lay.slices;
  p.cta_heads = lay.cta_heads;
  // (both rules below go by the size of the page list, all that the host knows
  // of the keys: a list far larger than the pages in use costs time, see the header)
  // requests of few keys are not worth cutting: the CTAs for it would only
  // lengthen the launch (tables of 8 key tiles a request on average, or more)
  p.num_sms = shape.num_sms;
  // one row tile and two CTAs an SM up to 4 key tiles a request on average: 32
  // prompts of up to 100 tokens at 32 / 8 heads 27.6 us against 36.2, of up to
  // 400 104 against 108, 16 of up to 1024 172 against 163
  p.short_keys = int64_t(batch->num_page_indices) * cache->page_size <= int64_t(4) * 128 * batch->batch_size;
  p.split_ctas = int64_t(batch->num_page_indices) * cache->page_size >= int64_t(8) * 128 * batch->batch_size
                     ? 2 * shape.num_sms : 0;
  // the bound alone decides whether the tensor-core kernel is launched; where
  // it is not, the small-query kernel takes every request
  const bool prefill = shape.max_rows > pa::kKv4SmallRows;
  p.small_rows = prefill ? pa::kKv4SmallRows : 0x7FFFFFFF;
  p.scale_log2 = float(1.4426950408889634 / std::sqrt(double(cache->head_dim)) * double(cache->k_scale));
  p.v_scale = cache->v_scale;
  cudaError_t e = cudaSuccess;
  if (prefill) e = pa::launch_kv4_prefill(p, shape, batch->dtype, reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaErrorLaunchOutOfResources)  // what the launcher returns where the build's registers differ
    return cuda_err(e, "4-bit prefill launch (are the built kernel's registers those that its warps hand over?)");
  if (e != cudaSuccess) return cuda_err(e, "4-bit prefill launch");
  e = pa::launch_kv4_attention(p, shape, batch->dtype, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_err(e, "4-bit attention launch");
  return PA_OK;
}

pagedattn_status pagedattn_status_word(int32_t* word, pagedattn_stream_t stream, int32_t* flags) {
  if (!word || !flags) return set_err(PA_ERR_INVALID_ARG, "word and flags are required");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int32_t v = 0;
  cudaError_t e = cudaMemcpyAsync(&v, word, sizeof(v), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaMemsetAsync(word, 0, sizeof(v), st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_err(e, "status word read");
  *flags = v;
  if (v & PA_DEV_TIMEOUT) return set_err(PA_ERR_TIMEOUT, "an in-kernel wait gave up after its bound");
  if (v) return set_err(PA_ERR_DEVICE_CHECK, "an in-kernel check fired (flags " + std::to_string(v) + ")");
  return PA_OK;
}

}  // extern "C"
