// C entry points of the calls over the 16-bit cache through device tables
// (declared in include/pagedattn.h): argument checks and launches.
#include <cmath>
#include <cstring>
#include <string>

#include "checks.h"
#include "common.cuh"
#include "paged.h"

using pa::aligned;
using pa::check_dtype;
using pa::check_heads;
using pa::cuda_err;
using pa::device_sms;
using pa::page_shift;
using pa::set_err;

namespace {

constexpr int32_t kMostTokens = 1 << 30;

pagedattn_status check_cache(const pagedattn_kv_cache* c, pa::Kv4Geom* g) {
  if (!c) return set_err(PA_ERR_INVALID_ARG, "cache is NULL");
  if (!c->data || !aligned(c->data, 16))
    return set_err(PA_ERR_INVALID_ARG, "the cache's data is required and must be 16-byte aligned");
  if (!c->bounds != !c->bound_scales)
    return set_err(PA_ERR_INVALID_ARG, "bounds and bound_scales come together");
  if (!aligned(c->bounds, 16) || !aligned(c->bound_scales, 4))
    return set_err(PA_ERR_INVALID_ARG, "the cache's bounds must be 16-byte aligned, bound_scales 4-byte");
  pagedattn_status s = check_heads(c->num_kv_heads, c->num_kv_heads, c->head_dim);
  if (s != PA_OK) return s;
  s = check_dtype(c->dtype);
  if (s != PA_OK) return s;
  const int shift = page_shift(c->page_size);
  if (shift < 0) return set_err(PA_ERR_UNSUPPORTED, "page_size must be a power of two in [1, 128]");
  if (c->num_pages < 1) return set_err(PA_ERR_INVALID_ARG, "num_pages must be positive");
  if (c->kv_layout != PA_LAYOUT_NHD && c->kv_layout != PA_LAYOUT_HND)
    return set_err(PA_ERR_UNSUPPORTED, "kv_layout must be PA_LAYOUT_NHD or PA_LAYOUT_HND");
  g->Hkv = c->num_kv_heads;
  g->ps = c->page_size;
  g->ps_shift = shift;
  g->num_pages = c->num_pages;
  const bool hnd = c->kv_layout == PA_LAYOUT_HND;
  g->slot_rows = hnd ? 1 : c->num_kv_heads;
  g->head_rows = hnd ? c->page_size : 1;
  return PA_OK;
}

pagedattn_status check_bounds(const pagedattn_kv_cache* c) {
  if (!c->bounds) return set_err(PA_ERR_INVALID_ARG, "the cache has no bounds");
  return PA_OK;
}

pagedattn_status check_rotation(const pagedattn_rotation* r, int32_t head_dim, const int32_t* positions,
                                int64_t position_stride) {
  if (!r->turns || !aligned(r->turns, 8)) return set_err(PA_ERR_INVALID_ARG, "turns is required and must be 8-byte aligned");
  if (r->rotary_dim < 16 || r->rotary_dim % 16 || r->rotary_dim > head_dim)
    return set_err(PA_ERR_UNSUPPORTED, "rotary_dim must be a multiple of 16 in [16, head_dim]");
  if (r->num_axes < 1) return set_err(PA_ERR_INVALID_ARG, "num_axes must be positive");
  if (!(std::fabs(r->scale) <= 1e15f)) return set_err(PA_ERR_INVALID_ARG, "the rotation's scale must lie in [-1e15, 1e15]");
  if (!positions || !aligned(positions, 4)) return set_err(PA_ERR_INVALID_ARG, "positions is required");
  if (position_stride < 0) return set_err(PA_ERR_INVALID_ARG, "position_stride is negative");
  return PA_OK;
}

pagedattn_status check_stride(int64_t stride, int64_t width, int32_t n, const char* name) {
  if (n > 1 && (stride < width || stride % 8))
    return set_err(PA_ERR_INVALID_ARG, std::string(name) + " must be a multiple of 8 that holds a token's heads");
  return PA_OK;
}

void set_rotation(pa::RowsParams* p, const pagedattn_rotation* r, const int32_t* positions, int64_t stride, bool inverse) {
  p->turns = r->turns;
  p->axes = r->axes;
  p->num_axes = r->num_axes;
  p->positions = positions;
  p->position_stride = stride;
  p->pairs = r->rotary_dim / 2;
  p->scale = r->scale;
  p->sign = inverse ? -1.f : 1.f;
}

pagedattn_status check_shape(int32_t Hkv, int32_t D, int32_t page_size, const pagedattn_block_batch* b,
                             pa::BlockShape* shape) {
  if (!b) return set_err(PA_ERR_INVALID_ARG, "batch is NULL");
  pagedattn_status s = check_heads(b->num_qo_heads, Hkv, D);
  if (s != PA_OK) return s;
  if (page_shift(page_size) < 0) return set_err(PA_ERR_UNSUPPORTED, "page_size must be a power of two in [1, 128]");
  if (b->batch_size < 0 || b->num_tokens < 0 || b->num_page_indices < 0 || b->max_pages < 0 || b->max_qo_len < 0)
    return set_err(PA_ERR_INVALID_ARG, "a size is negative");
  if (b->batch_size > (1 << 30)) return set_err(PA_ERR_UNSUPPORTED, "batch_size must be at most 2^30");
  if (int64_t(b->num_tokens) * b->num_qo_heads > 0x3FFFFFFF)
    return set_err(PA_ERR_UNSUPPORTED, "num_tokens * num_qo_heads must be below 2^30");
  if (b->num_blocks < 1 || b->num_blocks > pa::kMaxListed)
    return set_err(PA_ERR_UNSUPPORTED, "num_blocks must lie in [1, " + std::to_string(pa::kMaxListed) + "]");
  s = device_sms(&shape->num_sms);
  if (s != PA_OK) return s;
  shape->D = D;
  shape->Hkv = Hkv;
  shape->G = b->num_qo_heads / Hkv;
  shape->num_tokens = b->num_tokens;
  shape->num_blocks = b->num_blocks;
  shape->max_pages = b->max_pages;
  shape->batch = b->batch_size;
  shape->page_size = page_size;
  shape->max_qo_len = b->max_qo_len;
  return PA_OK;
}

// What the selection and the attention both check.
pagedattn_status check_batch(const pagedattn_kv_cache* cache, const pagedattn_block_batch* b, const int32_t* blocks,
                             const void* q, int64_t q_stride, void* workspace, size_t workspace_bytes,
                             pa::BlockParams* p, pa::BlockShape* shape, pa::BlockLayout* lay, bool* empty) {
  pagedattn_status s = check_cache(cache, &p->g);
  if (s != PA_OK) return s;
  if (!workspace || !aligned(workspace, 256))
    return set_err(PA_ERR_INVALID_ARG, "a 256-byte aligned workspace is required");
  s = check_shape(cache->num_kv_heads, cache->head_dim, cache->page_size, b, shape);
  if (s != PA_OK) return s;
  *lay = pa::block_layout(*shape);
  if (workspace_bytes < lay->total)
    return set_err(PA_ERR_WORKSPACE_TOO_SMALL, "workspace needs " + std::to_string(lay->total) + " bytes, got " +
                                                   std::to_string(workspace_bytes));
  *empty = b->batch_size == 0 || b->num_tokens == 0;
  if (*empty) return PA_OK;
  if (!q || !aligned(q, 16)) return set_err(PA_ERR_INVALID_ARG, "q is required and must be 16-byte aligned");
  if (!blocks || !aligned(blocks, 4)) return set_err(PA_ERR_INVALID_ARG, "blocks is required");
  s = check_stride(q_stride, int64_t(b->num_qo_heads) * cache->head_dim, b->num_tokens, "q_stride");
  if (s != PA_OK) return s;
  if (!b->qo_indptr || !b->kv_page_indptr || !b->kv_last_page_len || (b->num_page_indices > 0 && !b->kv_page_indices))
    return set_err(PA_ERR_INVALID_ARG, "qo_indptr, kv_page_indptr, kv_page_indices and kv_last_page_len are required");
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p->q = q;
  p->data = cache->data;
  p->bounds = cache->bounds;
  p->bound_scales = cache->bound_scales;
  p->qo_indptr = b->qo_indptr;
  p->page_indptr = b->kv_page_indptr;
  p->pages = b->kv_page_indices;
  p->last_page_len = b->kv_last_page_len;
  p->blocks = const_cast<int32_t*>(blocks);
  p->status = reinterpret_cast<int32_t*>(ws);
  p->counters = reinterpret_cast<int32_t*>(ws + lay->off_counters);
  p->keys = reinterpret_cast<uint32_t*>(ws + lay->off_scratch);
  p->part_o = reinterpret_cast<float*>(ws + lay->off_scratch);
  p->part_lse = reinterpret_cast<float*>(ws + lay->off_part_lse);
  p->tile_indptr = reinterpret_cast<int32_t*>(ws + lay->off_indptr);
  p->small_indptr = p->tile_indptr + b->batch_size + 1;
  p->items = reinterpret_cast<pa::BlockItem*>(ws + lay->off_items);
  p->entries = reinterpret_cast<int2*>(ws + lay->off_entries);
  p->masks = reinterpret_cast<uint16_t*>(ws + lay->off_masks);
  p->hnd = cache->kv_layout == PA_LAYOUT_HND;
  p->num_sms = shape->num_sms;
  p->q_stride = q_stride;
  p->batch = b->batch_size;
  p->num_page_indices = b->num_page_indices;
  p->num_tokens = b->num_tokens;
  p->Hq = b->num_qo_heads;
  p->G = shape->G;
  p->num_blocks = b->num_blocks;
  p->first = b->first;
  p->last = b->last;
  p->max_pages = b->max_pages;
  p->scale_log2 = float(1.4426950408889634 / std::sqrt(double(cache->head_dim)));
  return PA_OK;
}

}  // namespace

namespace pa {

BlockLayout block_layout(const BlockShape& s) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  BlockLayout l;
  l.off_counters = 256;
  l.off_scratch = l.off_counters + up(size_t(kCutItems) * s.num_sms * 4);
  // Keys of items that are cut, or that are too many for shared memory: then in
  // launches of as many tokens as 64 MB hold.
  int64_t tokens = s.num_tokens, rows = int64_t(s.num_tokens) * s.Hkv;
  if (s.max_pages > kKeptKeys) {
    const int64_t fit = (int64_t(64) << 20) / (int64_t(s.max_pages) * 4 * s.Hkv);
    tokens = fit < 1 ? 1 : (fit < tokens ? fit : tokens);
    rows = tokens * s.Hkv;
  } else if (rows > int64_t(kCutItems) * s.num_sms) {
    rows = int64_t(kCutItems) * s.num_sms;
  }
  l.select_tokens = int32_t(tokens > 0 ? tokens : 1);
  const TileShape t = tile_shape(s);
  const int64_t parts = attend_part_rows(s) + tile_part_rows(s, t);
  const SelectShape chunk = select_shape(s);
  size_t keys = size_t(rows) * s.max_pages * 4;
  const size_t states = size_t(parts) * s.D * 4, tile_keys = chunk.tokens ? size_t(chunk.ctas) * 16 * chunk.row * 4 : 0;
  if (tile_keys > keys) keys = tile_keys;
  l.off_part_lse = l.off_scratch + up(states);
  const size_t attend_end = l.off_part_lse + up(size_t(parts) * 4);
  size_t end = l.off_scratch + up(keys) > attend_end ? l.off_scratch + up(keys) : attend_end;
  // chunks: the requests' sums, and the unions of the lists with their masks
  const size_t items = size_t(t.max_tiles) * s.Hkv;
  l.off_indptr = end;
  l.off_items = l.off_indptr + (t.use || chunk.tokens ? up((size_t(s.batch) + 2) * 8) : 0);
  l.off_entries = l.off_items + up(items * sizeof(BlockItem));
  l.off_masks = l.off_entries + up(items * t.max_entries * sizeof(int2));
  l.total = l.off_masks + up(items * (t.use ? t.max_entries / (128 / s.page_size) : 0) * t.tokens * 2);
  return l;
}

}  // namespace pa

extern "C" {

pagedattn_status pagedattn_rope(const pagedattn_rotation* rotation, const pagedattn_rope_rows* rows,
                                pagedattn_stream_t stream) {
  if (!rotation || !rows) return set_err(PA_ERR_INVALID_ARG, "rotation and rows are required");
  pagedattn_status s = check_dtype(rows->dtype);
  if (s != PA_OK) return s;
  const int32_t n = rows->num_tokens, D = rows->head_dim;
  if (n < 0 || rows->num_q_heads < 0 || rows->num_k_heads < 0) return set_err(PA_ERR_INVALID_ARG, "a size is negative");
  if (n > kMostTokens) return set_err(PA_ERR_UNSUPPORTED, "num_tokens must be at most 2^30");
  if (rows->num_q_heads > 65535 || rows->num_k_heads > 65535) return set_err(PA_ERR_UNSUPPORTED, "more than 65535 heads");
  if (D < 16 || D > 256 || D % 16) return set_err(PA_ERR_UNSUPPORTED, "head_dim must be a multiple of 16 in [16, 256]");
  if (n == 0 || rows->num_q_heads + rows->num_k_heads == 0) return PA_OK;
  s = check_rotation(rotation, D, rows->positions, rows->position_stride);
  if (s != PA_OK) return s;
  pa::RowsParams p;
  std::memset(&p, 0, sizeof(p));
  int parts = 0;
  auto add = [&](const void* in, void* out, int64_t in_stride, int64_t out_stride, int32_t heads, const char* name) {
    if (heads == 0) return PA_OK;
    if (!in || !out || !aligned(in, 16) || !aligned(out, 16))
      return set_err(PA_ERR_INVALID_ARG, std::string(name) + " and its output are required and must be 16-byte aligned");
    for (int64_t st : {in_stride, out_stride}) {
      const pagedattn_status e = check_stride(st, int64_t(heads) * D, n, "a token stride");
      if (e != PA_OK) return e;
    }
    if (in == out && in_stride != out_stride && n > 1)
      return set_err(PA_ERR_INVALID_ARG, std::string(name) + " in place needs the same stride");
    p.part[parts++] = pa::RowsPart{in, out, in_stride, out_stride, heads, 0, 0, 1};
    return PA_OK;
  };
  s = add(rows->q, rows->q_out, rows->q_stride, rows->q_out_stride, rows->num_q_heads, "q");
  if (s != PA_OK) return s;
  s = add(rows->k, rows->k_out, rows->k_stride, rows->k_out_stride, rows->num_k_heads, "k");
  if (s != PA_OK) return s;
  int sms = 0;
  s = device_sms(&sms);
  if (s != PA_OK) return s;
  set_rotation(&p, rotation, rows->positions, rows->position_stride, rows->inverse != 0);
  p.n = n;
  p.D = D;
  const cudaError_t e = pa::launch_rows(p, parts, rotation->interleaved != 0, rows->dtype, sms,
                                        reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_err(e, "rotation launch");
  return PA_OK;
}

pagedattn_status pagedattn_kv_append(const pagedattn_kv_cache* cache, const pagedattn_rotation* rotation,
                                     const pagedattn_kv_rows* rows, pagedattn_stream_t stream) {
  pa::RowsParams p;
  std::memset(&p, 0, sizeof(p));
  pagedattn_status s = check_cache(cache, &p.g);
  if (s != PA_OK) return s;
  if (!rows) return set_err(PA_ERR_INVALID_ARG, "rows is NULL");
  const int32_t n = rows->num_tokens, D = cache->head_dim;
  if (n < 0 || rows->num_qo_heads < 0) return set_err(PA_ERR_INVALID_ARG, "a size is negative");
  if (n > kMostTokens) return set_err(PA_ERR_UNSUPPORTED, "num_tokens must be at most 2^30");
  if (rows->num_qo_heads > 65535) return set_err(PA_ERR_UNSUPPORTED, "more than 65535 heads");
  if (n == 0) return PA_OK;
  if (!rows->k || !rows->v || !rows->slot_mapping || !rows->status)
    return set_err(PA_ERR_INVALID_ARG, "k, v, slot_mapping and status are required");
  if (!aligned(rows->k, 16) || !aligned(rows->v, 16) || !aligned(rows->q, 16) || !aligned(rows->q_out, 16))
    return set_err(PA_ERR_INVALID_ARG, "k, v, q and q_out must be 16-byte aligned");
  if (!aligned(rows->slot_mapping, 8)) return set_err(PA_ERR_INVALID_ARG, "slot_mapping must be 8-byte aligned");
  const int64_t width = int64_t(cache->num_kv_heads) * D, q_width = int64_t(rows->num_qo_heads) * D;
  if ((s = check_stride(rows->k_stride, width, n, "k_stride")) != PA_OK) return s;
  if ((s = check_stride(rows->v_stride, width, n, "v_stride")) != PA_OK) return s;
  if (rotation && (s = check_rotation(rotation, D, rows->positions, rows->position_stride)) != PA_OK) return s;
  int parts = 0;
  if (rows->q && rows->num_qo_heads > 0) {
    if (!rotation) return set_err(PA_ERR_INVALID_ARG, "q needs a rotation");
    if (!rows->q_out) return set_err(PA_ERR_INVALID_ARG, "q_out is required with q");
    if ((s = check_stride(rows->q_stride, q_width, n, "q_stride")) != PA_OK) return s;
    if ((s = check_stride(rows->q_out_stride, q_width, n, "q_out_stride")) != PA_OK) return s;
    if (rows->q == rows->q_out && rows->q_stride != rows->q_out_stride && n > 1)
      return set_err(PA_ERR_INVALID_ARG, "q in place needs the same stride");
    p.part[parts++] = pa::RowsPart{rows->q, rows->q_out, rows->q_stride, rows->q_out_stride, rows->num_qo_heads, 0, 0, 1};
  }
  p.part[parts++] = pa::RowsPart{rows->k, nullptr, rows->k_stride, 0, cache->num_kv_heads, 0, 0, rotation ? 1 : 0};
  p.part[parts++] = pa::RowsPart{rows->v, nullptr, rows->v_stride, 0, cache->num_kv_heads, 0, 1, 0};
  int sms = 0;
  s = device_sms(&sms);
  if (s != PA_OK) return s;
  if (rotation) set_rotation(&p, rotation, rows->positions, rows->position_stride, false);
  p.cache = cache->data;
  p.slots = rows->slot_mapping;
  p.status = rows->status;
  p.n = n;
  p.D = D;
  const cudaError_t e = pa::launch_rows(p, parts, rotation && rotation->interleaved, cache->dtype, sms,
                                        reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_err(e, "append launch");
  if (cache->bounds) return pagedattn_kv_bounds(cache, rows->slot_mapping, n, rows->status, stream);
  return PA_OK;
}

pagedattn_status pagedattn_kv_bounds(const pagedattn_kv_cache* cache, const int64_t* slot_mapping, int32_t num_tokens,
                                     int32_t* status, pagedattn_stream_t stream) {
  pa::BoundsParams p;
  std::memset(&p, 0, sizeof(p));
  pagedattn_status s = check_cache(cache, &p.g);
  if (s != PA_OK) return s;
  s = check_bounds(cache);
  if (s != PA_OK) return s;
  if (num_tokens < 0) return set_err(PA_ERR_INVALID_ARG, "num_tokens is negative");
  if (num_tokens > kMostTokens) return set_err(PA_ERR_UNSUPPORTED, "num_tokens must be at most 2^30");
  if (num_tokens == 0) return PA_OK;
  if (!slot_mapping || !status) return set_err(PA_ERR_INVALID_ARG, "slot_mapping and status are required");
  if (!aligned(slot_mapping, 8)) return set_err(PA_ERR_INVALID_ARG, "slot_mapping must be 8-byte aligned");
  int sms = 0;
  s = device_sms(&sms);
  if (s != PA_OK) return s;
  p.data = cache->data;
  p.bounds = cache->bounds;
  p.scales = cache->bound_scales;
  p.slots = slot_mapping;
  p.status = status;
  p.n = num_tokens;
  const cudaError_t e = pa::launch_bounds(p, cache->head_dim, cache->dtype, sms, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_err(e, "bounds launch");
  return PA_OK;
}

pagedattn_status pagedattn_blocks_workspace_size(int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                                                 const pagedattn_block_batch* batch, size_t* bytes) {
  if (!bytes) return set_err(PA_ERR_INVALID_ARG, "bytes is NULL");
  pa::BlockShape shape;
  const pagedattn_status s = check_shape(num_kv_heads, head_dim, page_size, batch, &shape);
  if (s != PA_OK) return s;
  *bytes = pa::block_layout(shape).total;
  return PA_OK;
}

pagedattn_status pagedattn_select_blocks(const pagedattn_kv_cache* cache, const pagedattn_block_batch* batch,
                                         const void* q, int64_t q_stride, int32_t* blocks, void* workspace,
                                         size_t workspace_bytes, pagedattn_stream_t stream) {
  pa::BlockParams p;
  std::memset(&p, 0, sizeof(p));
  pa::BlockShape shape;
  pa::BlockLayout lay;
  bool empty = false;
  pagedattn_status s = check_batch(cache, batch, blocks, q, q_stride, workspace, workspace_bytes, &p, &shape, &lay, &empty);
  if (s != PA_OK) return s;
  s = check_bounds(cache);
  if (s != PA_OK) return s;
  if (batch->first < 0 || batch->last < 1 || int64_t(batch->first) + batch->last > batch->num_blocks)
    return set_err(PA_ERR_INVALID_ARG, "first must not be negative, last positive, and both fit num_blocks");
  if (empty) return PA_OK;
  const cudaError_t e = pa::launch_select(p, shape, lay.select_tokens, cache->dtype, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_err(e, "selection launch");
  return PA_OK;
}

pagedattn_status pagedattn_blocks_run(const pagedattn_kv_cache* cache, const pagedattn_block_batch* batch,
                                      const int32_t* blocks, const void* q, int64_t q_stride, void* out, float* lse,
                                      void* workspace, size_t workspace_bytes, pagedattn_stream_t stream) {
  pa::BlockParams p;
  std::memset(&p, 0, sizeof(p));
  pa::BlockShape shape;
  pa::BlockLayout lay;
  bool empty = false;
  pagedattn_status s = check_batch(cache, batch, blocks, q, q_stride, workspace, workspace_bytes, &p, &shape, &lay, &empty);
  if (s != PA_OK || empty) return s;
  if (!out || !aligned(out, 16)) return set_err(PA_ERR_INVALID_ARG, "out is required and must be 16-byte aligned");
  if (!aligned(lse, 4)) return set_err(PA_ERR_INVALID_ARG, "lse must be 4-byte aligned");
  p.out = out;
  p.lse = lse;
  const pa::TileShape tiles = pa::tile_shape(shape);
  cudaError_t e = cudaSuccess;
  if (tiles.use) {
    // tensor maps over the cache, and over q in boxes of a row tile's tokens
    pa::HostPlan view;
    view.D = shape.D;
    view.Hkv = shape.Hkv;
    view.Hq = batch->num_qo_heads;
    view.G = shape.G;
    view.ps = cache->page_size;
    view.num_pages = cache->num_pages;
    view.hnd = p.hnd;
    view.dtype = cache->dtype;
    view.T = batch->num_tokens;
    CUtensorMap kv_map, q_map;
    s = pa::encode_kv_map(&kv_map, view, cache->data, 64, uint32_t(cache->page_size), CU_TENSOR_MAP_SWIZZLE_128B);
    if (s != PA_OK) return s;
    s = pa::encode_q_map(&q_map, view, q, 128, batch->num_tokens > 1 ? q_stride : 0);
    if (s != PA_OK) return s;
    p.max_entries = tiles.max_entries;
    p.max_tiles = tiles.max_tiles;
    p.tile_tokens = tiles.tokens;
    p.tile_rows = tiles.rows;
    p.long_tokens = tiles.long_tokens;
    p.least_long = tiles.least_long;
    e = pa::launch_block_tiles(p, shape, tiles, kv_map, q_map, cache->dtype, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_err(e, "chunk attention launch");
    p.listed = 1;
    p.part_base = pa::tile_part_rows(shape, tiles);
  }
  e = pa::launch_block_attention(p, shape, cache->dtype, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_err(e, "attention launch");
  return PA_OK;
}

}  // extern "C"
