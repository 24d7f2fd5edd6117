// Host-side internals of the calls over the 16-bit cache through device
// tables: kernel parameters and launchers.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/pagedattn.h"
#include "kv4.h"

namespace pa {

// ---------------------------------------------------------------------------
// rows.cu

// One run of heads of a token's row: where it is read and where it goes.
struct RowsPart {
  const void* in;
  void* out;                      // nullptr: the cache
  int64_t in_stride, out_stride;  // elements between tokens
  int32_t heads, groups;          // groups: of heads that a thread takes one after the other
  int32_t half;                   // of the cache: 0 K, 1 V
  int32_t rotate;
};

struct RowsParams {
  RowsPart part[3];
  void* cache;
  const int64_t* slots;
  int32_t* status;
  const uint64_t* turns;
  const int32_t* axes;  // nullptr: axis 0
  const int32_t* positions;
  int64_t position_stride;
  Kv4Geom g;  // of the cache; a row is head_dim values
  int32_t n, D, pairs, num_axes, group_heads;
  float scale, sign;  // sign -1: the inverse rotation
};

cudaError_t launch_rows(RowsParams p, int parts, bool interleaved, int dtype, int num_sms, cudaStream_t stream);

struct BoundsParams {
  const void* data;
  int8_t* bounds;
  float* scales;
  const int64_t* slots;
  int32_t* status;
  Kv4Geom g;
  int32_t n, warp_tokens;
};

cudaError_t launch_bounds(BoundsParams p, int D, int dtype, int num_sms, cudaStream_t stream);

// ---------------------------------------------------------------------------
// select.cu and block_attn.cu

// The tokens of two row tiles of a long request, for one kv head.
struct BlockItem {
  int32_t token, tokens;   // first one in q, how many
  int32_t entries;         // of the union of their lists
  int32_t diag;            // first step of 128 keys with a block that some token sees in part
  int32_t pos, kv_len;     // position of the first token, keys of the request
  int32_t few;             // some token may see fewer than 128 keys
  int32_t unused;
};

struct BlockParams {
  const void* q;
  const void* data;
  const int8_t* bounds;
  const float* bound_scales;
  const int32_t *qo_indptr, *page_indptr, *pages, *last_page_len;
  int32_t* blocks;  // [num_tokens][Hkv][num_blocks]: written by the selection, read by the attention
  void* out;
  float* lse;
  int32_t* status;
  int32_t* counters;  // slices done of each item; 0 between calls
  uint32_t* keys;     // selection: order keys of the scores, [item of the launch][max_pages]
  float* part_o;      // attention: normalised partial states, [slice][rows][D]
  float* part_lse;    // their log-sums, base 2
  int64_t part_base;  // first row of the single tokens' states, behind those of chunks
  // chunks (block_prefill.cu)
  // [batch + 1]: row-tile pairs of the requests before, tokens of the short ones; behind these the parts of an item
  int32_t *tile_indptr, *small_indptr;
  BlockItem* items;                     // [max_tiles][Hkv]
  int2* entries;                        // of each item, [max_entries]: page id, block
  uint16_t* masks;                      // of each item, [step of 128 keys][tile_tokens]: a bit for 8 keys
  int64_t q_stride;
  Kv4Geom g;
  int32_t max_entries, max_tiles, tile_tokens, tile_rows, long_tokens, hnd;
  int32_t listed;      // the tokens that small_indptr counts, not all
  int32_t least_long;  // tokens of long requests for which these are worth their own kernels
  int32_t num_sms;
  int32_t batch, num_page_indices, num_tokens, Hq, G, num_blocks, first, last, max_pages;
  int32_t token0, slices;  // first token of the launch; slices of an item (listed attention: the most)
  int32_t ctas;            // listed attention: CTAs of a full card
  float scale_log2;
};

struct BlockShape {  // what the launches and their workspace depend on
  int32_t D, Hkv, G, num_sms, num_tokens, num_blocks, max_pages, batch, page_size, max_qo_len;
};

struct BlockLayout {
  // the scratch holds the selection's keys, or the attention's partial states
  size_t off_counters, off_scratch, off_part_lse, off_indptr, off_items, off_entries, off_masks, total;
  int32_t select_tokens;  // tokens of a launch of the selection
};

// Selection: tokens that a CTA takes together (0: each by itself), and the fewest of a request that goes there.
struct SelectShape {
  int32_t tokens, long_tokens, least_long, max_tiles;
  int32_t row, ctas;  // keys kept of a token; CTAs with keys in global memory (0: in shared memory)
};
SelectShape select_shape(const BlockShape& s);
BlockLayout block_layout(const BlockShape& s);

// Items are cut into slices only where they are fewer than this a SM.
constexpr int kCutItems = 4;
constexpr int kKeptKeys = 8192;  // of an item, in shared memory
constexpr int kMaxParts = 16;    // of a chunk's item, along its keys
constexpr int kMaxListed = 4096;

struct AttendShape {  // how a launch of the attention is cut
  int32_t rows, chunks, slices, ctas;  // query heads a CTA, CTAs for a group, most slices of a list, CTAs of a full card
};
AttendShape attend_shape(const BlockShape& s);
// The largest slices * items and rows of a slice that attend_shape gives.
int64_t attend_part_rows(const BlockShape& s);

// tile_indptr and small_indptr: the requests of long_tokens or more in tiles of tile_tokens, and the others' tokens.
cudaError_t launch_order_requests(const BlockParams& p, cudaStream_t stream);
cudaError_t launch_select(BlockParams p, const BlockShape& s, int select_tokens, int dtype, cudaStream_t stream);
// Chunks: which requests go to the tensor-core kernel, and what it keeps in the workspace.
struct TileShape {
  bool use;
  int32_t tokens, long_tokens;     // of an item; the fewest of a request that goes there
  int32_t rows, least_long;        // packed rows of an item; the fewest tokens of such requests in all
  int32_t max_tiles, max_entries;
  int64_t union_smem;
};
TileShape tile_shape(const BlockShape& s);
// Rows of partial states of the items that are cut: of two parts an SM.
inline int64_t tile_part_rows(const BlockShape& s, const TileShape& t) { return t.use ? int64_t(2) * s.num_sms * t.rows : 0; }
cudaError_t launch_block_tiles(BlockParams p, const BlockShape& s, const TileShape& t, const CUtensorMap& kv_map,
                               const CUtensorMap& q_map, int dtype, cudaStream_t stream);
cudaError_t launch_block_attention(BlockParams p, const BlockShape& s, int dtype, cudaStream_t stream);

}  // namespace pa
