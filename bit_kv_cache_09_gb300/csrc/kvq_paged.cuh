// kvq_paged.cuh — geometry, tile layout and kernel parameters of the paged 8-bit cache
// (library-internal; the memory map is in include/kvq.h).
//
// A tile is 8192 contiguous bytes: 32 tokens of codes (keys, then values) or 16 tokens of
// 16-bit tail rows. Inside it every lane of a warp finds its matrix-product operands (the
// k16 x n8 B operand of m16n8k16: two pairs of consecutive k per lane) in 16-byte pieces
// that lie lane after lane, so a tile is one bulk copy into shared memory and its reads
// there are conflict-free 16-byte loads, without any transposition in the decode kernel.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/kvq.h"

namespace kvq {

constexpr int kPagedDim = 128;        // d_head
constexpr int kTileBytes = 8192;      // one tile
constexpr int kTileCodeTokens = 32;   // tokens of a tile of codes
constexpr int kTileTailTokens = 16;   // tokens of a tile of 16-bit rows
constexpr int kPagedMaxRequests = 8192;

// Byte offsets inside a tile of codes: token t in [0, 32), channel c.
__host__ __device__ inline int tile_k_code(int t, int c) {
  const int ks = c >> 4, cc = c & 15;
  const int lane = (t & 7) * 4 + ((cc & 7) >> 1);
  return ((t >> 3) * 2 + (ks >> 2)) * 512 + lane * 16 + (ks & 3) * 4 + (cc >> 3) * 2 + (cc & 1);
}
__host__ __device__ inline int tile_v_code(int t, int c) {
  const int s = t >> 4, tt = t & 15, n = c >> 3;
  const int lane = (c & 7) * 4 + ((tt & 7) >> 1);
  return 4096 + (n >> 1) * 512 + lane * 16 + ((n & 1) * 2 + s) * 4 + (tt >> 3) * 2 + (tt & 1);
}
// Element (16-bit) offsets inside a tail tile: token t in [0, 16), channel c.
__host__ __device__ inline int tile_k_tail(int t, int c) {
  const int ks = c >> 4, cc = c & 15;
  const int lane = (t & 7) * 4 + ((cc & 7) >> 1);
  return ((t >> 3) * 4 + (ks >> 1)) * 256 + lane * 8 + ((ks & 1) * 2 + (cc >> 3)) * 2 + (cc & 1);
}
__host__ __device__ inline int tile_v_tail(int t, int c) {
  const int n = c >> 3;
  const int lane = (c & 7) * 4 + ((t & 7) >> 1);
  return 2048 + (n >> 1) * 256 + lane * 8 + ((n & 1) * 2 + (t >> 3)) * 2 + (t & 1);
}

struct PagedGeometry {
  int L, H, r, n_blocks, bt, R, max_blocks, max_new, fmt, dtype;
  int64_t codes_layer, scales_layer, tails_layer;  // bytes of one layer
  int64_t codes_head, tails_head;                  // bytes of one (block, head) and one (request, head)
  int64_t max_units;
};

// Validates a configuration and derives its geometry (host code, no CUDA calls).
inline kvq_status make_paged_geometry(const kvq_paged_config* c, PagedGeometry* g) {
  if (!c || !g) return KVQ_ERR_INVALID_ARG;
  if (c->n_layers < 1 || c->n_kv_heads < 1 || c->gqa_ratio < 1 || c->d_head < 1 || c->n_blocks < 1 ||
      c->block_tokens < 1 || c->n_requests < 1 || c->max_blocks < 1 || c->max_new < 1)
    return KVQ_ERR_INVALID_ARG;
  if (c->format != KVQ_PAGED_INT8 && c->format != KVQ_PAGED_E4M3) return KVQ_ERR_INVALID_ARG;
  if (c->dtype != KVQ_F16 && c->dtype != KVQ_BF16) return KVQ_ERR_INVALID_ARG;
  if (c->d_head != kPagedDim || c->gqa_ratio > 8 || c->n_kv_heads > 255 || c->n_requests > kPagedMaxRequests)
    return KVQ_ERR_UNSUPPORTED;
  if (c->block_tokens != 32 && c->block_tokens != 64 && c->block_tokens != 128) return KVQ_ERR_UNSUPPORTED;
  const int64_t lim = (int64_t(1) << 31) - (1 << 16), bt = c->block_tokens;
  if (c->n_blocks * bt >= lim || c->n_requests * bt >= lim || (int64_t(c->max_blocks) + 1) * bt >= lim ||
      c->max_new >= lim)
    return KVQ_ERR_UNSUPPORTED;
  // decode tiles of a layer are counted in 32 bits (each is 8 KB of memory per layer)
  if ((c->n_blocks * bt / kTileCodeTokens + c->n_requests * bt / kTileTailTokens) * c->n_kv_heads >= lim)
    return KVQ_ERR_UNSUPPORTED;
  if (int64_t(c->n_requests) * (int64_t(c->max_blocks) + 1) >= (int64_t(1) << 40) / (c->n_kv_heads * (bt / 16)))
    return KVQ_ERR_UNSUPPORTED;
  PagedGeometry x;
  x.L = c->n_layers;
  x.H = c->n_kv_heads;
  x.r = c->gqa_ratio;
  x.n_blocks = c->n_blocks;
  x.bt = c->block_tokens;
  x.R = c->n_requests;
  x.max_blocks = c->max_blocks;
  x.max_new = c->max_new;
  x.fmt = c->format;
  x.dtype = c->dtype;
  x.codes_head = bt / kTileCodeTokens * kTileBytes;
  x.tails_head = bt / kTileTailTokens * kTileBytes;
  x.codes_layer = (int64_t)x.n_blocks * x.H * x.codes_head;
  x.scales_layer = (int64_t)x.n_blocks * x.H * 8;
  x.tails_layer = (int64_t)x.R * x.H * x.tails_head;
  x.max_units = x.max_new / bt + x.R;
  // the byte counts of all layers stay within 63 bits
  if (x.L > (int64_t(1) << 62) / (x.codes_layer + x.tails_layer)) return KVQ_ERR_UNSUPPORTED;
  *g = x;
  return KVQ_OK;
}

struct TablesParams {
  int32_t* lens;
  int32_t* block_table;
  int32_t* free_list;
  int32_t* free_count;
  const int32_t* new_tokens;
  kvq_paged_step out;
  int R, bt, max_blocks, n_blocks, max_new, commit;
};

struct PagedAppendParams {
  uint8_t* codes;  // of the layer
  float* scales;
  uint16_t* tails;
  const int32_t* block_table;
  const int32_t* lens;
  const int32_t* q_start;
  const int4* units;
  uint32_t* status;
  const uint16_t* k;
  const uint16_t* v;
  int64_t k_stride, v_stride, n_rows;
  int64_t codes_head, tails_head;  // bytes
  int H, R, bt, max_blocks, n_blocks;
};

struct PagedDequantParams {
  const uint8_t* codes;
  const float* scales;
  const uint16_t* tails;
  const int32_t* slots;
  float* k_out;
  float* v_out;
  int64_t n;
  int64_t codes_head, tails_head;
  int H, R, bt, n_blocks;
};

struct PagedDecodeParams {
  const uint8_t* codes;
  const float* scales;
  const uint8_t* tails;
  const int32_t* block_table;
  const int32_t* lens;
  const int32_t* q_start;
  const int32_t* tile_start;
  uint32_t* status;
  const uint16_t* q;
  int64_t q_stride;
  uint16_t* out;
  int zero_rest;      // rows without new tokens become zeros
  int early;          // the tables are read before the wait for the previous kernel
  float scale_log2;  // softmax_scale * log2(e)
  int64_t codes_head, tails_head;
  int H, r, R, bt, max_blocks, n_blocks;
  uint32_t* err;      // workspace
  uint32_t* tickets;
  float* parts;
  uint64_t wait_ns;
};

cudaError_t launch_paged_tables(const TablesParams& p, cudaStream_t stream);
cudaError_t launch_paged_append(const PagedAppendParams& p, int64_t max_units, int fmt, int dtype, cudaStream_t stream);
cudaError_t launch_paged_dequant(const PagedDequantParams& p, int fmt, int dtype, cudaStream_t stream);
cudaError_t launch_paged_decode(const PagedDecodeParams& p, int fmt, int dtype, cudaStream_t stream);

// Workspace of the decode attention: error word at 0, tickets [R * H] at 256, then partial
// results.
constexpr size_t kPagedTickets = 256;
inline size_t paged_workspace_parts(const PagedGeometry& g) {
  return kPagedTickets + ((size_t)g.R * g.H * 4 + 255) / 256 * 256;
}
size_t paged_workspace_bytes(const PagedGeometry& g);

}  // namespace kvq
