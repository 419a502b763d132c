// kvq_paged_api.cu — C ABI of the paged 8-bit cache and of the prompt attention: argument
// checks and launch descriptions. Host code only; a failed check launches nothing.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "kvq_kernels.h"
#include "kvq_paged.cuh"
#include "kvq_prompt.h"

using kvq::PagedGeometry;

namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - (1 << 16);

bool aligned(const void* p, uintptr_t a) { return p && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool bufs_ok(const kvq_paged_buffers* b) {
  return b && aligned(b->codes, 256) && aligned(b->scales, 256) && aligned(b->tails, 256);
}

bool step_ok(const kvq_paged_step* s) {
  return s && aligned(s->lens, 4) && aligned(s->free_count, 4) && aligned(s->q_start, 4) && aligned(s->positions, 4) &&
         aligned(s->slots, 4) && aligned(s->units, 16) && aligned(s->tile_start, 4) && aligned(s->status, 4);
}

bool stride_ok(int64_t stride) { return stride >= 0 && stride < (int64_t(1) << 31) && stride % 8 == 0; }

constexpr float kLog2E = 1.4426950408889634f;

bool scale_ok(float x) {  // the kernels take x * log2(e)
  const float y = x * kLog2E;
  return y - y == 0.0f;
}

kvq_status of(cudaError_t e) { return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA; }

}  // namespace

extern "C" {

kvq_status kvq_paged_buffer_sizes(const kvq_paged_config* cfg, size_t bytes[KVQ_PAGED_NUM_BUFFERS]) {
  if (!bytes) return KVQ_ERR_INVALID_ARG;
  PagedGeometry g;
  const kvq_status st = kvq::make_paged_geometry(cfg, &g);
  if (st != KVQ_OK) return st;
  bytes[KVQ_PAGED_BUF_CODES] = (size_t)(g.L * g.codes_layer);
  bytes[KVQ_PAGED_BUF_SCALES] = (size_t)(g.L * g.scales_layer);
  bytes[KVQ_PAGED_BUF_TAILS] = (size_t)(g.L * g.tails_layer);
  return KVQ_OK;
}

kvq_status kvq_paged_step_tables(const kvq_paged_config* cfg, const kvq_paged_state* state, const int32_t* new_tokens,
                                 const kvq_paged_step* step, int32_t commit, void* stream) {
  PagedGeometry g;
  const kvq_status st = kvq::make_paged_geometry(cfg, &g);
  if (st != KVQ_OK) return st;
  if (!state || !aligned(state->lens, 4) || !aligned(state->block_table, 4) || !aligned(state->free_list, 4) ||
      !aligned(state->free_count, 4) || !aligned(new_tokens, 4) || !step_ok(step))
    return KVQ_ERR_INVALID_ARG;
  // the state is read while the step is written
  if (step->lens == state->lens || step->free_count == state->free_count || new_tokens == step->lens ||
      new_tokens == state->lens || (commit != 0 && commit != 1))
    return KVQ_ERR_INVALID_ARG;
  kvq::TablesParams p;
  p.lens = state->lens;
  p.block_table = state->block_table;
  p.free_list = state->free_list;
  p.free_count = state->free_count;
  p.new_tokens = new_tokens;
  p.out = *step;
  p.R = g.R;
  p.bt = g.bt;
  p.max_blocks = g.max_blocks;
  p.n_blocks = g.n_blocks;
  p.max_new = g.max_new;
  p.commit = commit;
  return of(kvq::launch_paged_tables(p, static_cast<cudaStream_t>(stream)));
}

kvq_status kvq_paged_append(const kvq_paged_config* cfg, const kvq_paged_buffers* bufs, const int32_t* block_table,
                            const kvq_paged_step* step, int32_t layer, int64_t n_rows, const void* k, int64_t k_stride,
                            const void* v, int64_t v_stride, void* stream) {
  PagedGeometry g;
  const kvq_status st = kvq::make_paged_geometry(cfg, &g);
  if (st != KVQ_OK) return st;
  if (!bufs_ok(bufs) || !aligned(block_table, 4) || !step_ok(step)) return KVQ_ERR_INVALID_ARG;
  if (layer < 0 || layer >= g.L || n_rows < 0 || n_rows >= kMaxRows) return KVQ_ERR_INVALID_ARG;
  if (n_rows > 0 && (!aligned(k, 16) || !aligned(v, 16))) return KVQ_ERR_INVALID_ARG;
  if (!stride_ok(k_stride) || !stride_ok(v_stride)) return KVQ_ERR_INVALID_ARG;
  kvq::PagedAppendParams p;
  p.codes = static_cast<uint8_t*>(bufs->codes) + layer * g.codes_layer;
  p.scales = bufs->scales + layer * (g.scales_layer / 4);
  p.tails = static_cast<uint16_t*>(bufs->tails) + layer * (g.tails_layer / 2);
  p.block_table = block_table;
  p.lens = step->lens;
  p.q_start = step->q_start;
  p.units = reinterpret_cast<const int4*>(step->units);
  p.status = step->status;
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.n_rows = n_rows;
  p.codes_head = g.codes_head;
  p.tails_head = g.tails_head;
  p.H = g.H;
  p.R = g.R;
  p.bt = g.bt;
  p.max_blocks = g.max_blocks;
  p.n_blocks = g.n_blocks;
  // every request with new tokens has one unit, or one per block that it finishes
  const int64_t rows = std::min<int64_t>(n_rows, g.max_new);
  const int64_t units = std::max<int64_t>(1, std::min<int64_t>(g.max_units, rows / g.bt + std::min<int64_t>(rows, g.R)));
  return of(kvq::launch_paged_append(p, units, g.fmt, g.dtype, static_cast<cudaStream_t>(stream)));
}

kvq_status kvq_paged_dequantize(const kvq_paged_config* cfg, const kvq_paged_buffers* bufs, int32_t layer, int64_t n,
                                const int32_t* slots, float* k_out, float* v_out, void* stream) {
  PagedGeometry g;
  const kvq_status st = kvq::make_paged_geometry(cfg, &g);
  if (st != KVQ_OK) return st;
  if (!bufs_ok(bufs) || layer < 0 || layer >= g.L || n < 0 || n >= kMaxRows) return KVQ_ERR_INVALID_ARG;
  if (n == 0) return KVQ_OK;
  if (!aligned(slots, 4) || !aligned(k_out, 16) || !aligned(v_out, 16)) return KVQ_ERR_INVALID_ARG;
  kvq::PagedDequantParams p;
  p.codes = static_cast<const uint8_t*>(bufs->codes) + layer * g.codes_layer;
  p.scales = bufs->scales + layer * (g.scales_layer / 4);
  p.tails = static_cast<const uint16_t*>(bufs->tails) + layer * (g.tails_layer / 2);
  p.slots = slots;
  p.k_out = k_out;
  p.v_out = v_out;
  p.n = n;
  p.codes_head = g.codes_head;
  p.tails_head = g.tails_head;
  p.H = g.H;
  p.R = g.R;
  p.bt = g.bt;
  p.n_blocks = g.n_blocks;
  return of(kvq::launch_paged_dequant(p, g.fmt, g.dtype, static_cast<cudaStream_t>(stream)));
}

size_t kvq_paged_workspace_size(const kvq_paged_config* cfg) {
  PagedGeometry g;
  return kvq::make_paged_geometry(cfg, &g) == KVQ_OK ? kvq::paged_workspace_bytes(g) : 0;
}

kvq_status kvq_paged_decode_attention(const kvq_paged_config* cfg, const kvq_paged_buffers* bufs,
                                      const int32_t* block_table, const kvq_paged_step* step, int32_t layer,
                                      const void* q, int64_t q_stride, float softmax_scale, void* out,
                                      uint32_t flags, void* ws, size_t ws_bytes, void* stream) {
  PagedGeometry g;
  const kvq_status st = kvq::make_paged_geometry(cfg, &g);
  if (st != KVQ_OK) return st;
  if (!bufs_ok(bufs) || !aligned(block_table, 4) || !step_ok(step)) return KVQ_ERR_INVALID_ARG;
  if (layer < 0 || layer >= g.L || !aligned(q, 16) || !aligned(out, 16)) return KVQ_ERR_INVALID_ARG;
  if (!stride_ok(q_stride) || !scale_ok(softmax_scale)) return KVQ_ERR_INVALID_ARG;
  if (flags & ~(KVQ_PAGED_ZERO_REST | KVQ_PAGED_EARLY_TABLES | KVQ_PAGED_ZERO_WAIT_LIMIT)) return KVQ_ERR_INVALID_ARG;
  if (!aligned(ws, 256) || ws_bytes < kvq::paged_workspace_bytes(g)) return KVQ_ERR_WORKSPACE;
  kvq::PagedDecodeParams p;
  p.codes = static_cast<const uint8_t*>(bufs->codes) + layer * g.codes_layer;
  p.scales = bufs->scales + layer * (g.scales_layer / 4);
  p.tails = static_cast<const uint8_t*>(bufs->tails) + layer * g.tails_layer;
  p.block_table = block_table;
  p.lens = step->lens;
  p.q_start = step->q_start;
  p.tile_start = step->tile_start;
  p.status = step->status;
  p.q = static_cast<const uint16_t*>(q);
  p.q_stride = q_stride;
  p.out = static_cast<uint16_t*>(out);
  p.zero_rest = (flags & KVQ_PAGED_ZERO_REST) != 0;
  p.early = (flags & KVQ_PAGED_EARLY_TABLES) != 0;
  p.scale_log2 = softmax_scale * kLog2E;
  p.codes_head = g.codes_head;
  p.tails_head = g.tails_head;
  p.H = g.H;
  p.r = g.r;
  p.R = g.R;
  p.bt = g.bt;
  p.max_blocks = g.max_blocks;
  p.n_blocks = g.n_blocks;
  p.err = static_cast<uint32_t*>(ws);
  p.tickets = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + kvq::kPagedTickets);
  p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kvq::paged_workspace_parts(g));
  p.wait_ns = (flags & KVQ_PAGED_ZERO_WAIT_LIMIT) ? 0 : kvq::kDefaultWaitNs;
  return of(kvq::launch_paged_decode(p, g.fmt, g.dtype, static_cast<cudaStream_t>(stream)));
}

size_t kvq_prompt_workspace_size(void) { return kvq::prompt_workspace_bytes(); }

kvq_status kvq_prompt_attention(const kvq_prompt_args* a, void* ws, size_t ws_bytes, void* stream) {
  if (!a) return KVQ_ERR_INVALID_ARG;
  if (a->n_kv_heads < 1 || a->gqa_ratio < 1 || a->n_seqs < 1 || a->n_q < 0 || a->n_kv < 0) return KVQ_ERR_INVALID_ARG;
  if ((a->dtype != KVQ_F16 && a->dtype != KVQ_BF16) || (a->causal != 0 && a->causal != 1)) return KVQ_ERR_INVALID_ARG;
  if (a->flags & ~(KVQ_PROMPT_ZERO_REST | KVQ_PROMPT_ZERO_WAIT_LIMIT)) return KVQ_ERR_INVALID_ARG;
  if (a->d_head != 128 || a->gqa_ratio > 8 || a->n_kv_heads > 255 || a->n_seqs > 65535 || a->n_q >= kMaxRows ||
      a->n_kv >= kMaxRows)
    return KVQ_ERR_UNSUPPORTED;
  if (!scale_ok(a->softmax_scale) || a->softmax_scale < 0.0f) return KVQ_ERR_INVALID_ARG;
  if (!aligned(a->q_start, 4) || !aligned(a->kv_start, 4)) return KVQ_ERR_INVALID_ARG;
  if (!stride_ok(a->q_stride) || !stride_ok(a->k_stride) || !stride_ok(a->v_stride) || !stride_ok(a->out_stride))
    return KVQ_ERR_INVALID_ARG;
  const int64_t nq = (int64_t)a->n_kv_heads * a->gqa_ratio;
  if (a->n_q > 1 && (a->q_stride < nq * 128 || a->out_stride < nq * 128)) return KVQ_ERR_INVALID_ARG;  // rows overlap
  if (a->n_kv > 1 && (a->k_stride < a->n_kv_heads * 128 || a->v_stride < a->n_kv_heads * 128)) return KVQ_ERR_INVALID_ARG;
  if (a->n_q > 0 && (!aligned(a->q, 16) || !aligned(a->out, 16))) return KVQ_ERR_INVALID_ARG;
  if (a->n_q > 0 && (a->out == a->q || (a->n_kv > 0 && (a->out == a->k || a->out == a->v)))) return KVQ_ERR_INVALID_ARG;
  if (a->n_kv > 0 && (!aligned(a->k, 16) || !aligned(a->v, 16))) return KVQ_ERR_INVALID_ARG;
  if (a->lse && !aligned(a->lse, 4)) return KVQ_ERR_INVALID_ARG;
  if (!aligned(ws, 256) || ws_bytes < kvq::prompt_workspace_bytes()) return KVQ_ERR_WORKSPACE;
  if (a->n_q == 0) return KVQ_OK;
  kvq::PromptParams p;
  p.q = static_cast<const uint16_t*>(a->q);
  p.k = static_cast<const uint16_t*>(a->k);
  p.v = static_cast<const uint16_t*>(a->v);
  p.out = static_cast<uint16_t*>(a->out);
  p.lse = a->lse;
  p.q_start = a->q_start;
  p.kv_start = a->kv_start;
  p.q_stride = a->q_stride;
  p.k_stride = a->k_stride;
  p.v_stride = a->v_stride;
  p.out_stride = a->out_stride;
  p.n_q = (int32_t)a->n_q;
  p.n_kv = (int32_t)a->n_kv;
  p.n_seqs = a->n_seqs;
  p.H = a->n_kv_heads;
  p.r = a->gqa_ratio;
  p.causal = a->causal;
  p.zero_rest = (a->flags & KVQ_PROMPT_ZERO_REST) != 0;
  p.scale_log2 = a->softmax_scale * kLog2E;
  p.err = static_cast<uint32_t*>(ws);
  p.tickets = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + kvq::kPromptTickets);
  p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kvq::kPromptParts);
  p.wait_ns = (a->flags & KVQ_PROMPT_ZERO_WAIT_LIMIT) ? 0 : kvq::kDefaultWaitNs;
  return of(kvq::launch_prompt(p, a->dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
