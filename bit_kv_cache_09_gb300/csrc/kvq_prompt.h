// kvq_prompt.h — launch description of the prompt attention (library-internal).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/kvq.h"

namespace kvq {

struct PromptParams {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  float* lse;
  const int32_t *q_start, *kv_start;
  int64_t q_stride, k_stride, v_stride, out_stride;  // elements
  int32_t n_q, n_kv, n_seqs, H, r, causal, zero_rest;
  float scale_log2;  // softmax_scale * log2(e)
  uint32_t* tickets; // workspace: [kPromptSplit], zero between calls
  float* parts;
  uint32_t* err;
  uint64_t wait_ns;
};

// Workspace: error word at 0, tickets at 256, parts of split items behind them.
constexpr int kPromptSplit = 152;  // CTAs of a launch that may split (the card's SMs)
constexpr size_t kPromptTickets = 256, kPromptParts = 1024;
size_t prompt_workspace_bytes();
cudaError_t launch_prompt(const PromptParams& p, int dtype, cudaStream_t stream);

}  // namespace kvq
