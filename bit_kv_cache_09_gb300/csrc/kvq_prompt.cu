// kvq_prompt.cu — attention of packed prompts.
//
// One warp per (query row, query head): lanes score 32 keys at a time, a running maximum
// and sum carries the softmax, and each lane accumulates 4 channels of the values.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "kvq_kernels.h"
#include "kvq_prompt.h"

namespace kvq {
namespace {

constexpr int kWarps = 8, kDim = 128;

template <bool BF16>
__device__ __forceinline__ float2 pair(uint32_t w) {
  if (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

template <bool BF16>
__global__ void __launch_bounds__(kWarps * 32) prompt_kernel(const PromptParams p) {
  __shared__ float q_s[kWarps][kDim];
  pdl_wait();
  pdl_allow_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, nq = p.H * p.r;
  const int64_t item = (int64_t)blockIdx.x * kWarps + warp;
  const int row = (int)(item / nq), head = (int)(item % nq), h = head / p.r;
  if (row >= p.n_q) return;
  int lo = 0, hi = p.n_seqs;  // last sequence that starts at or before the row
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (p.q_start[mid] <= row) lo = mid; else hi = mid;
  }
  const int q0 = max(p.q_start[lo], 0), q1 = min(p.q_start[lo + 1], p.n_q);
  if (row < q0 || row >= q1) {
    if (p.zero_rest) *reinterpret_cast<uint2*>(p.out + row * p.out_stride + head * kDim + lane * 4) = make_uint2(0u, 0u);
    if (p.zero_rest && p.lse && lane == 0) p.lse[(int64_t)row * nq + head] = -INFINITY;
    return;
  }
  const int k0 = min(max(p.kv_start[lo], 0), p.n_kv), k1 = min(max(p.kv_start[lo + 1], k0), p.n_kv);
  const int see = p.causal ? max(0, min(k1 - k0, row - q0 + 1 + (k1 - k0) - (q1 - q0))) : k1 - k0;
  for (int c = lane; c < kDim / 2; c += 32) {
    const float2 f = pair<BF16>(*reinterpret_cast<const uint32_t*>(p.q + row * p.q_stride + head * kDim + 2 * c));
    q_s[warp][2 * c] = f.x;
    q_s[warp][2 * c + 1] = f.y;
  }
  __syncwarp();
  float m = -INFINITY, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j0 = 0; j0 < see; j0 += 32) {
    const int j = j0 + lane;
    float s = -INFINITY;
    if (j < see) {
      const uint4* kr = reinterpret_cast<const uint4*>(p.k + (k0 + j) * p.k_stride + h * kDim);
      s = 0.0f;
      for (int c = 0; c < kDim / 8; ++c) {
        const uint4 x = kr[c];
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = pair<BF16>(w[i]);
          s = fmaf(f.x, q_s[warp][c * 8 + i * 2], s);
          s = fmaf(f.y, q_s[warp][c * 8 + i * 2 + 1], s);
        }
      }
      s *= p.scale_log2;
    }
    float mn = s;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, x));
    mn = fmaxf(m, mn);
    const float a = exp2f(m - mn), e = j < see ? exp2f(s - mn) : 0.0f;
    m = mn;
    float sum = e;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    l = l * a + sum;
    for (int c = 0; c < 4; ++c) o[c] *= a;
    const int n = min(32, see - j0);
    for (int t = 0; t < n; ++t) {
      const float w = __shfl_sync(0xffffffffu, e, t);
      const uint2 x = *reinterpret_cast<const uint2*>(p.v + (k0 + j0 + t) * p.v_stride + h * kDim + lane * 4);
      const float2 f0 = pair<BF16>(x.x), f1 = pair<BF16>(x.y);
      o[0] = fmaf(w, f0.x, o[0]);
      o[1] = fmaf(w, f0.y, o[1]);
      o[2] = fmaf(w, f1.x, o[2]);
      o[3] = fmaf(w, f1.y, o[3]);
    }
  }
  const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
  for (int c = 0; c < 4; ++c) {
    const float y = see > 0 ? o[c] * inv : 0.0f;
    p.out[row * p.out_stride + head * kDim + lane * 4 + c] =
        BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(y)) : __half_as_ushort(__float2half_rn(y));
  }
  if (p.lse && lane == 0)
    p.lse[(int64_t)row * nq + head] = see > 0 ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

cudaError_t launch_prompt(const PromptParams& p, int dtype, cudaStream_t stream) {
  const int64_t items = (int64_t)p.n_q * p.H * p.r;
  const dim3 grid((unsigned)((items + kWarps - 1) / kWarps));
  return dtype == KVQ_BF16 ? launch_pdl(prompt_kernel<true>, grid, dim3(kWarps * 32), 0, stream, p)
                           : launch_pdl(prompt_kernel<false>, grid, dim3(kWarps * 32), 0, stream, p);
}

}  // namespace kvq
