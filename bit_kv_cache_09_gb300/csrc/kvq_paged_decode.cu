// kvq_paged_decode.cu — decode attention over the paged 8-bit cache.
//
// One CTA per (request, kv head); its warps take tokens in turn, a lane holds 4 channels
// of the key and value and of the accumulators of all query heads of the kv head, with a
// running maximum and sum per warp that are joined at the end.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "kvq_kernels.h"
#include "kvq_paged.cuh"

namespace kvq {
namespace {

constexpr int kWarps = 8;

template <bool BF16>
__device__ __forceinline__ float to_float(uint16_t x) {
  if (BF16) return __uint_as_float((uint32_t)x << 16);
  return __half2float(__ushort_as_half(x));
}

template <int FMT, bool BF16>
__global__ void __launch_bounds__(kWarps * 32) paged_decode_kernel(const PagedDecodeParams p) {
  __shared__ float m_s[kWarps][8], l_s[kWarps][8];
  __shared__ float o_s[kWarps][8][kPagedDim];
  pdl_wait();
  pdl_allow_dependents();
  const int row = blockIdx.x, h = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  if (p.q_start[row + 1] == p.q_start[row]) {
    uint32_t* o = reinterpret_cast<uint32_t*>(p.out + ((int64_t)row * p.H + h) * p.r * kPagedDim);
    for (int i = threadIdx.x; p.zero_rest && i < p.r * kPagedDim / 2; i += kWarps * 32) o[i] = 0u;
    return;
  }
  const int len = p.lens[row], full = len / p.bt * p.bt, c0 = lane * 4;
  float q[8][4], o[8][4], m[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.0f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      o[i][c] = 0.0f;
      q[i][c] = i < p.r ? to_float<BF16>(p.q[row * p.q_stride + (int64_t)(h * p.r + i) * kPagedDim + c0 + c]) : 0.0f;
    }
  }
  for (int t = warp; t < len; t += kWarps) {
    float k[4], v[4];
    if (t < full) {
      const int id = p.block_table[(int64_t)row * p.max_blocks + t / p.bt];
      if (id < 0 || id >= p.n_blocks) {
        if (lane == 0) atomicOr(&p.status[0], KVQ_PAGED_ERR_TABLE);
        continue;
      }
      const int off = t % p.bt;
      const uint8_t* tile = p.codes + ((int64_t)id * p.H + h) * p.codes_head + (off / kTileCodeTokens) * kTileBytes;
      const float2 sc = *reinterpret_cast<const float2*>(p.scales + ((int64_t)id * p.H + h) * 2);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint8_t a = tile[tile_k_code(off % 32, c0 + c)], b = tile[tile_v_code(off % 32, c0 + c)];
        if (FMT == KVQ_PAGED_INT8) {
          k[c] = sc.x * (float)((int)a - 128);
          v[c] = sc.y * (float)((int)b - 128);
        } else {
          k[c] = sc.x * __half2float(__half(__nv_cvt_fp8_to_halfraw(a, __NV_E4M3)));
          v[c] = sc.y * __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
        }
      }
    } else {
      const int off = t - full;
      const uint16_t* tile = reinterpret_cast<const uint16_t*>(p.tails + ((int64_t)row * p.H + h) * p.tails_head +
                                                               (off / kTileTailTokens) * kTileBytes);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        k[c] = to_float<BF16>(tile[tile_k_tail(off % 16, c0 + c)]);
        v[c] = to_float<BF16>(tile[tile_v_tail(off % 16, c0 + c)]);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= p.r) break;
      float s = q[i][0] * k[0] + q[i][1] * k[1] + q[i][2] * k[2] + q[i][3] * k[3];
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s *= p.scale_log2;
      const float mn = fmaxf(m[i], s), a = exp2f(m[i] - mn), e = exp2f(s - mn);
      m[i] = mn;
      l[i] = l[i] * a + e;
#pragma unroll
      for (int c = 0; c < 4; ++c) o[i][c] = o[i][c] * a + e * v[c];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (lane == 0) {
      m_s[warp][i] = m[i];
      l_s[warp][i] = l[i];
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) o_s[warp][i][c0 + c] = o[i][c];
  }
  __syncthreads();
  for (int x = threadIdx.x; x < p.r * kPagedDim; x += kWarps * 32) {
    const int i = x / kPagedDim, c = x % kPagedDim;
    float M = -INFINITY, L = 0.0f, O = 0.0f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, m_s[w][i]);
    for (int w = 0; w < kWarps; ++w) {
      const float e = m_s[w][i] == -INFINITY ? 0.0f : exp2f(m_s[w][i] - M);
      L += e * l_s[w][i];
      O += e * o_s[w][i][c];
    }
    const float y = O / L;
    p.out[((int64_t)row * p.H * p.r + h * p.r + i) * kPagedDim + c] =
        BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(y)) : __half_as_ushort(__float2half_rn(y));
  }
}

}  // namespace

size_t paged_workspace_bytes(const PagedGeometry& g) { return 256; }

cudaError_t launch_paged_decode(const PagedDecodeParams& p, int fmt, int dtype, cudaStream_t stream) {
  const dim3 grid(p.R, p.H), block(kWarps * 32);
  if (fmt == KVQ_PAGED_INT8)
    return dtype == KVQ_BF16 ? launch_pdl(paged_decode_kernel<KVQ_PAGED_INT8, true>, grid, block, 0, stream, p)
                             : launch_pdl(paged_decode_kernel<KVQ_PAGED_INT8, false>, grid, block, 0, stream, p);
  return dtype == KVQ_BF16 ? launch_pdl(paged_decode_kernel<KVQ_PAGED_E4M3, true>, grid, block, 0, stream, p)
                           : launch_pdl(paged_decode_kernel<KVQ_PAGED_E4M3, false>, grid, block, 0, stream, p);
}

}  // namespace kvq
