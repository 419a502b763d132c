// kvq_paged_quant.cu — append to and read back from the paged 8-bit cache.
//
// Append: one CTA per (work unit of the step, kv head). A unit is a block that the step
// finishes; the first unit of a request also replaces the request's tail rows once it has
// read them (a request that finishes no block has one unit that only copies). The CTA
// holds the block's 16-bit rows in registers, takes max|x| of keys and of values over all
// of them, divides, rounds and writes the codes in tile order through shared memory: each
// row is read once and each code written once.
//
// Quotients are binary32, rounded to nearest (this file is compiled with -fmad=false).
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "kvq_kernels.h"
#include "kvq_paged.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 256;
constexpr int kRowThreads = 16;                      // threads of a row, 8 channels each
constexpr int kRowsPass = kThreads / kRowThreads;    // rows of a pass
constexpr int kCodeStride = kPagedDim + 8;           // bytes of a staged row of codes

template <bool BF16>
__device__ __forceinline__ float2 to_float2(uint32_t w) {
  if (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Largest magnitude of the CTA's entries, from the largest bit pattern without the sign
// (infinities and NaN order above every number).
template <bool BF16>
__device__ __forceinline__ float scale_of(uint32_t abs_bits, float top) {
  const uint32_t inf = BF16 ? 0x7f80u : 0x7c00u;
  if (abs_bits >= inf) return __int_as_float(0x7fffffff);
  const float amax = to_float2<BF16>(abs_bits).x;
  return amax == 0.0f ? 1.0f : fmaxf(__fdiv_rn(amax, top), 1.17549435e-38f);
}

template <int FMT>
__device__ __forceinline__ uint32_t code_of(float x, float scale) {
  const float y = __fdiv_rn(x, scale);
  if (FMT == KVQ_PAGED_INT8) return (uint32_t)(max(-127, min(127, __float2int_rn(y))) + 128);
  return (uint32_t)__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
}

template <int BT, int FMT, bool BF16>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const PagedAppendParams p) {
  constexpr int PASSES = BT / kRowsPass;
  __shared__ __align__(16) uint8_t codes_s[2][BT * kCodeStride];
  __shared__ uint32_t amax_s[2][kThreads / 32];
  pdl_wait();
  pdl_allow_dependents();
  const int unit = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  if (unit == 0 && h == 0 && tid == 0 && p.q_start[p.R] > p.n_rows) atomicOr(&p.status[0], KVQ_PAGED_ERR_ROWS);
  if (unit >= (int)p.status[1]) return;
  const int2 u = p.units[unit];
  const int row = u.x, block = u.y;
  if (row < 0 || row >= p.R) return;
  const int q0 = p.q_start[row], n_new = p.q_start[row + 1] - q0;
  const int after = p.lens[row], before = after - n_new;
  const int full0 = before / BT, full1 = after / BT;
  uint16_t* tail = p.tails + ((int64_t)row * p.H + h) * (p.tails_head / 2);
  const int rt = tid / kRowThreads, c0 = (tid % kRowThreads) * 8;
  const int64_t head_off = (int64_t)h * kPagedDim + c0;

  if (block >= 0) {
    const int id = block < p.max_blocks ? p.block_table[(int64_t)row * p.max_blocks + block] : -1;
    uint4 kx[PASSES], vx[PASSES];
    uint32_t ka = 0u, va = 0u;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int t = i * kRowsPass + rt, pos = block * BT + t;
      kx[i] = vx[i] = make_uint4(0u, 0u, 0u, 0u);
      if (pos >= before) {
        const int64_t r = (int64_t)q0 + (pos - before);
        if (r < p.n_rows) {
          kx[i] = *reinterpret_cast<const uint4*>(p.k + r * p.k_stride + head_off);
          vx[i] = *reinterpret_cast<const uint4*>(p.v + r * p.v_stride + head_off);
        }
      } else {  // kept in the tail since an earlier step
        const uint16_t* tt = tail + (t / kTileTailTokens) * (kTileBytes / 2);
        uint32_t* kw = reinterpret_cast<uint32_t*>(&kx[i]);
        uint32_t* vw = reinterpret_cast<uint32_t*>(&vx[i]);
#pragma unroll
        for (int c = 0; c < 8; c += 2) {
          kw[c / 2] = *reinterpret_cast<const uint32_t*>(tt + tile_k_tail(t % kTileTailTokens, c0 + c));
          vw[c / 2] = (uint32_t)tt[tile_v_tail(t % kTileTailTokens, c0 + c)] |
                      ((uint32_t)tt[tile_v_tail(t % kTileTailTokens, c0 + c + 1)] << 16);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const uint32_t* kw = reinterpret_cast<const uint32_t*>(&kx[i]);
      const uint32_t* vw = reinterpret_cast<const uint32_t*>(&vx[i]);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        ka = __vmaxu2(ka, kw[w] & 0x7fff7fffu);
        va = __vmaxu2(va, vw[w] & 0x7fff7fffu);
      }
    }
    ka = max(ka & 0xffffu, ka >> 16);
    va = max(va & 0xffffu, va >> 16);
    ka = __reduce_max_sync(0xffffffffu, ka);
    va = __reduce_max_sync(0xffffffffu, va);
    if ((tid & 31) == 0) {
      amax_s[0][tid / 32] = ka;
      amax_s[1][tid / 32] = va;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      ka = max(ka, amax_s[0][w]);
      va = max(va, amax_s[1][w]);
    }
    const float top = FMT == KVQ_PAGED_INT8 ? 127.0f : 448.0f;
    const float ks = scale_of<BF16>(ka, top), vs = scale_of<BF16>(va, top);
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int t = i * kRowsPass + rt;
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(a ? &vx[i] : &kx[i]);
        const float s = a ? vs : ks;
        uint32_t o[2] = {0u, 0u};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float2 f = to_float2<BF16>(w[c]);
          o[c / 2] |= (code_of<FMT>(f.x, s) | (code_of<FMT>(f.y, s) << 8)) << (16 * (c & 1));
        }
        *reinterpret_cast<uint2*>(&codes_s[a][t * kCodeStride + c0]) = make_uint2(o[0], o[1]);
      }
    }
    __syncthreads();
    if (id >= 0 && id < p.n_blocks) {
      uint8_t* out = p.codes + ((int64_t)id * p.H + h) * p.codes_head;
      for (int i = tid; i < BT * 16; i += kThreads) {  // 16-byte pieces: 256 of keys, 256 of values per tile
        const int tile = i >> 9, a = (i >> 8) & 1, chunk = (i >> 5) & 7, g = (i >> 2) & 7, l = i & 3;
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (a == 0) {  // words of four k16 steps of token 8 (chunk / 2) + g
            const uint8_t* src = &codes_s[0][(tile * 32 + (chunk >> 1) * 8 + g) * kCodeStride + (chunk & 1) * 64 + k * 16 + l * 2];
            w[k] = *reinterpret_cast<const uint16_t*>(src) | ((uint32_t)*reinterpret_cast<const uint16_t*>(src + 8) << 16);
          } else {  // channel 16 chunk + 8 (k / 2) + g of four tokens
            const uint8_t* src = &codes_s[1][(tile * 32 + (k & 1) * 16 + l * 2) * kCodeStride + chunk * 16 + (k >> 1) * 8 + g];
            w[k] = src[0] | ((uint32_t)src[kCodeStride] << 8) | ((uint32_t)src[8 * kCodeStride] << 16) |
                   ((uint32_t)src[9 * kCodeStride] << 24);
          }
        }
        *reinterpret_cast<uint4*>(out + (int64_t)i * 16) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if (tid == 0) {
        float* sc = p.scales + ((int64_t)id * p.H + h) * 2;
        sc[0] = ks;
        sc[1] = vs;
      }
    } else if (tid == 0) {
      atomicOr(&p.status[0], KVQ_PAGED_ERR_TABLE);
    }
  }
  if (block < 0 || block == full0) {  // the request's first unit keeps the rows of the unfinished block
    const int first = max(before, full1 * BT);
    for (int pos = first + rt; pos < after; pos += kRowsPass) {
      const int64_t r = (int64_t)q0 + (pos - before);
      if (r >= p.n_rows) continue;
      const uint4 kr = *reinterpret_cast<const uint4*>(p.k + r * p.k_stride + head_off);
      const uint4 vr = *reinterpret_cast<const uint4*>(p.v + r * p.v_stride + head_off);
      const int t = pos - full1 * BT;
      uint16_t* tt = tail + (t / kTileTailTokens) * (kTileBytes / 2);
      const uint32_t* kw = reinterpret_cast<const uint32_t*>(&kr);
      const uint32_t* vw = reinterpret_cast<const uint32_t*>(&vr);
#pragma unroll
      for (int c = 0; c < 8; c += 2) {
        *reinterpret_cast<uint32_t*>(tt + tile_k_tail(t % kTileTailTokens, c0 + c)) = kw[c / 2];
        tt[tile_v_tail(t % kTileTailTokens, c0 + c)] = (uint16_t)vw[c / 2];
        tt[tile_v_tail(t % kTileTailTokens, c0 + c + 1)] = (uint16_t)(vw[c / 2] >> 16);
      }
    }
  }
}

// Read back: 32 threads per (slot, kv head), 4 channels of the key and of the value each.
template <int FMT, bool BF16>
__global__ void __launch_bounds__(kThreads) paged_dequant_kernel(const PagedDequantParams p) {
  pdl_wait();
  pdl_allow_dependents();
  const int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  if (i >= p.n * p.H) return;
  const int64_t s_i = i / p.H;
  const int h = (int)(i - s_i * p.H), c0 = (threadIdx.x & 31) * 4;
  const int64_t slot = p.slots[s_i];
  float k[4], v[4];
  const float nan = __int_as_float(0x7fffffff);
  if (slot >= 0 && slot < (int64_t)p.n_blocks * p.bt) {
    const int64_t id = slot / p.bt;
    const int t = (int)(slot - id * p.bt);
    const uint8_t* tile = p.codes + (id * p.H + h) * p.codes_head + (t / kTileCodeTokens) * kTileBytes;
    const float2 sc = *reinterpret_cast<const float2*>(p.scales + (id * p.H + h) * 2);
    for (int c = 0; c < 4; ++c) {
      const uint8_t a = tile[tile_k_code(t % kTileCodeTokens, c0 + c)], b = tile[tile_v_code(t % kTileCodeTokens, c0 + c)];
      float fa, fb;
      if (FMT == KVQ_PAGED_INT8) {
        fa = (float)((int)a - 128);
        fb = (float)((int)b - 128);
      } else {
        fa = __half2float(__half(__nv_cvt_fp8_to_halfraw(a, __NV_E4M3)));
        fb = __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
      }
      k[c] = __fmul_rn(fa, sc.x);
      v[c] = __fmul_rn(fb, sc.y);
    }
  } else if (slot < 0 && -1 - slot < (int64_t)p.R * p.bt) {
    const int64_t at = -1 - slot, row = at / p.bt;
    const int t = (int)(at - row * p.bt);
    const uint16_t* tile = p.tails + (row * p.H + h) * (p.tails_head / 2) + (t / kTileTailTokens) * (kTileBytes / 2);
    for (int c = 0; c < 4; ++c) {
      k[c] = to_float2<BF16>(tile[tile_k_tail(t % kTileTailTokens, c0 + c)]).x;
      v[c] = to_float2<BF16>(tile[tile_v_tail(t % kTileTailTokens, c0 + c)]).x;
    }
  } else {
    for (int c = 0; c < 4; ++c) k[c] = v[c] = nan;
  }
  *reinterpret_cast<float4*>(p.k_out + i * kPagedDim + c0) = make_float4(k[0], k[1], k[2], k[3]);
  *reinterpret_cast<float4*>(p.v_out + i * kPagedDim + c0) = make_float4(v[0], v[1], v[2], v[3]);
}

template <int FMT, bool BF16>
cudaError_t append_bt(const PagedAppendParams& p, dim3 grid, cudaStream_t stream) {
  switch (p.bt) {
    case 32: return launch_pdl(paged_append_kernel<32, FMT, BF16>, grid, dim3(kThreads), 0, stream, p);
    case 64: return launch_pdl(paged_append_kernel<64, FMT, BF16>, grid, dim3(kThreads), 0, stream, p);
    default: return launch_pdl(paged_append_kernel<128, FMT, BF16>, grid, dim3(kThreads), 0, stream, p);
  }
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendParams& p, int64_t max_units, int fmt, int dtype, cudaStream_t stream) {
  const dim3 grid((unsigned)max_units, (unsigned)p.H);
  if (fmt == KVQ_PAGED_INT8)
    return dtype == KVQ_BF16 ? append_bt<KVQ_PAGED_INT8, true>(p, grid, stream) : append_bt<KVQ_PAGED_INT8, false>(p, grid, stream);
  return dtype == KVQ_BF16 ? append_bt<KVQ_PAGED_E4M3, true>(p, grid, stream) : append_bt<KVQ_PAGED_E4M3, false>(p, grid, stream);
}

cudaError_t launch_paged_dequant(const PagedDequantParams& p, int fmt, int dtype, cudaStream_t stream) {
  const int64_t ctas = (p.n * p.H + kThreads / 32 - 1) / (kThreads / 32);
  const dim3 grid((unsigned)ctas), block(kThreads);
  if (fmt == KVQ_PAGED_INT8)
    return dtype == KVQ_BF16 ? launch_pdl(paged_dequant_kernel<KVQ_PAGED_INT8, true>, grid, block, 0, stream, p)
                             : launch_pdl(paged_dequant_kernel<KVQ_PAGED_INT8, false>, grid, block, 0, stream, p);
  return dtype == KVQ_BF16 ? launch_pdl(paged_dequant_kernel<KVQ_PAGED_E4M3, true>, grid, block, 0, stream, p)
                           : launch_pdl(paged_dequant_kernel<KVQ_PAGED_E4M3, false>, grid, block, 0, stream, p);
}

}  // namespace kvq
