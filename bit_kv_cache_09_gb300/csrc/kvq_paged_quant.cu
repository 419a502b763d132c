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
//
// Both kernels are bound by HBM in principle: 768 bytes per token and head for the append, 1280 for the
// read back. Measured on GB300, 32.8 k tokens of 24 prompts, 8 heads: append 48 us (4.2 TB/s; 58 % of
// the issue slots are busy, about five instructions per two entries go into the exact quotient), read
// back 60 us (5.6 TB/s, four fifths of it writes).
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "kvq_kernels.h"
#include "kvq_paged.cuh"

namespace kvq {
namespace {

constexpr int kChunkStride = 528;  // bytes of a staged 512-byte chunk of a tile: shifts its banks by 4 words

template <bool BF16>
__device__ __forceinline__ float2 to_float2(uint32_t w) {
  if (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Scale of a block from its entries' largest bit pattern without the sign (infinities and NaN order
// above every number).
template <bool BF16>
__device__ __forceinline__ float scale_of(uint32_t abs_bits, float top) {
  const uint32_t inf = BF16 ? 0x7f80u : 0x7c00u;
  if (abs_bits >= inf) return __int_as_float(0x7fffffff);
  const float amax = to_float2<BF16>(abs_bits).x;
  return amax == 0.0f ? 1.0f : fmaxf(__fdiv_rn(amax, top), 1.17549435e-38f);
}

// x / s in binary32, rounded to nearest. With inv = RN(1/s), x inv is within 2 units in the last
// place of x / s; one correction by the exact remainder x - q s brings it within one, and Markstein's
// theorem (IBM J. Res. Dev. 34, 1990: a quotient within one unit, corrected once more with a
// correctly rounded reciprocal, is the correctly rounded quotient) makes the next one exact. The
// remainders are exact while nothing underflows: scales below 2^-60 or above 2^100 take the
// division itself.
struct Divisor {
  float s;
  uint64_t s2, inv2;  // -s and 1/s, twice
  bool plain;
};
__device__ __forceinline__ uint64_t both(float a, float b) {
  uint64_t x;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
  return x;
}
__device__ __forceinline__ float2 split(uint64_t x) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(x));
  return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t x;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(x) : "l"(a), "l"(b), "l"(c));
  return x;
}
__device__ __forceinline__ Divisor divisor(float s) {
  const float inv = __frcp_rn(s);
  return Divisor{s, both(-s, -s), both(inv, inv), !(s >= 8.673617379884035e-19f && s <= 1.2676506002282294e30f)};
}
// Two quotients at a time (two binary32 operations per instruction).
__device__ __forceinline__ float2 quotient(float2 f, const Divisor& d) {
  const uint64_t x = both(f.x, f.y);
  uint64_t q = fma2(x, d.inv2, 0ull);  // + 0: the rounded product
  q = fma2(fma2(q, d.s2, x), d.inv2, q);
  return split(fma2(fma2(q, d.s2, x), d.inv2, q));
}

// Codes of four quotients, one per byte. int8: |y| <= 127 + 2^-16, so adding 1.5 2^23 + 128 leaves
// rint(y) + 128 in the low byte.
template <int FMT>
__device__ __forceinline__ uint32_t codes4(float2 a, float2 b) {
  if (FMT == KVQ_PAGED_INT8) {
    const float m = 12583040.0f;
    const uint32_t x = __float_as_uint(__fadd_rn(a.x, m)), y = __float_as_uint(__fadd_rn(a.y, m));
    const uint32_t z = __float_as_uint(__fadd_rn(b.x, m)), w = __float_as_uint(__fadd_rn(b.y, m));
    return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
  }
  return (uint32_t)__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3) |
         ((uint32_t)__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3) << 16);
}

// 8 channels of a row: two words of codes.
template <int FMT, bool BF16>
__device__ __forceinline__ uint2 codes8(const uint4& x, const Divisor& d) {
  float2 y[4] = {to_float2<BF16>(x.x), to_float2<BF16>(x.y), to_float2<BF16>(x.z), to_float2<BF16>(x.w)};
  if (d.plain) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = make_float2(__fdiv_rn(y[i].x, d.s), __fdiv_rn(y[i].y, d.s));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = quotient(y[i], d);
  }
  return make_uint2(codes4<FMT>(y[0], y[1]), codes4<FMT>(y[2], y[3]));
}

// A thread holds channels 8n .. 8n + 7 of the four rows 16s + {2i, 2i + 1, 2i + 8, 2i + 9}: one
// operand word of the value tile per channel, or with its neighbour of the other half of 16
// channels the operand words of the key tile. Keys and values of a unit are two CTAs: a CTA lives
// for three round trips and the arithmetic of its rows, and what moves is what the resident CTAs
// hold; with both in one CTA a token of each of 32 requests takes 13.5 us instead of 12.4 (read back
// included), a batch of prompts the same.
template <int BT, int FMT, bool BF16>
__global__ void __launch_bounds__(BT * 4, 1536 / (BT * 4)) paged_append_kernel(const PagedAppendParams p) {
  constexpr int THREADS = BT * 4, WARPS = THREADS / 32, CHUNKS = BT / 4;  // 512-byte chunks of the block's keys or values
  __shared__ __align__(16) uint8_t stage[CHUNKS * kChunkStride];
  __shared__ uint32_t amax_s[WARPS];
  pdl_wait();
  pdl_allow_dependents();
  const int unit = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  const bool key = blockIdx.z == 0;
  const uint32_t n_units = p.status[1];
  const int4 u = p.units[unit];  // within the list whether the step has that many or not
  if (unit == 0 && h == 0 && key && tid == 0 && p.q_start[p.R] > p.n_rows) atomicOr(&p.status[0], KVQ_PAGED_ERR_ROWS);
  if (unit >= (int)n_units) return;
  const int row = u.x, block = u.y, q0 = u.z, before = u.w;
  if (row < 0 || row >= p.R) return;
  const int after = p.lens[row];
  const int full0 = before / BT, full1 = after / BT;
  uint16_t* tail = p.tails + ((int64_t)row * p.H + h) * (p.tails_head / 2);
  const int n = tid & 15, i = (tid >> 4) & 3, s = tid >> 6;
  const uint16_t* src = (key ? p.k : p.v) + h * kPagedDim + n * 8;
  const int64_t stride = key ? p.k_stride : p.v_stride;
  auto tok = [&](int k) { return 16 * s + 2 * i + (k & 1) + (k >> 1) * 8; };  // of the thread's row k

  if (block >= 0) {
    const int id = block < p.max_blocks ? p.block_table[(int64_t)row * p.max_blocks + block] : -1;
    uint4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int t = tok(k), pos = block * BT + t;
      x[k] = make_uint4(0u, 0u, 0u, 0u);
      if (pos >= before) {
        const int64_t r = (int64_t)q0 + (pos - before);
        if (r < p.n_rows) x[k] = *reinterpret_cast<const uint4*>(src + r * stride);
      } else {  // kept in the tail since an earlier step
        const uint16_t* tt = tail + s * (kTileBytes / 2);
        uint32_t* w = reinterpret_cast<uint32_t*>(&x[k]);
#pragma unroll
        for (int c = 0; c < 8; c += 2) {
          if (key)
            w[c / 2] = *reinterpret_cast<const uint32_t*>(tt + tile_k_tail(t & 15, n * 8 + c));
          else
            w[c / 2] = (uint32_t)tt[tile_v_tail(t & 15, n * 8 + c)] | ((uint32_t)tt[tile_v_tail(t & 15, n * 8 + c + 1)] << 16);
        }
      }
    }
    uint32_t top_bits = 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&x[k]);
#pragma unroll
      for (int c = 0; c < 4; ++c) top_bits = __vmaxu2(top_bits, w[c] & 0x7fff7fffu);
    }
    top_bits = __reduce_max_sync(0xffffffffu, max(top_bits & 0xffffu, top_bits >> 16));
    if ((tid & 31) == 0) amax_s[tid / 32] = top_bits;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WARPS; ++w) top_bits = max(top_bits, amax_s[w]);
    const float scale = scale_of<BF16>(top_bits, FMT == KVQ_PAGED_INT8 ? 127.0f : 448.0f);
    const Divisor d = divisor(scale);
    uint8_t* tile = stage + (s >> 1) * 8 * kChunkStride;
    uint2 c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) c[k] = codes8<FMT, BF16>(x[k], d);
    if (key) {
      // this thread keeps two of the four channel pairs of its 16 channels and gets the other half's
      // codes of those
      const int odd = n & 1;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? c[k].x : c[k].y, 1);
        const uint32_t lo = odd ? got : c[k].x, hi = odd ? c[k].y : got;  // channels 0..7 and 8..15: pairs 2 odd, 2 odd + 1
        const int t = tok(k) & 31;
        uint32_t* dst = reinterpret_cast<uint32_t*>(tile + ((t >> 3) * 2 + (n >> 3)) * kChunkStride +
                                                    ((t & 7) * 4 + 2 * odd) * 16 + ((n >> 1) & 3) * 4);
        dst[0] = __byte_perm(lo, hi, 0x5410);
        dst[4] = __byte_perm(lo, hi, 0x7632);
      }
    } else {  // byte k of a word is row k
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        const uint32_t w0 = g < 4 ? c[0].x : c[0].y, w1 = g < 4 ? c[1].x : c[1].y;
        const uint32_t w2 = g < 4 ? c[2].x : c[2].y, w3 = g < 4 ? c[3].x : c[3].y;
        const uint32_t sel = (g & 3) | ((4 + (g & 3)) << 4);
        *reinterpret_cast<uint32_t*>(tile + (n >> 1) * kChunkStride + (g * 4 + i) * 16 + ((n & 1) * 2 + (s & 1)) * 4) =
            __byte_perm(__byte_perm(w0, w1, sel), __byte_perm(w2, w3, sel), 0x5410);
      }
    }
    __syncthreads();
    if (id >= 0 && id < p.n_blocks) {
      uint8_t* out = p.codes + ((int64_t)id * p.H + h) * p.codes_head + (key ? 0 : kTileBytes / 2);
#pragma unroll
      for (int y = tid; y < BT * 8; y += THREADS)  // 256 pieces of 16 bytes from each tile
        *reinterpret_cast<uint4*>(out + (y >> 8) * kTileBytes + (y & 255) * 16) =
            *reinterpret_cast<const uint4*>(stage + (y >> 5) * kChunkStride + (y & 31) * 16);
      if (tid == 0) p.scales[((int64_t)id * p.H + h) * 2 + (key ? 0 : 1)] = scale;
    } else if (tid == 0) {
      atomicOr(&p.status[0], KVQ_PAGED_ERR_TABLE);
    }
  }
  if (block < 0 || block == full0) {  // the request's first unit keeps the rows of the unfinished block
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int t = tok(k), pos = full1 * BT + t;
      const int64_t r = (int64_t)q0 + (pos - before);
      if (pos < before || pos >= after || r >= p.n_rows) continue;
      const uint4 x = *reinterpret_cast<const uint4*>(src + r * stride);
      uint16_t* tt = tail + s * (kTileBytes / 2);
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&x);
#pragma unroll
      for (int c = 0; c < 8; c += 2) {
        if (key) {
          *reinterpret_cast<uint32_t*>(tt + tile_k_tail(t & 15, n * 8 + c)) = w[c / 2];
        } else {
          tt[tile_v_tail(t & 15, n * 8 + c)] = (uint16_t)w[c / 2];
          tt[tile_v_tail(t & 15, n * 8 + c + 1)] = (uint16_t)(w[c / 2] >> 16);
        }
      }
    }
  }
}

// Four codes of a word as binary32.
template <int FMT>
__device__ __forceinline__ float4 values4(uint32_t w) {
  if (FMT == KVQ_PAGED_INT8)
    return make_float4((float)((int)(w & 255u) - 128), (float)((int)((w >> 8) & 255u) - 128),
                       (float)((int)((w >> 16) & 255u) - 128), (float)((int)(w >> 24) - 128));
  const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
  const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
  const float2 x = __half22float2(__half2(a)), y = __half22float2(__half2(b));
  return make_float4(x.x, x.y, y.x, y.y);
}

constexpr int kReadSlots = 32;  // list entries of a CTA

// Read back. Where 32 entries of the list are the 32 tokens of a tile in order (the slots of a
// prompt are, but for its ends), a warp reads the tile as it lies, 16 bytes a lane, and writes
// whole sectors: 2 channels of a key from each of 4 lanes, or 8 channels of a value from 8. Other
// entries are gathered one by one. A run may begin up to 31 entries before this CTA's share (it is
// the earlier CTA's then) or end up to 31 behind it.
template <int FMT, bool BF16, int THREADS>
__global__ void __launch_bounds__(THREADS) paged_dequant_kernel(const PagedDequantParams p) {
  constexpr int kReadWarps = THREADS / 32;
  constexpr int SPAN = kReadSlots + 64;  // 32 entries on both sides
  __shared__ int slot_s[SPAN];
  __shared__ uint32_t next_s[SPAN / 32 + 1];  // bit x: entry x follows entry x - 1 in the same tile
  __shared__ uint16_t runs[kReadSlots], rest[kReadSlots];
  __shared__ int n_runs, n_rest;
  pdl_wait();
  pdl_allow_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, h = blockIdx.y;
  const int64_t base = (int64_t)blockIdx.x * kReadSlots - 32;  // list index of slot_s[0]
  const int64_t n_slots = (int64_t)p.n_blocks * p.bt;
  if (tid == 0) n_runs = n_rest = 0;
  if (tid < SPAN) {
    const int64_t x = base + tid;
    const bool in = x >= 0 && x < p.n;
    const int slot = in ? p.slots[x] : -1;
    const int prev = in && x > 0 ? p.slots[x - 1] : -1;
    slot_s[tid] = slot;
    const uint32_t bits = __ballot_sync(0xffffffffu, in && slot > 0 && slot < n_slots && (slot & 31) != 0 && slot - 1 == prev);
    if (lane == 0) next_s[warp] = bits;
  }
  if (tid == 0) next_s[SPAN / 32] = 0u;
  __syncthreads();
  // whether a whole tile begins at entry x of the span
  auto whole = [&](int x) {
    if (x < 0 || x >= SPAN - 31 || base + x < 0 || slot_s[x] < 0 || slot_s[x] >= n_slots || (slot_s[x] & 31)) return false;
    const int y = x + 1;
    return (__funnelshift_r(next_s[y >> 5], next_s[(y >> 5) + 1], y & 31) & 0x7fffffffu) == 0x7fffffffu;
  };
  if (tid < kReadSlots && base + 32 + tid < p.n) {
    const int x = tid + 32, slot = slot_s[x];
    if (whole(x)) runs[atomicAdd(&n_runs, 1)] = (uint16_t)x;
    if (slot < 0 || !whole(x - (slot & 31))) rest[atomicAdd(&n_rest, 1)] = (uint16_t)x;
  }
  __syncthreads();
  const int g = lane >> 2, l = lane & 3;
  for (int k = warp; k < 4 * n_runs; k += kReadWarps) {  // quarters of tiles: half of the keys or values
    const int x = runs[k >> 2], slot = slot_s[x], half = (k & 1) * 4;
    const int64_t id = slot / p.bt;
    const uint4* tile = reinterpret_cast<const uint4*>(p.codes + (id * p.H + h) * p.codes_head +
                                                       (slot - id * p.bt) / kTileCodeTokens * kTileBytes) + lane;
    const float2 sc = *reinterpret_cast<const float2*>(p.scales + (id * p.H + h) * 2);
    const int64_t step = (int64_t)p.H * kPagedDim, first = ((base + x) * p.H + h) * kPagedDim;
    uint4 w[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) w[c] = tile[((k & 2) * 4 + half + c) * 32];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t u[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
      const int chunk = half + c;
      if (!(k & 2)) {
        float* o = p.k_out + first + ((chunk >> 1) * 8 + g) * step + (chunk & 1) * 64 + l * 2;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 f = values4<FMT>(u[q]);
          *reinterpret_cast<float2*>(o + q * 16) = make_float2(__fmul_rn(f.x, sc.x), __fmul_rn(f.y, sc.x));
          *reinterpret_cast<float2*>(o + q * 16 + 8) = make_float2(__fmul_rn(f.z, sc.x), __fmul_rn(f.w, sc.x));
        }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float* o = p.v_out + first + ((q & 1) * 16 + l * 2) * step + (chunk * 2 + (q >> 1)) * 8 + g;
          const float4 f = values4<FMT>(u[q]);
          o[0] = __fmul_rn(f.x, sc.y);
          o[step] = __fmul_rn(f.y, sc.y);
          o[8 * step] = __fmul_rn(f.z, sc.y);
          o[9 * step] = __fmul_rn(f.w, sc.y);
        }
      }
    }
  }
  const int c0 = lane * 4;
  for (int k0 = warp; k0 < n_rest; k0 += 4 * kReadWarps) {  // the loads of four entries at a time
    uint32_t kc[4][2], vc[4][2];  // codes in [0], or 16-bit entries
    float2 sc[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = k0 + u * kReadWarps;
      if (k >= n_rest) break;
      const int64_t slot = slot_s[rest[k]];
      kc[u][0] = kc[u][1] = vc[u][0] = vc[u][1] = 0u;
      sc[u] = make_float2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff));
      if (slot >= 0 && slot < n_slots) {
        const int64_t id = slot / p.bt;
        const int t = (int)(slot - id * p.bt);
        const uint8_t* tile = p.codes + (id * p.H + h) * p.codes_head + (t / kTileCodeTokens) * kTileBytes;
        sc[u] = *reinterpret_cast<const float2*>(p.scales + (id * p.H + h) * 2);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          kc[u][0] |= (uint32_t)tile[tile_k_code(t % kTileCodeTokens, c0 + c)] << (8 * c);
          vc[u][0] |= (uint32_t)tile[tile_v_code(t % kTileCodeTokens, c0 + c)] << (8 * c);
        }
      } else if (slot < 0 && -1 - slot < (int64_t)p.R * p.bt) {
        const int64_t at = -1 - slot, row = at / p.bt;
        const int t = (int)(at - row * p.bt);
        const uint16_t* tile = p.tails + (row * p.H + h) * (p.tails_head / 2) + (t / kTileTailTokens) * (kTileBytes / 2);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          kc[u][c >> 1] |= (uint32_t)tile[tile_k_tail(t % kTileTailTokens, c0 + c)] << (16 * (c & 1));
          vc[u][c >> 1] |= (uint32_t)tile[tile_v_tail(t % kTileTailTokens, c0 + c)] << (16 * (c & 1));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = k0 + u * kReadWarps;
      if (k >= n_rest) break;
      const int64_t slot = slot_s[rest[k]];
      float4 kf, vf;
      if (slot < 0 && -1 - slot < (int64_t)p.R * p.bt) {
        const float2 a = to_float2<BF16>(kc[u][0]), b = to_float2<BF16>(kc[u][1]);
        const float2 c = to_float2<BF16>(vc[u][0]), d = to_float2<BF16>(vc[u][1]);
        kf = make_float4(a.x, a.y, b.x, b.y);
        vf = make_float4(c.x, c.y, d.x, d.y);
      } else {  // outside the cache the scales are NaN
        kf = values4<FMT>(kc[u][0]);
        vf = values4<FMT>(vc[u][0]);
        kf = make_float4(__fmul_rn(kf.x, sc[u].x), __fmul_rn(kf.y, sc[u].x), __fmul_rn(kf.z, sc[u].x), __fmul_rn(kf.w, sc[u].x));
        vf = make_float4(__fmul_rn(vf.x, sc[u].y), __fmul_rn(vf.y, sc[u].y), __fmul_rn(vf.z, sc[u].y), __fmul_rn(vf.w, sc[u].y));
      }
      const int64_t o = ((base + rest[k]) * p.H + h) * kPagedDim + c0;
      *reinterpret_cast<float4*>(p.k_out + o) = kf;
      *reinterpret_cast<float4*>(p.v_out + o) = vf;
    }
  }
}

template <int FMT, bool BF16>
cudaError_t append_bt(const PagedAppendParams& p, dim3 grid, cudaStream_t stream) {
  switch (p.bt) {
    case 32: return launch_pdl(paged_append_kernel<32, FMT, BF16>, grid, dim3(128), 0, stream, p);
    case 64: return launch_pdl(paged_append_kernel<64, FMT, BF16>, grid, dim3(256), 0, stream, p);
    default: return launch_pdl(paged_append_kernel<128, FMT, BF16>, grid, dim3(512), 0, stream, p);
  }
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendParams& p, int64_t max_units, int fmt, int dtype, cudaStream_t stream) {
  const dim3 grid((unsigned)max_units, (unsigned)p.H, 2);
  if (fmt == KVQ_PAGED_INT8)
    return dtype == KVQ_BF16 ? append_bt<KVQ_PAGED_INT8, true>(p, grid, stream) : append_bt<KVQ_PAGED_INT8, false>(p, grid, stream);
  return dtype == KVQ_BF16 ? append_bt<KVQ_PAGED_E4M3, true>(p, grid, stream) : append_bt<KVQ_PAGED_E4M3, false>(p, grid, stream);
}

template <int FMT, bool BF16>
cudaError_t dequant_threads(const PagedDequantParams& p, cudaStream_t stream) {
  const dim3 grid((unsigned)((p.n + kReadSlots - 1) / kReadSlots), (unsigned)p.H);
  // Entries that are gathered one by one take a warp each, a whole tile takes four warps: more warps
  // shorten a small list, fewer and more CTAs suit a long one (8 heads: 1677 entries 13.6 us with 256
  // threads against 15.9 with 128 (append before it included), 32778 entries 113.5 against 107.5).
  if ((int64_t)grid.x * grid.y <= 2048)
    return launch_pdl(paged_dequant_kernel<FMT, BF16, 256>, grid, dim3(256), 0, stream, p);
  return launch_pdl(paged_dequant_kernel<FMT, BF16, 128>, grid, dim3(128), 0, stream, p);
}

cudaError_t launch_paged_dequant(const PagedDequantParams& p, int fmt, int dtype, cudaStream_t stream) {
  if (fmt == KVQ_PAGED_INT8)
    return dtype == KVQ_BF16 ? dequant_threads<KVQ_PAGED_INT8, true>(p, stream) : dequant_threads<KVQ_PAGED_INT8, false>(p, stream);
  return dtype == KVQ_BF16 ? dequant_threads<KVQ_PAGED_E4M3, true>(p, stream) : dequant_threads<KVQ_PAGED_E4M3, false>(p, stream);
}

}  // namespace kvq
