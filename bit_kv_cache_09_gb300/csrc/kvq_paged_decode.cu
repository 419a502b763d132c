// kvq_paged_decode.cu — decode attention over the paged 8-bit cache.
//
// For every request with new tokens, kv head and its r query heads:
//   s_t = scale q . k_t,  m = max s_t,  o = sum 2^(s_t - m) v_t / sum 2^(s_t - m)
// in one pass over the cache with a running maximum and sum.
//
// Bound by HBM: 256 bytes of codes per token and head against 4 * 128 * r operations, which
// go to the tensor cores (m16n8k16, queries as rows, the codes of 8 tokens or 8 channels as
// columns) straight from the bytes of a tile; nothing is transposed or staged twice.
//
// Work split: the tiles (8 KB: 32 tokens of codes or 16 rows of a tail) of all requests and
// heads form one list, [request][head][tile]. The grid is one CTA per SM whatever the
// lengths are, each CTA takes an equal share of the list and each of its 8 warps an equal
// share of that, so ragged batches balance to a tile and lengths need not be known on the
// host. A warp streams its tiles through 3 stages of its own with 8 KB bulk copies (up to
// 192 KB in flight per SM). A (request, head) that one warp holds whole is written at once;
// otherwise the warps of a CTA join their parts through shared memory, and the CTAs of a
// pair through the workspace, where the last to arrive does it (in the order of the list,
// whoever is last, so results do not depend on timing).
//
// Measured on GB300 (8 kv heads): 16 requests of 8 k tokens, r = 4, int8: 50.5 us (5.3 TB/s; the loop
// itself runs at the copy rate, 2.5 us go to the tables, 4 to the joins, 4 between launches); 2 of
// 65 k tokens, r = 8, e4m3: 54.5 us; 64 ragged requests of 36 k tokens in all: 26 us; one of 4 k: 8.8 us.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "kvq_kernels.h"
#include "kvq_paged.cuh"

namespace kvq {
namespace {

constexpr int kWarps = 8;
constexpr int kStages = 3;       // per warp
constexpr int kRows = 8;         // query heads of a kv head, at most
constexpr int kMaxCtas = 256;    // parts in the workspace
constexpr int kPartFloats = kRows * (kPagedDim + 2);  // o [8][128], m [8], l [8]

// Softmax weights are held times 2^15: binary16 then resolves weights of 2^-39 of the largest
// one (2^-29 at full precision), so that a long flat tail of the softmax is not lost.
constexpr float kWeightExp = 15.0f;

struct Smem {
  uint8_t ring[kWarps][kStages][kTileBytes];
  float head[kWarps][kPartFloats];  // parts of pairs that an earlier warp or CTA began
  uint64_t bars[kWarps][kStages];
  int pair_head[kWarps], pair_tail[kWarps];  // pair of each part, -1: none
  int ends[kWarps];                          // the head part reaches its pair's end
  int last[2];
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1) {
  // rows 8..15 of A are zero
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%5}, {%7,%8}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(0u), "r"(a2), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%5}, {%7,%8}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(0u), "r"(a2), "r"(b0), "r"(b1));
}

// Two codes (bytes 0 and 1, or 2 and 3, of a word) as binary16, exactly. int8: the stored
// u = q + 128 under the exponent byte 0x64 is 1024 + u; less 1152 that is q. (Products with
// u itself and one correction by 128 sum p save the subtraction, but leave up to 2^-17 of
// the block's largest value where the exact result is 0.) e4m3: converted.
template <int FMT, int HI>
__device__ __forceinline__ uint32_t codes2(uint32_t w) {
  if (FMT == KVQ_PAGED_INT8) {
    const uint32_t u = __byte_perm(w, 0x64646464u, HI ? 0x4342 : 0x4140), c = 0x64806480u;  // c: 1152, 1152
    const __half2 q = __hsub2(*reinterpret_cast<const __half2*>(&u), *reinterpret_cast<const __half2*>(&c));
    return *reinterpret_cast<const uint32_t*>(&q);
  }
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(HI ? w >> 16 : w & 0xffffu), __NV_E4M3);
  return (uint32_t)h.x | ((uint32_t)h.y << 16);
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
__device__ __forceinline__ uint32_t pack_bf162(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_bf162(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What a lane knows of one tile of the list.
struct TileInfo {
  const uint8_t* src;  // nullptr: a block number outside the pool
  int pair;            // request * H + head
  int tokens;          // > 0: a tile of codes; <= 0: minus the tokens of a tail tile
  int flags;           // 1: first tile of its pair, 2: last
  int block_head;      // of a tile of codes: block * H + head
  float ks, vs;
};

// 32 request rows from `row` on, one per lane: where their tiles start and how long they are.
struct RowWindow {
  int row, start, len;
};

__device__ __forceinline__ RowWindow row_window(const PagedDecodeParams& p, int row) {
  const int i = min(row + (int)(threadIdx.x & 31), p.R);
  return RowWindow{row, p.tile_start[i], p.lens[min(i, p.R - 1)]};
}

// One round of a search for the last row of lo .. hi - 1 whose tiles start at or before v, with
// tile_start[lo] <= v < tile_start[hi]: 32 samples, lane i holding sample i, leave 1/32 of the rows.
__device__ __forceinline__ int search_step(int lo, int hi) { return (hi - lo + 31) >> 5; }
__device__ __forceinline__ void narrow(int& lo, int& hi, int v, int sample) {
  const int step = search_step(lo, hi), i = lo + (int)(threadIdx.x & 31) * step;
  lo += (__popc(__ballot_sync(0xffffffffu, i < hi && sample <= v)) - 1) * step;
  hi = min(lo + step, hi);
}

// Moves the window up to at most 31 rows before the row of tile v (all lanes, the same v).
__device__ __forceinline__ void seek(const PagedDecodeParams& p, RowWindow& w, int lo, int hi, int v) {
  while (hi - lo > 31) narrow(lo, hi, v, p.tile_start[min(lo + (int)(threadIdx.x & 31) * search_step(lo, hi), hi)]);
  w = row_window(p, lo);
}

// Tile x of the list for every lane with x < end (all lanes call it, with rising x).
__device__ __forceinline__ TileInfo tile_info(const PagedDecodeParams& p, RowWindow& w, int x, int end) {
  TileInfo ti{nullptr, -1, 32, 0, -1, 0.0f, 0.0f};
  const int v = min(x, end - 1) / p.H;
  int row = 0, t0 = 0, t1 = 1, len = 0;
  for (bool todo = x < end;;) {
    int k = 0;  // last row of the window that starts at or before v
#pragma unroll
    for (int step = 16; step > 0; step >>= 1)
      if (__shfl_sync(0xffffffffu, w.start, k + step) <= v) k += step;
    const int a = __shfl_sync(0xffffffffu, w.start, k), b = __shfl_sync(0xffffffffu, w.start, min(k + 1, 31));
    const int c = __shfl_sync(0xffffffffu, w.len, k);
    if (todo && k < 31) {  // the row and the next one's start are in the window
      row = w.row + k;
      t0 = a;
      t1 = b;
      len = c;
      todo = false;
    }
    const uint32_t left = __ballot_sync(0xffffffffu, todo);
    if (!left) break;
    seek(p, w, w.row + 31, p.R, __shfl_sync(0xffffffffu, v, __ffs(left) - 1));
  }
  if (x >= end) return ti;
  const int nt = t1 - t0, rem = x - t0 * p.H, h = rem / nt, t = rem - h * nt;
  const int full = len / p.bt, per = p.bt / kTileCodeTokens;
  ti.pair = row * p.H + h;
  ti.flags = (t == 0 ? 1 : 0) | (t == nt - 1 ? 2 : 0);
  if (t < full * per) {
    const int block = t / per;
    const int id = block < p.max_blocks ? p.block_table[(int64_t)row * p.max_blocks + block] : -1;
    if (id >= 0 && id < p.n_blocks) {
      ti.block_head = id * p.H + h;
      ti.src = p.codes + (int64_t)ti.block_head * p.codes_head + (t - block * per) * kTileBytes;
    } else {
      atomicOr(&p.status[0], KVQ_PAGED_ERR_TABLE);
    }
  } else {
    const int tt = t - full * per;
    ti.tokens = -min(kTileTailTokens, len - full * p.bt - tt * kTileTailTokens);
    ti.src = p.tails + (int64_t)ti.pair * p.tails_head + tt * kTileBytes;
  }
  return ti;
}

__device__ __forceinline__ void load_scales(const PagedDecodeParams& p, TileInfo& ti) {
  if (ti.block_head < 0) return;
  const float2 sc = *reinterpret_cast<const float2*>(p.scales + (int64_t)ti.block_head * 2);
  ti.ks = sc.x;
  ti.vs = sc.y;
}

__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// Waits for a phase of a stage's barrier, at most wait_ns (0: gives up at once).
__device__ __forceinline__ bool wait_stage(uint64_t* bar, uint32_t parity, uint64_t wait_ns) {
  uint32_t ok = 0;
  uint64_t t0 = 0;
  if (wait_ns == 0) return false;
  for (int i = 0;; ++i) {
    asm volatile(
        "{\n.reg .pred q;\nmbarrier.try_wait.parity.shared::cta.b64 q, [%1], %2;\nselp.u32 %0, 1, 0, q;\n}"
        : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    if (ok) return true;
    if (i == 64) t0 = now_ns();
    if (i > 64 && now_ns() - t0 > wait_ns) return false;
  }
}

// Counts the CTA in at its pair. The release covers what the CTA's other threads wrote before the
// barrier in front, the acquire what the CTAs counted before wrote.
__device__ __forceinline__ uint32_t take_ticket(uint32_t* ticket) {
  uint32_t n;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(n) : "l"(ticket) : "memory");
  return n;
}

template <int FMT, bool BF16>
__global__ void __launch_bounds__(kWarps * 32, 1) paged_decode_kernel(const PagedDecodeParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, qi = lane & 3;
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s)
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(&sm.bars[warp][s])) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    sm.pair_head[warp] = sm.pair_tail[warp] = -1;
    sm.ends[warp] = 0;
  }
  __syncwarp();
  // With early tables only the lengths and block numbers are read in front of the wait for the
  // previous kernel, which may still be writing tails, codes, scales and queries.
  if (!p.early) pdl_wait();

  const int H = p.H, r = p.r;
  // one round trip: the number of tiles, and the first rows or samples of the search for this warp's row
  RowWindow window = row_window(p, 0);
  const int sample = p.tile_start[min(lane * search_step(0, p.R), p.R)];
  const int total = p.tile_start[p.R] * H;
  // at least one tile per warp, so that short lists need no joining across CTAs
  const int ctas = max(1, min((int)gridDim.x, total / kWarps));
  const int cta = blockIdx.x;
  const int a_cta = (int)((int64_t)total * min(cta, ctas) / ctas), b_cta = (int)((int64_t)total * min(cta + 1, ctas) / ctas);
  const int x_beg = a_cta + (b_cta - a_cta) * warp / kWarps, x_end = a_cta + (b_cta - a_cta) * (warp + 1) / kWarps;
  if (p.R > 31 && x_beg < x_end) {
    int lo = 0, hi = p.R;
    narrow(lo, hi, x_beg / H, sample);
    seek(p, window, lo, hi, x_beg / H);
  }
  TileInfo next = tile_info(p, window, x_beg + lane, x_end);
  if (p.early) pdl_wait();
  pdl_allow_dependents();
  if (p.zero_rest) {  // rows without new tokens, shared out over the CTAs
    for (int row = cta; row < p.R; row += gridDim.x)
      if (p.q_start[row + 1] == p.q_start[row]) {
        uint32_t* o = reinterpret_cast<uint32_t*>(p.out + (int64_t)row * H * r * kPagedDim);
        for (int i = threadIdx.x; i < H * r * kPagedDim / 2; i += kWarps * 32) o[i] = 0u;
      }
  }
  if (cta >= ctas || total == 0) return;
  load_scales(p, next);
  TileInfo cur = next;
  int issue = x_beg, next_base = x_beg, cur_base = x_beg;
  bool dead = false;  // a wait ran out: no more copies, the bookkeeping goes on
  auto issue_one = [&]() {  // starts the copy of tile `issue`
    if (issue - next_base == 32) {
      next_base = issue;
      next = tile_info(p, window, issue + lane, x_end);
      load_scales(p, next);
    }
    const int first_of = __shfl_sync(0xffffffffu, next.flags, issue - next_base) & 1;
    if (first_of || issue == x_beg) {  // the pair's queries are wanted soon
      const int pr = __shfl_sync(0xffffffffu, next.pair, issue - next_base);
      if (lane < 2 * r) {
        const int row = pr / H, h = pr - row * H;
        asm volatile("prefetch.global.L1 [%0];" ::"l"(p.q + (int64_t)row * p.q_stride + h * r * kPagedDim + lane * 64));
      }
    }
    const uint64_t src = __shfl_sync(0xffffffffu, (uint64_t)(uintptr_t)next.src, issue - next_base);
    const int s = (issue - x_beg) % kStages;
    if (lane == 0 && !dead) {
      const uint32_t bar = smem_u32(&sm.bars[warp][s]);
      if (src) {
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(kTileBytes) : "memory");
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                     ::"r"(smem_u32(sm.ring[warp][s])), "l"(src), "r"(kTileBytes), "r"(bar) : "memory");
      } else {
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
      }
    }
    ++issue;
  };
  while (issue < x_end && issue < x_beg + kStages) issue_one();

  uint32_t q16[8][2], qraw[BF16 ? 8 : 1][2];  // A fragments of the queries (row g)
  float o[16][2], m = -INFINITY, l = 0.0f, row_scale = 0.0f;  // l: of this lane's tokens
  int seg_first = 0;

  for (int x = x_beg; x < x_end; ++x) {
    if (x - cur_base == 32) {
      cur_base = x;
      cur = next;
    }
    const int src_lane = x - cur_base;
    const int tokens = __shfl_sync(0xffffffffu, cur.tokens, src_lane), flags = __shfl_sync(0xffffffffu, cur.flags, src_lane);
    const int pair = __shfl_sync(0xffffffffu, cur.pair, src_lane);
    const float ks = __shfl_sync(0xffffffffu, cur.ks, src_lane), vs = __shfl_sync(0xffffffffu, cur.vs, src_lane);
    const bool bad = __shfl_sync(0xffffffffu, cur.src == nullptr ? 1 : 0, src_lane);
    if (x == x_beg || (flags & 1)) {  // a new pair: its queries
      seg_first = flags & 1;
      m = -INFINITY;
      l = 0.0f;
#pragma unroll
      for (int n = 0; n < 16; ++n) o[n][0] = o[n][1] = 0.0f;
      const int row = pair / H, h = pair - row * H;
      const uint16_t* q = p.q + (int64_t)row * p.q_stride + (h * r + g) * kPagedDim + qi * 2;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        q16[k][0] = g < r ? *reinterpret_cast<const uint32_t*>(q + k * 16) : 0u;
        q16[k][1] = g < r ? *reinterpret_cast<const uint32_t*>(q + k * 16 + 8) : 0u;
      }
      row_scale = p.scale_log2;
      if constexpr (BF16) {  // a power of two brings the row's largest entry to [2^14, 2^15)
        uint32_t top = 0u;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          qraw[k][0] = q16[k][0];
          qraw[k][1] = q16[k][1];
          top = __vmaxu2(top, __vmaxu2(q16[k][0] & 0x7fff7fffu, q16[k][1] & 0x7fff7fffu));
        }
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = max((int)(top >> 7) - 127, -112);  // both factors stay normal numbers
        const float up = __int_as_float((127 + 14 - e) << 23);
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 f = unpack_bf162(q16[k][i]);
            q16[k][i] = pack_half2(f.x * up, f.y * up);
          }
        row_scale = p.scale_log2 * __int_as_float((127 + e - 14) << 23);
      }
    }
    const int s = (x - x_beg) % kStages;
    const uint32_t parity = ((x - x_beg) / kStages) & 1;
    if (!dead) {
      const bool ok = wait_stage(&sm.bars[warp][s], parity, p.wait_ns);
      if (!__all_sync(0xffffffffu, ok)) {
        dead = true;
        if (lane == 0) atomicOr(p.err, KVQ_DECODE_ERR_WAIT_TIMEOUT);
        for (int y = x; y < issue; ++y)  // let what is in flight land, again with a limit
          wait_stage(&sm.bars[warp][(y - x_beg) % kStages], ((y - x_beg) / kStages) & 1, kDefaultWaitNs);
      }
    }
    const uint4* tile = reinterpret_cast<const uint4*>(sm.ring[warp][s]) + lane;
    if (bad || dead) {
    } else if (tokens > 0) {
      float sc[4][4];
      const float f = row_scale * ks;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.0f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint4 w = tile[(j * 2 + c) * 32];
          mma_f16(sc[j], q16[c * 4][0], q16[c * 4][1], codes2<FMT, 0>(w.x), codes2<FMT, 1>(w.x));
          mma_f16(sc[j], q16[c * 4 + 1][0], q16[c * 4 + 1][1], codes2<FMT, 0>(w.y), codes2<FMT, 1>(w.y));
          mma_f16(sc[j], q16[c * 4 + 2][0], q16[c * 4 + 2][1], codes2<FMT, 0>(w.z), codes2<FMT, 1>(w.z));
          mma_f16(sc[j], q16[c * 4 + 3][0], q16[c * 4 + 3][1], codes2<FMT, 0>(w.w), codes2<FMT, 1>(w.w));
        }
      }
      float mt = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sc[j][0] *= f;
        sc[j][1] *= f;
        mt = fmaxf(mt, fmaxf(sc[j][0], sc[j][1]));
      }
      const float mn = fmaxf(m, quad_max(mt));
      const float alpha = exp2_fast(m - mn), off = kWeightExp - mn;
      const bool rescale = __any_sync(0xffffffffu, mn > m);
      m = mn;
      uint32_t pw[4];
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // rounded once to binary16; the sum takes the rounded weights
        pw[j] = pack_half2(exp2_fast(sc[j][0] + off), exp2_fast(sc[j][1] + off));
        const float2 e = unpack_half2(pw[j]);
        sum += e.x + e.y;
      }
      if (rescale) {
        l *= alpha;
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          o[n][0] *= alpha;
          o[n][1] *= alpha;
        }
      }
      l += sum;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint4 w = tile[(8 + c) * 32];
        float acc[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
        mma_f16(acc[0], pw[0], pw[1], codes2<FMT, 0>(w.x), codes2<FMT, 1>(w.x));
        mma_f16(acc[1], pw[0], pw[1], codes2<FMT, 0>(w.z), codes2<FMT, 1>(w.z));
        mma_f16(acc[0], pw[2], pw[3], codes2<FMT, 0>(w.y), codes2<FMT, 1>(w.y));
        mma_f16(acc[1], pw[2], pw[3], codes2<FMT, 0>(w.w), codes2<FMT, 1>(w.w));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          o[c * 2 + i][0] = fmaf(vs, acc[i][0], o[c * 2 + i][0]);
          o[c * 2 + i][1] = fmaf(vs, acc[i][1], o[c * 2 + i][1]);
        }
      }
    } else {  // 16 rows of 16 bits, the first -tokens of them valid
      const int valid = -tokens;
      float sc[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.0f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 w = tile[(j * 4 + c) * 32];
          if constexpr (BF16) {
            mma_bf16(sc[j], qraw[c * 2][0], qraw[c * 2][1], w.x, w.y);
            mma_bf16(sc[j], qraw[c * 2 + 1][0], qraw[c * 2 + 1][1], w.z, w.w);
          } else {
            mma_f16(sc[j], q16[c * 2][0], q16[c * 2][1], w.x, w.y);
            mma_f16(sc[j], q16[c * 2 + 1][0], q16[c * 2 + 1][1], w.z, w.w);
          }
        }
      }
      bool in[4];  // tokens 2 qi, 2 qi + 1, + 8
      float mt = -INFINITY;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        in[i] = (i >> 1) * 8 + qi * 2 + (i & 1) < valid;
        float& e = sc[i >> 1][i & 1];
        e = in[i] ? e * p.scale_log2 : -INFINITY;
        mt = fmaxf(mt, e);
      }
      const float mn = fmaxf(m, quad_max(mt)), base = mn == -INFINITY ? 0.0f : mn;  // scores of -inf so far: weights of 0
      const float alpha = exp2_fast(m - base), off = kWeightExp - base;
      m = mn;
      float e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = in[i] ? exp2_fast(sc[i >> 1][i & 1] + off) : 0.0f;
      uint32_t hi[2], lo[2] = {0u, 0u};
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if constexpr (BF16) {  // two bfloat16 parts hold 16 bits of the weight
          hi[j] = pack_bf162(e[j * 2], e[j * 2 + 1]);
          const float2 f = unpack_bf162(hi[j]);
          lo[j] = pack_bf162(e[j * 2] - f.x, e[j * 2 + 1] - f.y);
          sum += e[j * 2] + e[j * 2 + 1];
        } else {
          hi[j] = pack_half2(e[j * 2], e[j * 2 + 1]);
          const float2 f = unpack_half2(hi[j]);
          sum += f.x + f.y;
        }
      }
      l = l * alpha + sum;
      // value rows behind the last token are whatever an earlier request left: cleared
      const uint32_t k0 = (in[0] ? 0xffffu : 0u) | (in[1] ? 0xffff0000u : 0u);
      const uint32_t k1 = (in[2] ? 0xffffu : 0u) | (in[3] ? 0xffff0000u : 0u);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        uint4 w = tile[(8 + c) * 32];
        w.x &= k0;
        w.y &= k1;
        w.z &= k0;
        w.w &= k1;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float acc[4] = {o[c * 2 + i][0] * alpha, o[c * 2 + i][1] * alpha, 0.0f, 0.0f};
          const uint32_t b0 = i ? w.z : w.x, b1 = i ? w.w : w.y;
          if constexpr (BF16) {
            mma_bf16(acc, hi[0], hi[1], b0, b1);
            mma_bf16(acc, lo[0], lo[1], b0, b1);
          } else {
            mma_f16(acc, hi[0], hi[1], b0, b1);
          }
          o[c * 2 + i][0] = acc[0];
          o[c * 2 + i][1] = acc[1];
        }
      }
    }
    __syncwarp();  // every lane is done with the stage
    if (issue < x_end) issue_one();

    if ((flags & 2) || x == x_end - 1) {  // the pair's last tile, or this warp's
      l = quad_sum(l);
      if (seg_first && (flags & 2)) {  // the whole pair: write it
        const float inv = 1.0f / l;
        if (g < r) {
          uint16_t* out = p.out + ((int64_t)pair * r + g) * kPagedDim + qi * 2;
#pragma unroll
          for (int n = 0; n < 16; ++n) {
            const float a = o[n][0] * inv, b = o[n][1] * inv;
            *reinterpret_cast<uint32_t*>(out + n * 8) = BF16 ? pack_bf162(a, b) : pack_half2(a, b);
          }
        }
      } else {
        // a part that begins its pair is this warp's last one: its ring is free by then
        float* part = seg_first ? reinterpret_cast<float*>(sm.ring[warp][0]) : sm.head[warp];
        if (seg_first) {
          if (lane == 0) sm.pair_tail[warp] = pair;
        } else if (lane == 0) {
          sm.pair_head[warp] = pair;
          sm.ends[warp] = (flags & 2) ? 1 : 0;
        }
        if (g < r) {
#pragma unroll
          for (int n = 0; n < 16; ++n)
            *reinterpret_cast<float2*>(part + g * kPagedDim + n * 8 + qi * 2) = make_float2(o[n][0], o[n][1]);
          if (qi == 0) {
            part[kRows * kPagedDim + g] = m;
            part[kRows * kPagedDim + kRows + g] = l;
          }
        }
      }
    }
  }
  __syncthreads();

  // Join the parts of this CTA. They follow one another as head and tail parts of warps 0, 1,
  // ...; neighbours of the same pair form a group. Warp i does query head i of every group.
  const int c0 = lane * 4;
  int open_pair[2] = {-1, -1};  // begun before this CTA; going on behind it
  for (int first = 0; first < 2 * kWarps;) {
    const int pair = (first & 1) ? sm.pair_tail[first >> 1] : sm.pair_head[first >> 1];
    int next_part = first + 1;
    bool ends = !(first & 1) && sm.ends[first >> 1];
    if (pair >= 0) {
      for (; next_part < 2 * kWarps; ++next_part) {
        const int other = (next_part & 1) ? sm.pair_tail[next_part >> 1] : sm.pair_head[next_part >> 1];
        if (other < 0) continue;
        if (other != pair) break;
        ends = ends || sm.ends[next_part >> 1];
      }
      if (warp < r) {
        // part i of the group is the head part of warp i, but for a tail part that begins it; all loads
        // are independent of one another
        const int wa = first >> 1, wb = (next_part - 1) >> 1;
        float mi[kWarps], li[kWarps];
        float4 v[kWarps];
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
          const bool tail = i == wa && (first & 1);
          const bool is = i >= wa && i <= wb && (tail || sm.pair_head[i] == pair);
          const float* part = tail ? reinterpret_cast<const float*>(sm.ring[i][0]) : sm.head[i];
          mi[i] = is ? part[kRows * kPagedDim + warp] : -INFINITY;
          li[i] = is ? part[kRows * kPagedDim + kRows + warp] : 0.0f;
          v[i] = is ? *reinterpret_cast<const float4*>(part + warp * kPagedDim + c0) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        float M = -INFINITY, L = 0.0f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) M = fmaxf(M, mi[i]);
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
          const float w = mi[i] == -INFINITY ? 0.0f : exp2_fast(mi[i] - M);
          L = fmaf(w, li[i], L);
          acc.x = fmaf(w, v[i].x, acc.x);
          acc.y = fmaf(w, v[i].y, acc.y);
          acc.z = fmaf(w, v[i].z, acc.z);
          acc.w = fmaf(w, v[i].w, acc.w);
        }
        if ((first & 1) && ends) {  // begun and ended in this CTA
          const float inv = 1.0f / L;
          uint2 y;
          y.x = BF16 ? pack_bf162(acc.x * inv, acc.y * inv) : pack_half2(acc.x * inv, acc.y * inv);
          y.y = BF16 ? pack_bf162(acc.z * inv, acc.w * inv) : pack_half2(acc.z * inv, acc.w * inv);
          *reinterpret_cast<uint2*>(p.out + ((int64_t)pair * r + warp) * kPagedDim + c0) = y;
        } else {
          float* part = p.parts + ((int64_t)cta * 2 + (first & 1)) * kPartFloats;
          *reinterpret_cast<float4*>(part + warp * kPagedDim + c0) = acc;
          if (lane == 0) {
            part[kRows * kPagedDim + warp] = M;
            part[kRows * kPagedDim + kRows + warp] = L;
          }
        }
      }
      if (!(first & 1)) open_pair[0] = pair;
      else if (!ends) open_pair[1] = pair;
    }
    first = pair >= 0 ? next_part : first + 1;
  }
  if (open_pair[0] < 0 && open_pair[1] < 0) return;

  // At most one pair was begun before this CTA and one goes on behind it. The last CTA of a
  // pair to arrive joins its parts.
  __syncthreads();
  int from[2], to[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    from[k] = to[k] = 0;
    if (open_pair[k] < 0) continue;
    const int row = open_pair[k] / H, h = open_pair[k] - row * H;
    const int t0 = p.tile_start[row], nt = p.tile_start[row + 1] - t0;
    const int64_t beg = (int64_t)t0 * H + (int64_t)h * nt;
    // tile x belongs to CTA ((x + 1) ctas - 1) / total
    from[k] = (int)(((beg + 1) * ctas - 1) / total);
    to[k] = (int)(((beg + nt) * ctas - 1) / total);
    if (threadIdx.x == k * 32)
      sm.last[k] = take_ticket(&p.tickets[open_pair[k]]) == (uint32_t)(to[k] - from[k]);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (open_pair[k] < 0 || !sm.last[k]) continue;
    if (warp < r) {
      auto part_of = [&](int c) { return p.parts + ((int64_t)c * 2 + (c == from[k] ? 1 : 0)) * kPartFloats; };
      float M = -INFINITY, L = 0.0f;
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int c1 = from[k]; c1 <= to[k]; c1 += 16) {  // 16 parts in flight at a time
        float mi[16], li[16];
        float4 v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float* part = part_of(min(c1 + i, to[k]));
          mi[i] = c1 + i <= to[k] ? __ldcg(part + kRows * kPagedDim + warp) : -INFINITY;
          li[i] = __ldcg(part + kRows * kPagedDim + kRows + warp);
          v[i] = __ldcg(reinterpret_cast<const float4*>(part + warp * kPagedDim + c0));
        }
        float mn = M;
#pragma unroll
        for (int i = 0; i < 16; ++i) mn = fmaxf(mn, mi[i]);
        const float a = M == -INFINITY ? 0.0f : exp2_fast(M - mn);
        M = mn;
        L *= a;
        acc.x *= a;
        acc.y *= a;
        acc.z *= a;
        acc.w *= a;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float w = mi[i] == -INFINITY ? 0.0f : exp2_fast(mi[i] - M);
          L = fmaf(w, li[i], L);
          acc.x = fmaf(w, v[i].x, acc.x);
          acc.y = fmaf(w, v[i].y, acc.y);
          acc.z = fmaf(w, v[i].z, acc.z);
          acc.w = fmaf(w, v[i].w, acc.w);
        }
      }
      const float inv = 1.0f / L;
      uint2 y;
      y.x = BF16 ? pack_bf162(acc.x * inv, acc.y * inv) : pack_half2(acc.x * inv, acc.y * inv);
      y.y = BF16 ? pack_bf162(acc.z * inv, acc.w * inv) : pack_half2(acc.z * inv, acc.w * inv);
      *reinterpret_cast<uint2*>(p.out + ((int64_t)open_pair[k] * r + warp) * kPagedDim + c0) = y;
    }
    if (threadIdx.x == 0) p.tickets[open_pair[k]] = 0u;  // ready for the next call
  }
}

template <int FMT, bool BF16>
cudaError_t launch(const PagedDecodeParams& p, cudaStream_t stream) {
  static std::atomic<int> sm_count[64];  // per device; set once its kernel may use the shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int sms = dev < 64 ? sm_count[dev].load(std::memory_order_relaxed) : 0;
  if (sms == 0) {
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(paged_decode_kernel<FMT, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem));
    if (e != cudaSuccess) return e;
    if (dev < 64) sm_count[dev].store(sms, std::memory_order_relaxed);
  }
  return launch_pdl(paged_decode_kernel<FMT, BF16>, dim3(std::min(sms, kMaxCtas)), dim3(kWarps * 32), sizeof(Smem), stream, p);
}

}  // namespace

// Error word, tickets [R * H], parts [kMaxCtas][2][kPartFloats].
size_t paged_workspace_bytes(const PagedGeometry& g) {
  return paged_workspace_parts(g) + sizeof(float) * kMaxCtas * 2 * kPartFloats;
}

cudaError_t launch_paged_decode(const PagedDecodeParams& p, int fmt, int dtype, cudaStream_t stream) {
  if (fmt == KVQ_PAGED_INT8)
    return dtype == KVQ_BF16 ? launch<KVQ_PAGED_INT8, true>(p, stream) : launch<KVQ_PAGED_INT8, false>(p, stream);
  return dtype == KVQ_BF16 ? launch<KVQ_PAGED_E4M3, true>(p, stream) : launch<KVQ_PAGED_E4M3, false>(p, stream);
}

}  // namespace kvq
