// kvq_paged_tables.cu — block tables, slot maps and work lists of a serving step, built on
// the GPU from request lengths.
//
// Everything a step needs follows from prefix sums over the request rows: first packed row
// of each request (sum of new tokens), which free block each finished block gets (sum of
// blocks finished), where released blocks go (sum of blocks released), and the work lists
// of the append and the decode attention. With a stack of `count` free blocks and `rel`
// released ones, the i-th block finished takes stack entry count + rel - 1 - i; an entry at
// or above `count` is a released block that is still in its request's table row, so popping
// never waits for a push.
//
// Each CTA computes all prefix sums itself (a few thousand lengths from L2) and then writes
// its share of the outputs, so one launch does it and no CTA waits for another. The CTA
// that draws the last ticket, when every other one has read the old state, commits the
// lengths and the free count. Bound by latency (launch, one round trip for the lengths,
// one for block numbers) up to some ten thousand tokens, then by writing 8 bytes a token.
#include <cuda_runtime.h>

#include <algorithm>

#include "kvq_kernels.h"
#include "kvq_paged.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 256;
constexpr int kScans = 5;  // new tokens, blocks finished, blocks released, append units, decode tiles

__device__ __forceinline__ int tiles_of(int len, int bt) {  // decode work of `len` tokens, in tiles
  const int full = len / bt;
  return full * (bt / kTileCodeTokens) + (len - full * bt + kTileTailTokens - 1) / kTileTailTokens;
}

// Largest i in [0, n) with first[i] <= x (first[0] <= x; equal neighbours: the last one).
__device__ __forceinline__ int row_of(const int32_t* first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) paged_tables_kernel(const TablesParams p) {
  extern __shared__ int32_t pre[];  // kScans arrays of R + 1 prefix sums
  __shared__ long long warp_sum[kThreads / 32][kScans];
  __shared__ unsigned err_s;
  __shared__ int last_s;
  pdl_wait();
  pdl_allow_dependents();
  const int R = p.R, bt = p.bt, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* q0 = pre;              // new tokens
  int32_t* a0 = pre + (R + 1);    // blocks finished by this step
  int32_t* r0 = a0 + (R + 1);     // blocks released
  int32_t* u0 = r0 + (R + 1);     // append units
  int32_t* t0 = u0 + (R + 1);     // decode tiles
  if (tid == 0) err_s = 0u;
  __syncthreads();
  const int n_free = *p.free_count;
  unsigned err = (n_free < 0 || n_free > p.n_blocks) ? KVQ_PAGED_ERR_STATE : 0u;
  long long base[kScans] = {0, 0, 0, 0, 0}, held = 0;
  for (int i0 = 0; i0 < R; i0 += kThreads) {
    const int i = i0 + tid;
    long long v[kScans] = {0, 0, 0, 0, 0};
    if (i < R) {
      int len = p.lens[i], nw = p.new_tokens[i];
      if (len < 0 || len / bt > p.max_blocks) { err |= KVQ_PAGED_ERR_STATE; len = 0; }
      if (nw < -1 || nw > p.max_new) { err |= KVQ_PAGED_ERR_NEW; nw = 0; }
      if (nw > 0 && ((long long)len + nw) / bt > p.max_blocks) { err |= KVQ_PAGED_ERR_LENGTH; nw = 0; }
      const int had = len / bt;
      held += had;
      if (nw > 0) {
        const int done = (len + nw) / bt - had;
        v[0] = nw;
        v[1] = done;
        v[3] = done > 0 ? done : 1;
        v[4] = tiles_of(len + nw, bt);
      } else if (nw < 0) {
        v[2] = had;
      }
    }
    long long own[kScans];
#pragma unroll
    for (int k = 0; k < kScans; ++k) {
      own[k] = v[k];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, v[k], off);
        if (lane >= off) v[k] += y;
      }
      if (lane == 31) warp_sum[warp][k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kScans; ++k) {
      long long before = base[k], all = 0;
      for (int w = 0; w < kThreads / 32; ++w) {
        const long long s = warp_sum[w][k];
        if (w < warp) before += s;
        all += s;
      }
      if (i < R) pre[(size_t)k * (R + 1) + i] = (int32_t)(before + v[k] - own[k]);
      base[k] += all;
    }
    __syncthreads();
  }
  if (tid < kScans) pre[(size_t)tid * (R + 1) + R] = (int32_t)base[tid];
  for (int off = 16; off > 0; off >>= 1) held += __shfl_xor_sync(0xffffffffu, held, off);
  if (lane == 0) warp_sum[warp][0] = held;
  if (base[0] > p.max_new) err |= KVQ_PAGED_ERR_NEW;
  if (base[1] > (long long)n_free + base[2]) err |= KVQ_PAGED_ERR_BLOCKS;
  __syncthreads();
  held = 0;
  for (int w = 0; w < kThreads / 32; ++w) held += warp_sum[w][0];
  if (held + n_free > p.n_blocks) err |= KVQ_PAGED_ERR_STATE;
  if (err) atomicOr(&err_s, err);
  __syncthreads();
  err = err_s;
  const int gid = blockIdx.x * kThreads + tid, step = gridDim.x * kThreads;
  if (err) {  // refused as a whole: a step without new tokens
    for (int i = gid; i <= R; i += step) {
      p.out.q_start[i] = 0;
      p.out.tile_start[i] = 0;
      if (i < R) p.out.lens[i] = p.lens[i];
    }
    if (gid == 0) {
      p.out.free_count[0] = n_free;
      p.out.status[1] = 0u;
      atomicOr(&p.out.status[0], err);
    }
    return;  // nothing to commit; the ticket stays untouched
  }
  const int rel = (int)base[2], top = n_free + rel, left = top - (int)base[1];
  // stack entry e (below `top`) of the free blocks after the pushes
  auto entry = [&](int e) {
    if (e < n_free) return p.free_list[e];
    const int j = e - n_free;
    const int row = row_of(r0, R, j);
    return p.block_table[(int64_t)row * p.max_blocks + (j - r0[row])];
  };
  for (int i = gid; i <= R; i += step) {
    p.out.q_start[i] = q0[i];
    p.out.tile_start[i] = t0[i];
    if (i < R) {
      const int nw = p.new_tokens[i];
      p.out.lens[i] = nw < 0 ? 0 : p.lens[i] + nw;
    }
  }
  if (gid == 0) {
    p.out.free_count[0] = left;
    p.out.status[1] = (uint32_t)base[3];
  }
  for (int i = gid; i < (int)base[1]; i += step) {  // finished blocks get their numbers
    const int row = row_of(a0, R, i);
    p.block_table[(int64_t)row * p.max_blocks + p.lens[row] / bt + (i - a0[row])] = entry(top - 1 - i);
  }
  for (int e = n_free + gid; e < left; e += step) p.free_list[e] = entry(e);  // released and not taken again
  for (int i = gid; i < (int)base[3]; i += step) {
    const int row = row_of(u0, R, i);
    const bool fills = a0[row + 1] > a0[row];
    const int len = p.lens[row];
    // request, block to quantize, first packed row and tokens cached before
    reinterpret_cast<int4*>(p.out.units)[i] = make_int4(row, fills ? len / bt + (i - u0[row]) : -1, q0[row], len);
  }
  for (int i = gid; i < (int)base[0]; i += step) {
    const int row = row_of(q0, R, i);
    const int len = p.lens[row], pos = len + (i - q0[row]);
    const int block = pos / bt, off = pos - block * bt;
    const int full = (len + (q0[row + 1] - q0[row])) / bt;
    p.out.positions[i] = pos;
    p.out.slots[i] = block < full ? entry(top - 1 - (a0[row] + block - len / bt)) * bt + off : -1 - (row * bt + off);
  }
  if (!p.commit) return;
  __syncthreads();  // this CTA has read lens and free_count for the last time
  if (tid == 0) {
    __threadfence();
    const uint32_t t = atomicAdd(&p.out.status[2], 1u);
    last_s = t == gridDim.x - 1;
    if (last_s) p.out.status[2] = 0u;
  }
  __syncthreads();
  if (!last_s) return;
  for (int i = tid; i < R; i += kThreads) {
    const int nw = p.new_tokens[i];
    p.lens[i] = nw < 0 ? 0 : p.lens[i] + nw;
  }
  if (tid == 0) *p.free_count = left;
}

}  // namespace

cudaError_t launch_paged_tables(const TablesParams& p, cudaStream_t stream) {
  const size_t smem = (size_t)kScans * (p.R + 1) * sizeof(int32_t);
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(paged_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  const int64_t work = (int64_t)p.max_new + p.R;
  const int ctas = (int)std::min<int64_t>(128, (work + 1023) / 1024);
  return launch_pdl(paged_tables_kernel, dim3(ctas), dim3(kThreads), smem, stream, p);
}

}  // namespace kvq
