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
// one for block numbers) up to some ten thousand tokens, then by finding the row of each token.
// Measured on GB300: 64 requests with a token each 5.1 us, 1000 requests with 65 k tokens 9.4 us.
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

// What one request row adds to the sums; `err` collects what is wrong with it.
struct RowAdds {
  int v[kScans];
  int len, held;  // tokens (0 if out of range) and finished blocks before the step
};
__device__ __forceinline__ RowAdds row_adds(const TablesParams& p, int len, int nw, unsigned& err) {
  RowAdds r{{0, 0, 0, 0, 0}, len, 0};
  const int bt = p.bt;
  if (len < 0 || len / bt > p.max_blocks) { err |= KVQ_PAGED_ERR_STATE; r.len = len = 0; }
  if (nw < -1 || nw > p.max_new) { err |= KVQ_PAGED_ERR_NEW; nw = 0; }
  if (nw > 0 && ((long long)len + nw) / bt > p.max_blocks) { err |= KVQ_PAGED_ERR_LENGTH; nw = 0; }
  const int had = r.held = len / bt;
  if (nw > 0) {
    const int done = (len + nw) / bt - had;
    r.v[0] = nw;
    r.v[1] = done;
    r.v[3] = done > 0 ? done : 1;
    r.v[4] = tiles_of(len + nw, bt);
  } else if (nw < 0) {
    r.v[2] = had;
  }
  return r;
}

__global__ void __launch_bounds__(kThreads) paged_tables_kernel(const TablesParams p) {
  extern __shared__ int32_t pre[];  // kScans arrays of R + 1 prefix sums, lengths [R]
  __shared__ int warp_sum[kThreads / 32][kScans];
  __shared__ long long total_s[2];  // new tokens, blocks held: 64 bits, the others cannot overflow where these are in range
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
  int32_t* len_s = t0 + (R + 1);  // lengths before the step
  if (tid == 0) {
    err_s = 0u;
    total_s[0] = total_s[1] = 0;
  }
  const int n_free = *p.free_count;
  unsigned err = 0u;
  // Every thread sums neighbouring rows, whose loads are all under way at once; one scan joins the
  // threads; then each writes its rows' prefixes.
  const int per = (R + kThreads - 1) / kThreads, i0 = tid * per, i1 = min(R, i0 + per);
  int sum[kScans] = {0, 0, 0, 0, 0};
  long long tokens = 0, held = 0;
#pragma unroll 4
  for (int i = i0; i < i1; ++i) {
    const RowAdds r = row_adds(p, p.lens[i], p.new_tokens[i], err);
#pragma unroll
    for (int k = 0; k < kScans; ++k) sum[k] += r.v[k];
    tokens += r.v[0];
    held += r.held;
  }
  int before[kScans];
#pragma unroll
  for (int k = 0; k < kScans; ++k) {
    int v = sum[k];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, off);
      if (lane >= off) v += y;
    }
    if (lane == 31) warp_sum[warp][k] = v;
    before[k] = v - sum[k];
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    tokens += __shfl_xor_sync(0xffffffffu, tokens, off);
    held += __shfl_xor_sync(0xffffffffu, held, off);
  }
  __syncthreads();
  if (lane == 0) {
    atomicAdd(reinterpret_cast<unsigned long long*>(&total_s[0]), (unsigned long long)tokens);
    atomicAdd(reinterpret_cast<unsigned long long*>(&total_s[1]), (unsigned long long)held);
  }
  int all[kScans];
#pragma unroll
  for (int k = 0; k < kScans; ++k) {
    all[k] = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      const int s = warp_sum[w][k];
      if (w < warp) before[k] += s;
      all[k] += s;
    }
  }
#pragma unroll 4
  for (int i = i0; i < i1; ++i) {
    unsigned same = 0u;
    const RowAdds r = row_adds(p, p.lens[i], p.new_tokens[i], same);
#pragma unroll
    for (int k = 0; k < kScans; ++k) {
      pre[(size_t)k * (R + 1) + i] = before[k];
      before[k] += r.v[k];
    }
    len_s[i] = r.len;
  }
  if (tid < kScans) {
    int x = 0;
    for (int w = 0; w < kThreads / 32; ++w) x += warp_sum[w][tid];
    pre[(size_t)tid * (R + 1) + R] = x;
  }
  if (err) atomicOr(&err_s, err);
  __syncthreads();
  err = err_s;
  if (n_free < 0 || n_free > p.n_blocks || total_s[1] + n_free > p.n_blocks) err |= KVQ_PAGED_ERR_STATE;
  if (total_s[0] > p.max_new) err |= KVQ_PAGED_ERR_NEW;
  // (sums that overflowed belong to a step that is refused already)
  if ((long long)all[1] > (long long)n_free + all[2]) err |= KVQ_PAGED_ERR_BLOCKS;
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
  const int rel = all[2], top = n_free + rel, left = top - all[1];
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
      p.out.lens[i] = nw < 0 ? 0 : len_s[i] + nw;
    }
  }
  if (gid == 0) {
    p.out.free_count[0] = left;
    p.out.status[1] = (uint32_t)all[3];
  }
  for (int i = gid; i < all[1]; i += step) {  // finished blocks get their numbers
    const int row = row_of(a0, R, i);
    p.block_table[(int64_t)row * p.max_blocks + len_s[row] / bt + (i - a0[row])] = entry(top - 1 - i);
  }
  for (int e = n_free + gid; e < left; e += step) p.free_list[e] = entry(e);  // released and not taken again
  for (int i = gid; i < all[3]; i += step) {
    const int row = row_of(u0, R, i);
    const bool fills = a0[row + 1] > a0[row];
    const int len = len_s[row];
    // request, block to quantize, first packed row and tokens cached before
    reinterpret_cast<int4*>(p.out.units)[i] = make_int4(row, fills ? len / bt + (i - u0[row]) : -1, q0[row], len);
  }
  for (int i = gid; i < all[0]; i += step) {
    const int row = row_of(q0, R, i);
    const int len = len_s[row], pos = len + (i - q0[row]);
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
  const size_t smem = (size_t)(kScans + 1) * (p.R + 1) * sizeof(int32_t);
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(paged_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  const int64_t work = (int64_t)p.max_new + p.R;
  const int ctas = (int)std::min<int64_t>(152, (work + 511) / 512);
  return launch_pdl(paged_tables_kernel, dim3(ctas), dim3(kThreads), smem, stream, p);
}

}  // namespace kvq
