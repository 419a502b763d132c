// kvq_prompt.cu — attention of packed prompts on the 5th-generation tensor cores.
//
//   s_ij = scale q_i . k_j,  m_i = max_j s_ij,  o_i = sum_j 2^(s_ij - m_i) v_j / sum_j 2^(s_ij - m_i)
// in one pass over the keys with a running maximum and sum per row.
//
// Bound by the tensor cores: 4 * 128 operations per (query row, key). A CTA holds two tiles
// of 128 query rows. A tile is 128 / r tokens of all r query heads of one kv head (the rows of
// a token lie behind one another), so a key tile serves every head of its group. Keys and values
// come in tiles of 128 tokens through a ring of 5 stages filled by TMA. Per key tile j and
// query tile t the MMA warp issues O_t += P_t(j) V_j and S_t(j+1) = Q_t K_{j+1}^T; while
// one tile's four softmax warps turn S into P, the tensor cores work for the other tile.
// S (binary32) and P (16 bits, over the columns of S) and O live in tensor memory:
//   columns 0..127 S_0 / P_0, 128..255 S_1 / P_1, 256..383 O_0, 384..511 O_1.
// A softmax thread owns one row, so maxima and sums need no exchange. The running maximum
// only moves (and O is only rescaled) when a row's maximum grew by more than 2^8: weights
// stay below 2^15, within binary16.
//
// Measured on GB300, 8 kv heads of 4 query heads: 8192 tokens 347 us (1.58 PFLOP/s); a key tile takes
// 2500 cycles for both query tiles against 2048 of the products alone, a CTA 12 k cycles to start and
// to end. Leaving the exponentials out altogether changes 351 us to 348: the products set the pace.
// Their operands in shared memory do too: S reads 128 bytes a cycle.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "kvq_kernels.h"
#include "kvq_prompt.h"

namespace kvq {
namespace {

constexpr int kDim = 128;
constexpr int kTile = 128;                    // query rows of a tile, keys of a tile
constexpr int kPanel = kTile * 128;           // bytes: 128 rows of 64 channels, 128-byte swizzle
constexpr int kTileBytes2 = 2 * kPanel;       // a 128 x 128 tile: two panels
constexpr int kStages = 5;
constexpr int kThreads = 384;                 // 2 x 4 softmax warps; MMA warp, TMA warp and two that look at values
// Registers of a thread: 168 at launch (384 x 168 = 64512); the softmax warps take 208, the
// last four give theirs back (8 x 32 x 208 + 4 x 32 x 88 = 64512).
constexpr int kMmaWarp = 8, kTmaWarp = 9, kScanWarp = 10;
constexpr int kMaxParts = 16;                 // CTAs of a split item
constexpr int kPartTiles = 8;                 // key tiles of a part, at least
constexpr int kPartFloats = kTile * (kDim + 2);  // of one tile's part: o [128][128], m [128], l [128]
constexpr float kMoveAt = 8.0f;               // the maximum moves when it grew by 2^8
// Weights are held times 2^7: with the above below 2^15, and binary16 resolves 2^-31 of the
// largest weight, so that a long flat tail of the softmax is not lost.
constexpr float kWeightExp = 7.0f;

// A sequence's rows, kept inside the arrays whatever the starts say.
struct Span {
  int q0, lq, k0, lk;
};

struct Smem {
  uint8_t q[2][kTileBytes2];
  uint8_t kv[kStages][kTileBytes2];
  uint64_t q_full[2], kv_full[kStages], kv_empty[kStages], s_full[2], p_half[2], p_ready[2], o_full[2], done;
  uint32_t tmem;
  Span span;
  int found, tile, h, part, parts, abort, last, spoiled;
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void bar_init(uint64_t* b, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n.reg .pred q;\nmbarrier.try_wait.parity.shared::cta.b64 q, [%1], %2;\nselp.u32 %0, 1, 0, q;\n}"
               : "=r"(ok) : "r"(smem_u32(b)), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

__device__ __forceinline__ bool bar_give_up(volatile int* abort, uint32_t* err) {
  *abort = 1;
  atomicOr(err, KVQ_DECODE_ERR_WAIT_TIMEOUT);
  return false;
}

// Waits for a phase, at most wait_ns or until another warp gave up. The first to give up says so
// in the error word and to the CTA; every role then leaves its loop.
__device__ __forceinline__ bool bar_wait_slow(uint64_t* b, uint32_t parity, uint64_t wait_ns, volatile int* abort, uint32_t* err) {
  const uint64_t t0 = now_ns();
  for (;;) {
    if (bar_try(b, parity)) return true;
    if (*abort) return false;
    if (now_ns() - t0 > wait_ns) return bar_give_up(abort, err);
  }
}
// A limit of 0 gives up at once.
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity, const PromptParams& p, Smem& sm) {
  if (p.wait_ns == 0) return bar_give_up(&sm.abort, p.err);
  for (int i = 0; i < 8; ++i)
    if (bar_try(b, parity)) return true;
  return bar_wait_slow(b, parity, p.wait_ns, &sm.abort, p.err);
}

// One lane of the (converged) warp. Code behind this predicate, and not behind a test of the lane
// number, issues its MMAs without a loop that makes their operands uniform: 8 of them take 160 to
// 310 cycles instead of 600 to 950, more than the 512 that the tensor cores need.
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(is));
  return is != 0;
}

__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int c, int head, int token, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(smem_u32(dst)), "l"(map), "r"(c), "r"(head), "r"(token), "r"(smem_u32(bar)) : "memory");
}

// Shared-memory operand descriptors, 128-byte swizzle. A tile is two panels of 64 channels;
// groups of 8 rows are 1024 bytes apart.
constexpr uint64_t kDescBase = (uint64_t(2) << 61) | (uint64_t(1) << 46) | (uint64_t(1024 >> 4) << 32);
__device__ __forceinline__ uint64_t desc_rows(uint32_t addr) {  // rows x channels: the product runs along a row
  return kDescBase | (uint64_t(1) << 16) | (addr >> 4);
}
__device__ __forceinline__ uint64_t desc_cols(uint32_t addr) {  // the product runs over the rows; panels side by side
  return kDescBase | (uint64_t(kPanel >> 4) << 16) | (addr >> 4);
}
// Instruction descriptor: binary32 accumulator, 16-bit operands, 128 x 128.
template <bool BF16>
__device__ constexpr uint32_t idesc(bool b_cols) {
  return (1u << 4) | (BF16 ? (1u << 7) | (1u << 10) : 0u) | (b_cols ? 1u << 16 : 0u) | ((kTile >> 3) << 17) | ((kTile >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool add) {
  asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
               ::"r"(d), "l"(a), "l"(b), "r"(id), "r"((uint32_t)add) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool add) {
  asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
               ::"r"(d), "r"(a), "l"(b), "r"(id), "r"((uint32_t)add) : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {  // arrives when every MMA issued so far is done
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

#define KVQ_R4(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3])
#define KVQ_R16(x, i) KVQ_R4(x, i), KVQ_R4(x, i + 4), KVQ_R4(x, i + 8), KVQ_R4(x, i + 12)
#define KVQ_W4(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3])
#define KVQ_W16(x, i) KVQ_W4(x, i), KVQ_W4(x, i + 4), KVQ_W4(x, i + 8), KVQ_W4(x, i + 12)
// 32 columns of this warp's 32 lanes (rows).
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* x) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : KVQ_R16(x, 0), KVQ_R16(x, 16) : "r"(addr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* x) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : KVQ_R16(x, 0) : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* x) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(addr), KVQ_W16(x, 0) : "memory");
}
// Waits for this thread's loads; then names the registers that they fill, so that nothing that reads
// those moves in front of the wait.
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
#define KVQ_U4(x, i) "+r"(x[i]), "+r"(x[i + 1]), "+r"(x[i + 2]), "+r"(x[i + 3])
#define KVQ_U16(x, i) KVQ_U4(x, i), KVQ_U4(x, i + 4), KVQ_U4(x, i + 8), KVQ_U4(x, i + 12)
template <int N>
__device__ __forceinline__ void tmem_wait_ld(uint32_t* x) {
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < N; i += 16) asm volatile("" : KVQ_U16(x, i));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two binary32 lanes in one register pair.
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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t x;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(x) : "l"(a), "l"(b));
  return x;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float x;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(x) : "f"(a), "f"(b), "f"(c));
  return x;
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ Span span_of(const PromptParams& p, int s) {
  Span x;
  x.q0 = min(max(p.q_start[s], 0), p.n_q);
  x.lq = min(max(p.q_start[s + 1], x.q0), p.n_q) - x.q0;
  x.k0 = min(max(p.kv_start[s], 0), p.n_kv);
  x.lk = min(max(p.kv_start[s + 1], x.k0), p.n_kv) - x.k0;
  return x;
}

// How many pairs of query tiles a sequence has.
__device__ __forceinline__ int pairs_of(const Span& x, int tokens) { return (x.lq + 2 * tokens - 1) / (2 * tokens); }

// Sequence, its rows and pair of tiles of item `want` of `parts` parts each (all lanes; SPLIT: parts and
// part are set, else 1 and 0); false: there are fewer. Causal rows further back see more keys, so late
// pairs come first: over all sequences where a lane can hold one each, sequence by sequence where
// there are more.
template <bool SPLIT>
__device__ __forceinline__ bool find_pair(const PromptParams& p, int item, int tokens, Span& sp, int& tile, int& h, int& part,
                                          int& parts) {
  const int lane = threadIdx.x & 31;
  part = 0;
  parts = 1;
  if (p.n_seqs <= 32) {
    Span x{0, 0, 0, 0};
    if (lane < p.n_seqs) x = span_of(p, lane);
    const int n = pairs_of(x, tokens);
    auto from = [&](int level) { return (int)__reduce_add_sync(0xffffffffu, (unsigned)max(0, n - level)); };
    const int pairs = from(0);
    // Where whole items would leave half of the SMs without work, they are split along the keys.
    if (SPLIT && pairs > 0 && 2 * pairs * p.H <= kPromptSplit) {
      parts = min(kPromptSplit / (pairs * p.H), kMaxParts);
      part = item % parts;
      item /= parts;
    }
    int want = item / p.H;
    h = item - want * p.H;
    if (pairs <= want) return false;
    int lo = 0, hi = (int)__reduce_max_sync(0xffffffffu, (unsigned)n);  // from(lo) > want >= from(hi) = 0
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (from(mid) > want) lo = mid; else hi = mid;
    }
    tile = lo;
    want -= from(lo + 1);
    uint32_t have = __ballot_sync(0xffffffffu, n > lo);
    for (; want > 0; --want) have &= have - 1;
    const int l = __ffs(have) - 1;
    sp = Span{__shfl_sync(0xffffffffu, x.q0, l), __shfl_sync(0xffffffffu, x.lq, l), __shfl_sync(0xffffffffu, x.k0, l),
              __shfl_sync(0xffffffffu, x.lk, l)};
    return true;
  }
  int want = item / p.H;
  h = item - want * p.H;
  // 8 sequences per lane, so that a round trip passes 256 of them (512 prompts of 32 tokens: 211 us, 308 with one per lane).
  constexpr int kEach = 8;
  for (int s0 = 0; s0 < p.n_seqs; s0 += 32 * kEach) {
    const int s = s0 + lane * kEach;
    int at[kEach + 1], n[kEach], sum = 0;
#pragma unroll
    for (int i = 0; i <= kEach; ++i) at[i] = min(max(p.q_start[min(s + i, p.n_seqs)], 0), p.n_q);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      n[i] = (max(at[i + 1] - at[i], 0) + 2 * tokens - 1) / (2 * tokens);
      sum += n[i];
    }
    int upto = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += y;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, upto > want);
    if (hit) {
      int mine = 0, end = upto - sum;  // this lane's sequence with the item, and the items up to its end
      bool open = true;
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (open) {
          mine = i;
          end += n[i];
          open = end <= want;
        }
      const int l = __ffs(hit) - 1;
      tile = __shfl_sync(0xffffffffu, end - 1, l) - want;
      sp = span_of(p, s0 + l * kEach + __shfl_sync(0xffffffffu, mine, l));
      return true;
    }
    want -= __shfl_sync(0xffffffffu, upto, 31);
  }
  return false;
}

// Rows r0 .. r0 + 3 (of the 256 of both tiles) of a split item, by one warp:
//   M = max_s m_s, o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s
// in the order of the parts, four at a time in flight.
template <bool BF16>
__device__ __forceinline__ void join_rows(const PromptParams& p, const Span& sp, int h, int t0, int tokens, int slot,
                                          int parts, int r0) {
  const int lane = threadIdx.x & 31, t = r0 / kTile, row0 = r0 % kTile;
  float M[4], L[4];
  float4 A[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    M[i] = -INFINITY;
    L[i] = 0.0f;
    A[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  if (t0 + t * tokens >= sp.lq) return;
  for (int s0 = 0; s0 < parts; s0 += 4) {
    float m[4][4], l[4][4];
    float4 v[4][4];
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* part = p.parts + (int64_t)((slot + min(s0 + s, parts - 1)) * 2 + t) * kPartFloats;
        const bool is = s0 + s < parts;
        m[s][i] = is ? __ldcg(part + kTile * kDim + row0 + i) : -INFINITY;
        l[s][i] = is ? __ldcg(part + kTile * kDim + kTile + row0 + i) : 0.0f;
        v[s][i] = __ldcg(reinterpret_cast<const float4*>(part + (row0 + i) * kDim) + lane);
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mn = M[i];
#pragma unroll
      for (int s = 0; s < 4; ++s) mn = fmaxf(mn, m[s][i]);
      const float a = M[i] == -INFINITY ? 0.0f : exp2_fast(M[i] - mn);
      L[i] *= a;
      A[i] = make_float4(A[i].x * a, A[i].y * a, A[i].z * a, A[i].w * a);
      M[i] = mn;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        // a part without a key for the row: weight 0, its outputs not even written
        const bool none = m[s][i] == -INFINITY;
        const float w = none ? 0.0f : exp2_fast(m[s][i] - mn);
        L[i] = fmaf(w, l[s][i], L[i]);  // NaN scores leave m at -inf and l NaN
        A[i].x = none ? A[i].x : fmaf(w, v[s][i].x, A[i].x);
        A[i].y = none ? A[i].y : fmaf(w, v[s][i].y, A[i].y);
        A[i].z = none ? A[i].z : fmaf(w, v[s][i].z, A[i].z);
        A[i].w = none ? A[i].w : fmaf(w, v[s][i].w, A[i].w);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = row0 + i, token = t0 + t * tokens + row / p.r, head = h * p.r + row % p.r;
    if (row >= tokens * p.r || token >= sp.lq) continue;
    const bool none = M[i] == -INFINITY && L[i] == 0.0f;
    const float inv = none ? 0.0f : 1.0f / L[i];
    const int64_t at = sp.q0 + token;
    *reinterpret_cast<uint2*>(p.out + at * p.out_stride + head * kDim + lane * 4) =
        make_uint2(pack2<BF16>(A[i].x * inv, A[i].y * inv), pack2<BF16>(A[i].z * inv, A[i].w * inv));
    if (p.lse && lane == 0)
      p.lse[at * (p.H * p.r) + head] = none ? -INFINITY : (M[i] - kWeightExp + log2f(L[i])) * 0.6931471805599453f;
  }
}

// Whether a value that some row of the pair of tiles sees and another does not, or one behind the
// last key in the last 16 of the value product, is not finite: its weight of 0 would make the
// other row's sums NaN. By warp w of n, from the rows in memory (at most 271 of 256 bytes, some
// 1 % of what a long item reads; 341 -> 347 us for 8192 tokens, 54.4 -> 56.7 for 12 ragged prompts).
template <bool BF16>
__device__ __forceinline__ bool spoiled_values(const PromptParams& p, const Span& sp, int h, int t0, int tokens, int w, int n) {
  const int lane = threadIdx.x & 31, shift = sp.lk - sp.lq;
  const int from = min(max(t0 + 1 + shift, 0), sp.lk), last = min(max(min(sp.lq, t0 + 2 * tokens) + shift, 0), sp.lk);
  const int to = min(sp.lk, (last + 15) & ~15);
  uint32_t top = 0u;
#pragma unroll 4
  for (int key = from + w * 2 + (lane >> 4); key < to; key += 2 * n) {
    const uint4 x = *reinterpret_cast<const uint4*>(p.v + (int64_t)(sp.k0 + key) * p.v_stride + h * kDim + (lane & 15) * 8);
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
  }
  return __any_sync(0xffffffffu, max(top & 0xffffu, top >> 16) >= (BF16 ? 0x7f80u : 0x7c00u));
}

// One row of the pair (0 .. 255) by one warp, a key at a time over those it sees: for items with
// spoiled values only, where the products of whole tiles cannot tell 0 from nothing.
template <bool BF16>
__device__ __forceinline__ void row_by_row(const PromptParams& p, const Span& sp, int h, int t0, int tokens, int row) {
  const int lane = threadIdx.x & 31, t = row / kTile, in = row % kTile;
  const int token = t0 + t * tokens + in / p.r, head = h * p.r + in % p.r;
  if (in >= tokens * p.r || token >= sp.lq) return;
  const int see = min(max(token + 1 + sp.lk - sp.lq, 0), sp.lk);
  if (see == 0) return;
  auto four = [&](const uint16_t* x) {
    const uint2 w = *reinterpret_cast<const uint2*>(x + lane * 4);
    const uint32_t u[2] = {w.x, w.y};
    float2 f[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      f[i] = BF16 ? make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u))
                  : __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    return make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
  };
  const int64_t at = sp.q0 + token;
  const float4 q = four(p.q + at * p.q_stride + head * kDim);
  float m = -INFINITY, l = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
  for (int j = 0; j < see; ++j) {
    const float4 k = four(p.k + (int64_t)(sp.k0 + j) * p.k_stride + h * kDim), v = four(p.v + (int64_t)(sp.k0 + j) * p.v_stride + h * kDim);
    float s = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, q.w * k.w)));
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
    s = p.scale_log2 == 0.0f ? 0.0f : s * p.scale_log2;
    const float mn = fmaxf(m, s), base = mn == -INFINITY ? 0.0f : mn;  // scores of -inf so far: weights of 0
    const float a = exp2_fast(m - base), e = exp2_fast(s - base);
    m = mn;
    l = l * a + e;
    o = make_float4(o.x * a + e * v.x, o.y * a + e * v.y, o.z * a + e * v.z, o.w * a + e * v.w);
  }
  const float inv = 1.0f / l;
  *reinterpret_cast<uint2*>(p.out + at * p.out_stride + head * kDim + lane * 4) =
      make_uint2(pack2<BF16>(o.x * inv, o.y * inv), pack2<BF16>(o.z * inv, o.w * inv));
}

// SPLIT: items may be split along the keys (a template parameter: with the join in it the kernel for
// whole items takes 361 instead of 342 us for 8192 tokens of 32 heads).
template <bool BF16, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const PromptParams p, const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                  const __grid_constant__ CUtensorMap v_map) {
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tokens = kTile / p.r;  // of a query tile
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      bar_init(&sm.q_full[i], 1);
      bar_init(&sm.s_full[i], 1);
      bar_init(&sm.p_half[i], kTile);
      bar_init(&sm.p_ready[i], kTile);
      bar_init(&sm.o_full[i], 1);
    }
    for (int i = 0; i < kStages; ++i) {
      bar_init(&sm.kv_full[i], 1);
      bar_init(&sm.kv_empty[i], 1);
    }
    bar_init(&sm.done, 1);
    sm.abort = 0;
    sm.spoiled = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kTmaWarp && lane < 3) {
    const CUtensorMap* map = lane == 0 ? &q_map : lane == 1 ? &k_map : &v_map;
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sm.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  pdl_allow_dependents();
  if (warp == 0) {
    Span sp{0, 0, 0, 0};
    int tile = 0, h = 0, part, parts;
    const bool found = find_pair<SPLIT>(p, blockIdx.x, tokens, sp, tile, h, part, parts);
    if (lane == 0) {
      sm.span = sp;
      sm.found = found;
      sm.tile = tile;
      sm.h = h;
      sm.part = part;
      sm.parts = parts;
    }
  }
  if (p.zero_rest) {  // rows of no sequence, shared out over the CTAs
    const int first = min(max(p.q_start[0], 0), p.n_q), last = min(max(p.q_start[p.n_seqs], 0), p.n_q);
    const int nq = p.H * p.r;
    for (int64_t i = blockIdx.x; i < (int64_t)first + (p.n_q - last); i += gridDim.x) {
      const int64_t row = i < first ? i : last + (i - first);
      for (int c = threadIdx.x; c < nq * (kDim / 8); c += kThreads)
        *reinterpret_cast<uint4*>(p.out + row * p.out_stride + c * 8) = make_uint4(0u, 0u, 0u, 0u);
      for (int c = threadIdx.x; p.lse && c < nq; c += kThreads) p.lse[row * nq + c] = -INFINITY;
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sm.tmem;
  const int h = sm.h;
  int parts = 1, slot = 0;  // of a split item; place of this CTA's part in the workspace
  Span sp = sm.span;
  if (sm.found) {
    const int t0 = sm.tile * 2 * tokens;  // first token, within the sequence
    const int shift = sp.lk - sp.lq;      // causal: token i sees keys 0 .. i + shift
    int n_keys[2], n[2];                  // keys that some row of the tile sees, key tiles
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int beg = t0 + t * tokens, end = min(sp.lq, beg + tokens);
      n_keys[t] = beg >= sp.lq ? 0 : p.causal ? min(max(end + shift, 0), sp.lk) : sp.lk;
      n[t] = (n_keys[t] + kTile - 1) / kTile;
    }
    int n_max = max(n[0], n[1]);
    const int see_all = sp.lk;
    int first_key = 0;
    if (SPLIT && sm.parts > 1) {  // this CTA's share of the key tiles; the rest of it counts keys from there
      parts = max(1, min(sm.parts, n_max / kPartTiles));
      const int part = sm.part, j0 = part < parts ? n_max * part / parts : 0, j1 = part < parts ? n_max * (part + 1) / parts : 0;
      slot = blockIdx.x;  // parts of an item have neighbouring slots, all below kPromptSplit
      first_key = j0 * kTile;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        n_keys[t] = min(max(n_keys[t] - first_key, 0), (j1 - j0) * kTile);
        n[t] = (n_keys[t] + kTile - 1) / kTile;
      }
      n_max = max(n[0], n[1]);
      sp.k0 += first_key;
      sp.lk -= first_key;
      if (part >= parts) parts = 0;  // fewer key tiles than parts: this CTA has none
    }

    if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp >= kScanWarp && p.causal) {
      const Span all{sp.q0, sp.lq, sp.k0 - first_key, see_all};
      if (spoiled_values<BF16>(p, all, h, t0, tokens, warp - kScanWarp, 2) && lane == 0) sm.spoiled = 1;
    }
    if (warp == kTmaWarp) {
      if (elect_one() && n_max > 0) {
        int c = 0, give_up = 0;  // key and value tiles sent for
        bool ok = true;
        auto load_kv = [&](const CUtensorMap* map, int j) {
          const int s = c % kStages;
          if (c >= kStages) ok = bar_wait(&sm.kv_empty[s], (c / kStages - 1) & 1, p, sm);
          if (!ok) return;
          bar_expect(&sm.kv_full[s], kTileBytes2);
          tma_load(sm.kv[s], map, 0, h, sp.k0 + j * kTile, &sm.kv_full[s]);
          tma_load(sm.kv[s] + kPanel, map, 64, h, sp.k0 + j * kTile, &sm.kv_full[s]);
          ++c;
        };
        auto load_q = [&](int t) {
          if (n[t] == 0) return;
          bar_expect(&sm.q_full[t], 2 * tokens * p.r * 128);
          tma_load(sm.q[t], &q_map, 0, h * p.r, sp.q0 + t0 + t * tokens, &sm.q_full[t]);
          tma_load(sm.q[t] + kPanel, &q_map, 64, h * p.r, sp.q0 + t0 + t * tokens, &sm.q_full[t]);
        };
        load_q(0);
        load_kv(&k_map, 0);
        load_q(1);
        load_kv(&v_map, 0);
        for (int j = 1; j < n_max && ok; ++j) {
          load_kv(&k_map, j);
          if (ok) load_kv(&v_map, j);
        }
        // Everything has landed before the CTA may end, whoever gave up on it.
        for (int t = 0; t < 2; ++t)
          if (n[t] > 0) bar_wait_slow(&sm.q_full[t], 0, kDefaultWaitNs, &give_up, p.err);
        for (int i = max(0, c - kStages); i < c; ++i)
          bar_wait_slow(&sm.kv_full[i % kStages], (i / kStages) & 1, kDefaultWaitNs, &give_up, p.err);
      }
      __syncwarp();
    } else if (warp == kMmaWarp) {
      if (elect_one() && n_max > 0) {
        bool ok = true;
        const uint32_t q_addr[2] = {smem_u32(sm.q[0]), smem_u32(sm.q[1])}, kv_addr = smem_u32(sm.kv[0]);
        auto scores = [&](int t, int stage) {  // S_t = Q_t K^T
          const uint64_t a = desc_rows(q_addr[t]), b = desc_rows(kv_addr + stage * kTileBytes2);
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            const uint32_t off = ((s >> 2) * kPanel + (s & 3) * 32) >> 4;
            mma_ss(tmem + t * kTile, a + off, b + off, idesc<BF16>(false), s > 0);
          }
          mma_commit(&sm.s_full[t]);
        };
        ok = bar_wait(&sm.kv_full[0], 0, p, sm);
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (ok && n[t] > 0) {
            ok = bar_wait(&sm.q_full[t], 0, p, sm);
            if (ok) scores(t, 0);
          }
        if (ok) mma_commit(&sm.kv_empty[0]);
        for (int j = 0; j < n_max && ok; ++j) {
          const int cv = 2 * j + 1, ck = 2 * j + 2, sv = cv % kStages, sk = ck % kStages;
          ok = bar_wait(&sm.kv_full[sv], (cv / kStages) & 1, p, sm);
          if (!ok) break;
          // Rows behind the sequence's last key belong to another sequence. Weights are 0 there,
          // but 0 times an infinity is not: the product stops at the last 16 rows that hold a
          // key, and what follows the last key among those is cleared.
          const int rest = sp.lk - j * kTile;
          if (rest < kTile && (rest & 15)) {
            for (int i = 0; i < (16 - (rest & 15)) * 16; ++i) {
              const int row = rest + (i >> 4), c = i & 15;
              *reinterpret_cast<uint4*>(sm.kv[sv] + (c >> 3) * kPanel + row * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          const uint64_t v_desc = desc_cols(kv_addr + sv * kTileBytes2);
          bool have_k = false;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (ok && j < n[t]) {
              const int steps = (n_keys[t] - j * kTile + 15) / 16;
#pragma unroll
              for (int half = 0; half < 2; ++half) {  // the first 64 keys while the weights of the others are made
                if (ok) ok = bar_wait(half ? &sm.p_ready[t] : &sm.p_half[t], j & 1, p, sm);
                if (ok) {
                  fence_after();
#pragma unroll
                  for (int s = half * 4; s < half * 4 + 4; ++s)
                    if (s < steps)
                      mma_ts(tmem + 256 + t * kTile, tmem + t * kTile + s * 8, v_desc + s * (2048 >> 4), idesc<BF16>(true),
                             j > 0 || s > 0);
                }
              }
              if (ok && j == n[t] - 1) mma_commit(&sm.o_full[t]);
            }
            if (ok && j + 1 < n[t]) {
              if (!have_k) ok = bar_wait(&sm.kv_full[sk], (ck / kStages) & 1, p, sm);
              have_k = true;
              if (ok) scores(t, sk);
            }
          }
          if (ok) {
            mma_commit(&sm.kv_empty[sv]);
            if (j + 1 < n_max) mma_commit(&sm.kv_empty[sk]);
          }
        }
        // nothing of this CTA is in flight when it ends
        int over = 0;
        mma_commit(&sm.done);
        bar_wait_slow(&sm.done, 0, kDefaultWaitNs, &over, p.err);
      }
      __syncwarp();
    } else if (warp < 8) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
      const int t = warp >> 2, row = (warp & 3) * 32 + lane;
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t s_addr = tmem + lanes + t * kTile, o_addr = tmem + lanes + 256 + t * kTile;
      const int token = t0 + t * tokens + row / p.r, head = h * p.r + row % p.r;
      const bool mine = row < tokens * p.r && token < sp.lq;
      // keys this row sees (rows of no token: as many as the tile, nothing to mask)
      const int see = !mine ? n[t] * kTile : (p.causal ? min(max(token + 1 + shift, 0), see_all) : see_all) - first_key;
      const float scale = p.scale_log2;
      float m = -INFINITY, l = 0.0f;  // m: maximum in use, of scale * s
      bool ok = true;
      for (int j = 0; j < n[t]; ++j) {
        ok = __all_sync(0xffffffffu, bar_wait(&sm.s_full[t], j & 1, p, sm));
        if (!ok) break;
        fence_after();
        uint32_t x[kTile];
#pragma unroll
        for (int c = 0; c < kTile; c += 32) tmem_ld32(s_addr + c, x + c);
        tmem_wait_ld<kTile>(x);
        const int left = see - j * kTile;  // visible keys of this tile
        if (__any_sync(0xffffffffu, left < kTile) || scale == 0.0f) {
#pragma unroll
          for (int c = 0; c < kTile; ++c) {
            const float s = scale == 0.0f ? 0.0f : __uint_as_float(x[c]);
            x[c] = __float_as_uint(c < left ? s : -INFINITY);
          }
        }
        float top[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) top[c] = __uint_as_float(x[c]);
#pragma unroll
        for (int c = 4; c < kTile - 4; c += 8)
#pragma unroll
          for (int i = 0; i < 4; ++i) top[i] = max3(top[i], __uint_as_float(x[c + i]), __uint_as_float(x[c + 4 + i]));
#pragma unroll
        for (int c = kTile - 4; c < kTile; ++c) top[c & 3] = fmaxf(top[c & 3], __uint_as_float(x[c]));
        const float scale_use = scale == 0.0f ? 1.0f : scale;
        const float mt = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale_use;
        const bool move = mt > m + kMoveAt || m == -INFINITY;
        const float m_old = m;
        if (move) m = fmaxf(m, mt);
        if (j > 0 && __any_sync(0xffffffffu, move && m_old != -INFINITY)) {
          // every MMA issued before S_t(j) is done, so O_t stands still
          const float a = exp2_fast(m_old - (m == -INFINITY ? 0.0f : m));
          const float f = m_old == -INFINITY || !move ? 1.0f : a;
          l *= f;
#pragma unroll
          for (int c = 0; c < kDim; c += 16) {
            uint32_t o[16];
            tmem_ld16(o_addr + c, o);
            tmem_wait_ld<16>(o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st16(o_addr + c, o);
          }
        }
        const float off = kWeightExp - (m == -INFINITY ? 0.0f : m);
        uint64_t sum[2] = {0ull, 0ull};
        const uint64_t scale2 = both(scale_use, scale_use), off2 = both(off, off);
#pragma unroll
        for (int c0 = 0; c0 < kTile; c0 += 32) {
          uint32_t w[16];
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float2 e = split(fma2(both(__uint_as_float(x[c0 + c]), __uint_as_float(x[c0 + c + 1])), scale2, off2));
            const float a = exp2_fast(e.x), b = exp2_fast(e.y);
            sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], both(a, b));
            w[c / 2] = pack2<BF16>(a, b);
          }
          tmem_st16(s_addr + c0 / 2, w);
          if (c0 == 32) {
            tmem_wait_st();
            fence_before();
            bar_arrive(&sm.p_half[t]);
          }
        }
        const float2 total = split(add2(sum[0], sum[1]));
        l += total.x + total.y;
        tmem_wait_st();
        fence_before();
        bar_arrive(&sm.p_ready[t]);
      }
      if (n[t] > 0 && ok) {
        ok = __all_sync(0xffffffffu, bar_wait(&sm.o_full[t], 0, p, sm));
        fence_after();
      }
      if (SPLIT && ok && parts > 1 && t0 + t * tokens < sp.lq) {  // a part: binary32, joined below
        float* part = p.parts + (int64_t)(slot * 2 + t) * kPartFloats;
#pragma unroll
        for (int c = 0; c < kDim; c += 32) {
          uint32_t o[32];
          __syncwarp();
          if (n[t] > 0) {
            tmem_ld32(o_addr + c, o);
            tmem_wait_ld<32>(o);
#pragma unroll
            for (int k = 0; k < 32; k += 8)
              asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(part + row * kDim + c + k), KVQ_W4(o, k),
                           KVQ_W4(o, k + 4) : "memory");
          }
        }
        part[kTile * kDim + row] = m;
        part[kTile * kDim + kTile + row] = l;
      } else if (ok && (!SPLIT || parts == 1) && t0 + t * tokens < sp.lq) {
        const float inv = see > 0 ? 1.0f / l : 0.0f;
        const int64_t at = sp.q0 + token;
        const bool wide = ((reinterpret_cast<uintptr_t>(p.out) | (uintptr_t)(p.out_stride * 2)) & 31) == 0;
        uint32_t o[kDim];
        if (n[t] > 0) {
#pragma unroll
          for (int c = 0; c < kDim; c += 32) tmem_ld32(o_addr + c, o + c);
          tmem_wait_ld<kDim>(o);
        }
        if (mine) {
          uint16_t* out = p.out + at * p.out_stride + head * kDim;
#pragma unroll
          for (int c = 0; c < kDim; c += 16) {
            uint32_t y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              y[i] = see > 0 ? pack2<BF16>(__uint_as_float(o[c + 2 * i]) * inv, __uint_as_float(o[c + 2 * i + 1]) * inv) : 0u;
            if (wide) {  // whole 32-byte sectors
              asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(out + c), KVQ_W4(y, 0), KVQ_W4(y, 4)
                           : "memory");
            } else {
              *reinterpret_cast<uint4*>(out + c) = make_uint4(y[0], y[1], y[2], y[3]);
              *reinterpret_cast<uint4*>(out + c + 8) = make_uint4(y[4], y[5], y[6], y[7]);
            }
          }
        }
        if (p.lse && mine)
          p.lse[at * (p.H * p.r) + head] = see > 0 ? (m - kWeightExp + log2f(l)) * 0.6931471805599453f : -INFINITY;
      }
    }
  }
  fence_before();
  __syncthreads();
  if (SPLIT && parts > 1) {  // the last CTA of a split item joins its parts
    const int first_slot = slot - sm.part;
    if (threadIdx.x == 0) {
      uint32_t* ticket = p.tickets + first_slot;
      uint32_t n;
      asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(n) : "l"(ticket) : "memory");
      sm.last = n == (uint32_t)(parts - 1);
      if (sm.last) *ticket = 0u;  // ready for the next call
    }
    __syncthreads();
    if (sm.last && warp < 8) {  // the warps that have the registers for it
      const int t0 = sm.tile * 2 * tokens;
      for (int r0 = warp * 4; r0 < 2 * kTile; r0 += 32) join_rows<BF16>(p, sp, h, t0, tokens, first_slot, parts, r0);
      __syncwarp();
    }
  }
  // (parts of a split item: by the CTA that joined them)
  if (sm.spoiled && warp < 8 && (parts == 1 || (SPLIT && parts > 1 && sm.last))) {
    const int t0 = sm.tile * 2 * tokens;
#pragma unroll 1
    for (int row = warp; row < 2 * kTile; row += 8) row_by_row<BF16>(p, sm.span, h, t0, tokens, row);
  }
  if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static std::atomic<void*> fn{nullptr};
  void* f = fn.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      return nullptr;
    fn.store(f, std::memory_order_release);
  }
  return reinterpret_cast<EncodeFn>(f);
}

// Rows [tokens][heads][128] of 16 bits; boxes of 64 channels x box_heads x box_tokens.
bool make_map(EncodeFn fn, CUtensorMap* map, const void* p, int heads, int64_t rows, int64_t stride, int box_heads,
              int box_tokens, int dtype) {
  *map = CUtensorMap{};
  if (rows == 0) return true;  // never used
  const cuuint64_t dims[3] = {kDim, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {kDim * 2, (cuuint64_t)(rows > 1 ? stride : (int64_t)heads * kDim) * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens}, ones[3] = {1, 1, 1};
  return fn(map, dtype == KVQ_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
            const_cast<void*>(p), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool BF16, bool SPLIT>
cudaError_t launch(const PromptParams& p, int64_t ctas, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                   cudaStream_t stream) {
  constexpr int smem = (int)sizeof(Smem) + 1024;
  static std::atomic<bool> ready[64];  // per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(prompt_kernel<BF16, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev].store(true, std::memory_order_relaxed);
  }
  return launch_pdl(prompt_kernel<BF16, SPLIT>, dim3((unsigned)ctas), dim3(kThreads), smem, stream, p, q, k, v);
}

}  // namespace

size_t prompt_workspace_bytes() { return kPromptParts + sizeof(float) * kPromptSplit * 2 * kPartFloats; }


cudaError_t launch_prompt(const PromptParams& p, int dtype, cudaStream_t stream) {
  const EncodeFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const int tokens = kTile / p.r;
  CUtensorMap q, k, v;
  if (!make_map(fn, &q, p.q, p.H * p.r, p.n_q, p.q_stride, p.r, tokens, dtype) ||
      !make_map(fn, &k, p.k, p.H, p.n_kv, p.k_stride, 1, kTile, dtype) ||
      !make_map(fn, &v, p.v, p.H, p.n_kv, p.v_stride, 1, kTile, dtype))
    return cudaErrorInvalidValue;
  // pairs of tiles: one per 2 * tokens tokens of a sequence, at least one for a sequence with a token
  const int64_t ctas = (p.n_q / (2 * tokens) + std::min(p.n_q, p.n_seqs)) * (int64_t)p.H;
  if (ctas >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  // Few query rows over many keys: one item per CTA would leave SMs idle (8 kv heads, 32 queries over
  // 32768 keys: 317 us whole, 78 split; 128 over 65536: 675 and 146). The items are counted on the
  // device; here only what they cannot exceed is known.
  if (ctas <= kPromptSplit && p.n_seqs <= 32 && p.n_kv >= 2 * kPartTiles * kTile)
    return dtype == KVQ_BF16 ? launch<true, true>(p, kPromptSplit, q, k, v, stream)
                             : launch<false, true>(p, kPromptSplit, q, k, v, stream);
  return dtype == KVQ_BF16 ? launch<true, false>(p, ctas, q, k, v, stream) : launch<false, false>(p, ctas, q, k, v, stream);
}

}  // namespace kvq
