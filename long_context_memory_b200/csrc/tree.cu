// A decode step over a tree of drafted tokens: the plan (ancestor masks and positions), the
// attention of the drafts over [selected documents' pooled rows; local cache; the drafts they
// see], and the append of the accepted drafts to the local cache.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "tree_notes.h"

namespace msa {

namespace {

constexpr int kMaxDrafts = 256;
constexpr int kMaskWords = kMaxDrafts / 32;
constexpr float kLog2e = 1.4426950408889634f;

// ---------------------------------------------------------------------------
// plan: one CTA per query, one thread per draft.  Pointer doubling: after round r a draft's mask
// holds its 2^r nearest ancestors (itself included) and jump[] the next one up, so a tree of
// depth d takes ceil(log2 d) rounds of shared-memory reads instead of a chain of d dependent ones.
// Bound by latency (launch, two dependent loads, the rounds): 1.9 us for one tree of 16, 2.2 us for 32
// trees of 127.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kMaxDrafts) tree_plan_kernel(const int32_t* __restrict__ parents,
                                                               const int32_t* __restrict__ n_draft,
                                                               const int32_t* __restrict__ loc_len, int M, int W,
                                                               int pos_offset, int32_t* __restrict__ mask,
                                                               int32_t* __restrict__ positions) {
  __shared__ uint32_t see[kMaxDrafts][kMaskWords + 1];
  __shared__ int jump[kMaxDrafts], depth[kMaxDrafts];
  pdl_enter();
  const int b = blockIdx.x, t = threadIdx.x;
  const int n = n_draft ? max(0, min(n_draft[b], M)) : M;
  uint32_t m[kMaskWords];
#pragma unroll
  for (int w = 0; w < kMaskWords; ++w) m[w] = (t >> 5) == w ? 1u << (t & 31) : 0u;
  int up = -1, d = 0;
  if (t < n) {
    up = parents[(size_t)b * M + t];
    if (up < -1 || up >= t) {
      raise_dev_error(kDevErrBadIndex);
      up = -1;
    }
    d = up >= 0;
  }
  while (__syncthreads_or(up >= 0)) {
#pragma unroll
    for (int w = 0; w < kMaskWords; ++w) see[t][w] = m[w];
    jump[t] = up;
    depth[t] = d;
    __syncthreads();
    if (up >= 0) {  // depth counts the steps to jump[]'s end of the chain so far
#pragma unroll
      for (int w = 0; w < kMaskWords; ++w) m[w] |= see[up][w];
      d += depth[up];
      up = jump[up];
    }
    __syncthreads();
  }
  if (t < M) {
    int32_t* row = mask + ((size_t)b * M + t) * W;
#pragma unroll
    for (int w = 0; w < kMaskWords; ++w)
      if (w < W) row[w] = t < n ? (int32_t)m[w] : 0;
    positions[(size_t)b * M + t] = pos_offset + loc_len[b] + (t < n ? d : 0);
  }
}

// ---------------------------------------------------------------------------
// commit: a warp per (query, accepted draft) copies its K and V rows, all loads of 2 KB each in flight
// before the first store.  Bound by latency: 1.5 us for 5 drafts, 2.5 us for 64 queries of up to 17.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(128) tree_commit_kernel(const uint4* __restrict__ K_draft,
                                                          const uint4* __restrict__ V_draft,
                                                          const int32_t* __restrict__ path,
                                                          const int32_t* __restrict__ n_path, int B, int M, int A,
                                                          int row_vec, uint4* __restrict__ K_loc,
                                                          uint4* __restrict__ V_loc, const int32_t* __restrict__ loc_len,
                                                          int t_loc_max, int32_t* __restrict__ new_len) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int b = (int)(item / A), i = (int)(item - (int64_t)b * A);
  if (b >= B) return;
  const int L = loc_len[b], n = max(0, min(n_path[b], A));
  const int src = path[(size_t)b * A + i];
  if (i == 0 && lane == 0) new_len[b] = (int)min((int64_t)L + n, (int64_t)max(L, t_loc_max));
  if (i >= n) return;
  const int64_t slot = (int64_t)L + i;
  if (src < 0 || src >= M || slot < 0 || slot >= t_loc_max) {
    if (lane == 0) raise_dev_error(kDevErrBadIndex);
    return;
  }
  const size_t from = ((size_t)b * M + src) * row_vec, to = ((size_t)b * t_loc_max + slot) * row_vec;
  for (int v = lane; v < row_vec; v += 128) {
    uint4 k[4], w[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (v + 32 * u < row_vec) {
        k[u] = K_draft[from + v + 32 * u];
        w[u] = V_draft[from + v + 32 * u];
      }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (v + 32 * u < row_vec) {
        K_loc[to + v + 32 * u] = k[u];
        V_loc[to + v + 32 * u] = w[u];
      }
  }
}

// ---------------------------------------------------------------------------
// attention
//
// The rows that share a KV head (drafts x GQA group) fill the 128 rows of tcgen05 tiles: a row tile
// is TT = 128 / G drafts with their G heads, a CTA takes NT row tiles at once (two when one does not
// hold all drafts), so K and V cross HBM once per 256 rows.  Two streams of scores, weights and
// outputs run beside each other, so that the tensor cores and one stream's softmax overlap the
// other's softmax: with two row tiles a stream is a row tile (each key tile goes through both); with
// one, the streams take the key tiles in turn, each with a maximum, sum and output of its own,
// joined at the item's end.  A stream's step costs
//   S = Q K^T   (tcgen05, operands in shared memory, fp32 scores in tensor memory),
//   P = exp2(S c - m)   (one thread per row, scores and weights in registers),
//   O += P V    (tcgen05, P bf16 in tensor memory over S, V in shared memory, O in tensor memory).
// P is rounded to bf16 because the tensor cores take bf16; its sum l is taken before the rounding,
// in fp32.  The reference maximum m of a row moves only when the running maximum passes it by
// 2^kSlack (O is then rescaled in tensor memory; weights stay below 2^kSlack otherwise, far
// inside bf16's and fp32's range), so that a tile normally touches O in the MMA alone.
//
// Keys of a query: its documents' pooled rows one after the other, the local rows, the drafts, each
// in tiles of 128.  Work is cut evenly: all tiles of all (query, row block) items stand in one line,
// the same for each KV head; the CTAs form groups of n_kv, a CTA per head, and group c of N takes
// tiles c W / N .. (c + 1) W / N (N = SMs / n_kv, or W where there are fewer tiles).  So ragged
// batches and single long queries fill the GPU alike, a group reads whole cache rows at about the
// same time, and few items are cut: one line over all heads left 4 SMs more at work, but cut nearly
// every head of a single query in one place more (16 drafts over the 1M-token memory 22 us against 19;
// 8 queries of one token over 32K local tokens 190 against 184).  The at most two items that a CTA
// shares with its neighbours leave partial results and a note for tree_combine_kernel, which merges
// them.
//
// A tile's rows arrive by TMA boxes.  A box costs the TMA unit about 55 cycles and 2.3 per row of
// 128 bytes (measured), so a document's run of rows is covered by at most two boxes, of the largest
// power of two that is not longer, the second one moved back to end with the run (the rows where
// they overlap arrive twice, the same bytes); a box may start at any row of the tile, since the
// 128-byte swizzle goes by the address.  Values are copied only where some draft sees them, into a
// ring whose other rows are zeros: whatever stands in the rows behind a sequence, and in drafts that
// nobody sees, never reaches a product.  (A key too many does no harm: its score is replaced.)
//
// Warps: 2 x 4 softmax warps (a stream each, a thread per row), one producer (item headers, document
// tables, TMA), one MMA issuer.  One CTA per SM (its ring fills the shared memory).
//
// Measured (heads of 128, 32 query and 8 KV heads): 16 drafts of one query over 16 documents and 4K
// local tokens 20 us, bound by the chain of a CTA's two to three tiles and the merge; 32 queries of 32
// drafts over 16 documents and 8K tokens (1.17 GB) 246-265 us, 4.4-4.8 TB/s, on inputs that were not used just
// before, 204-220 us (5.3-5.7) on such that were; 32 queries of 64 drafts over 8K local tokens 295-298 us, 930 TFLOP/s.
// Heads of 64, 7 queries of up to 127 drafts over up to 20K tokens: 59-81 us on different boxes, bound by the
// softmax threads: a key tile against two row tiles takes 3,100 cycles, in which the exponentials of its
// 256 x 128 scores are 2,048 (16 a cycle and SM, measured).  Of a stream's step its weights take 1,790 cycles beside
// the other stream's, the maximum 400, the wait for the next scores 690.  (A polynomial on the FMA pipes for a
// fifth to a third of the exponentials made it slower.)
// ---------------------------------------------------------------------------
constexpr int kTile = 128;        // keys per tile, rows per row tile
constexpr int kMaxRing = 6;
// Queries whose documents' rows every CTA counts itself; beyond, a kernel of their own counts them once.
// 8 drafts over 256 local tokens, 32/8 heads of 128, counted by every CTA against by the kernel: 4 queries of
// 16 documents 18.1 against 19.0 us, 8 of 2 21.4 against 22.5, 8 of 16 23.8 against 23.9, 8 of 64 33.5
// against 31.0, 16 of 1 27.6 against 26.4, 16 of 16 32.4 against 28.7, 32 of 16 49.7 against 40.1.
constexpr int kSmallB = 8;
constexpr float kSlack = 8.f;
constexpr int kTmemCols = 512;    // scores 2 x 128, outputs 2 x 128

constexpr int kTailRows[4] = {1, 8, 32, 128};

struct TreeMaps {
  CUtensorMap q;
  CUtensorMap bar[2][7];           // [K, V] pooled rows: boxes of 1, 2, 4 .. 64 rows
  CUtensorMap k_loc, k_draft;      // 128 rows
  CUtensorMap v_loc[4], v_draft[2];  // 1, 8, 32 and 128 rows; 1 and 8
};

struct TreeP {
  const int32_t *mask, *n_draft, *loc_len, *chunk_off, *topk_idx;
  __nv_bfloat16* out;
  // [2] per item (few items) or per CTA (many): query (-1: nothing to merge), first draft, KV head,
  // drafts | first and last group, first part's slot
  int4* merges;
  int by_item;
  int32_t* sel;      // [B] pooled rows of each query's documents (B > kSmallB)
  float* part_o;     // [2 N][D / 4][NT * 128][4] unnormalised (a warp's rows side by side)
  float* part_ml;    // [2 N][NT * 128][2] reference maximum, sum
  int B, M, W, n_q, n_kv, G, TT, n_rb, t_loc_max, n_docs, n_chunks, k, ring, pad, groups;
  float scale_log2;
};

enum { kHb = 0, kHt0, kHhk, kHsel, kHL, kHn, kHTc, kHTl, kHlo, kHhi, kHslot, kHWords = 16 };

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ int doc_rows(const TreeP& p, int doc) {
  return max(0, min(p.chunk_off[doc + 1] - p.chunk_off[doc], p.n_chunks));
}
__device__ __forceinline__ int drafts_of(const TreeP& p, int b) {
  return p.n_draft ? max(0, min(p.n_draft[b], p.M)) : p.M;
}
__device__ __forceinline__ int local_of(const TreeP& p, int b) { return max(0, min(p.loc_len[b], p.t_loc_max)); }
__device__ __forceinline__ int tiles_of(int sel, int L, int n) {
  return (sel + kTile - 1) / kTile + (L + kTile - 1) / kTile + (n + kTile - 1) / kTile;
}
// row blocks of a query that hold a draft in use
template <int NT>
__device__ __forceinline__ int blocks_of(const TreeP& p, int n) {
  return (n + NT * p.TT - 1) / (NT * p.TT);
}

// scores that the row does not see become -inf
__device__ __forceinline__ void hide(float (&s)[32], uint32_t see) {
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (!(see >> e & 1)) s[e] = -INFINITY;
}
__device__ __forceinline__ float max_of(const float (&s)[32], float m0) {
  float m[4] = {fmaxf(s[0], m0), s[1], s[2], s[3]};
#pragma unroll
  for (int e = 4; e < 32; ++e) m[e & 3] = fmaxf(m[e & 3], s[e]);
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// Largest of the tile's 128 scores of this row (quarters of 32 keys; two loads in flight).
template <bool MASKED>
__device__ __forceinline__ float row_max(uint32_t addr, const uint32_t (&see)[4]) {
  float sa[32], sb[32];
  float m = -INFINITY;
#pragma unroll
  for (int q = 0; q < 4; q += 2) {
    tmem_ld32(addr + 32 * q, sa);
    tmem_ld32(addr + 32 * q + 32, sb);
    tmem_ld_wait_for(sa);
    tmem_ld_wait_for(sb);
    if (MASKED) {
      hide(sa, see[q]);
      hide(sb, see[q + 1]);
    }
    m = max_of(sa, m);
    m = max_of(sb, m);
  }
  return m;
}

// The scores again, a quarter at a time with the next one's load in flight: weights 2^(s c + neg) as
// bf16 pairs to columns `to` .. (their own place, or those of quarters already read); returns their
// fp32 sum.
template <bool MASKED>
__device__ __forceinline__ float row_weights(uint32_t addr, uint32_t to, const uint32_t (&see)[4], float c, float neg,
                                             uint64_t* read_bar) {
  float sa[32], sb[32];
  const uint64_t c2 = pack_f32x2(c, c), neg2 = pack_f32x2(neg, neg);
  uint64_t sum[2] = {0, 0};  // two pairs of fp32 zeros
  tmem_ld32(addr, sa);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float(&cur)[32] = q & 1 ? sb : sa;
    tmem_ld_wait_for(cur);
    if (q < 3) tmem_ld32(addr + 32 * (q + 1), q & 1 ? sa : sb);
    if (q == 3 && read_bar) {  // the scores are read: their place is free
      tc_fence_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(read_bar);
    }
    if (MASKED) hide(cur, see[q]);
    uint32_t u[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float2 y = unpack_f32x2(fma_f32x2(pack_f32x2(cur[2 * e], cur[2 * e + 1]), c2, neg2));
      const float a = ex2(y.x), z = ex2(y.y);
      sum[e & 1] = add_f32x2(sum[e & 1], pack_f32x2(a, z));
      u[e] = pack_bf16x2(a, z);
    }
    tmem_st16(to + 16 * q, u);
  }
  const float2 both = unpack_f32x2(add_f32x2(sum[0], sum[1]));
  return both.x + both.y;
}

// each query's pooled rows (large batches only): a warp per query
__global__ void __launch_bounds__(256) tree_select_kernel(const int32_t* __restrict__ topk_idx,
                                                          const int32_t* __restrict__ chunk_off, int B, int k,
                                                          int n_docs, int n_chunks, int32_t* __restrict__ sel) {
  pdl_enter();
  const int b = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (b >= B) return;
  int g = 0;
  for (int r = lane; r < k; r += 32) {
    const int doc = topk_idx[(size_t)b * k + r];
    if (doc >= 0 && doc < n_docs) g += max(0, min(chunk_off[doc + 1] - chunk_off[doc], n_chunks));
    else raise_dev_error(kDevErrBadIndex);  // (the attention lists only documents of queries with tiles)
  }
  g = __reduce_add_sync(0xffffffffu, g);
  if (lane == 0) sel[b] = g;
}

// floor(a b / c) for a b < 2^63, with 32-bit arithmetic where it fits
__device__ __forceinline__ long long muldiv(long long a, int b, int c) {
  const long long ab = a * b;
  return ab >> 32 ? ab / c : (long long)((uint32_t)ab / (uint32_t)c);
}
__device__ __forceinline__ int divide(long long a, long long b) {  // floor(a / b), the result an int
  return (a | b) >> 32 ? (int)(a / b) : (int)((uint32_t)a / (uint32_t)b);
}

// boxes of one size that cover a run of n <= 128 rows, the last one moved back to end with it
struct Cover {
  int size, count, level;
};
__device__ __forceinline__ Cover cover_doc(int n) {  // sizes 1, 2, 4 .. 64: at most two boxes
  Cover c;
  c.level = min(6, 31 - __clz(max(n, 1)));
  c.size = 1 << c.level;
  c.count = n <= 0 ? 0 : n == c.size ? 1 : 2;
  return c;
}
__device__ __forceinline__ Cover cover_tail(int n) {  // sizes 1, 8, 32, 128
  Cover c;
  c.level = n >= 128 ? 3 : n >= 32 ? 2 : n >= 8 ? 1 : 0;
  c.size = c.level == 3 ? 128 : c.level == 2 ? 32 : c.level == 1 ? 8 : 1;
  c.count = (n + c.size - 1) / c.size;
  return c;
}

__device__ __forceinline__ uint32_t first_rows(int n) { return n >= 8 ? 0xFFu : n > 0 ? (1u << n) - 1 : 0u; }

// The rows of a value tile that no box brings (lane i < 16 has the bits of the rows 8 i .. that one
// does) still hold an older tile's, maybe of a query whose values are not finite: zeros.  Called by
// the producer warp for the last tile of a sequence; out of line, off the other tiles' path.
template <int DB>
__device__ __noinline__ void clear_rest(uint8_t* dst, uint32_t bits) {
  const int lane = threadIdx.x & 31;
  for (int g = 0; g < kTile / 8; ++g) {
    const uint32_t m = __shfl_sync(0xffffffffu, bits, g);
    if (m == 0xFFu) continue;
#pragma unroll
    for (int u = 0; u < 2; ++u) {  // four rows at once, eight lanes a row of 128 bytes
      const int r = u * 4 + (lane >> 3);
      if (!(m >> r & 1))
#pragma unroll
        for (int d = 0; d < DB; ++d)
          *reinterpret_cast<uint4*>(dst + d * (kTile * 128) + (g * 8 + r) * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
}

template <int D, int NT>
__global__ void __launch_bounds__(320, 1) tree_attend_kernel(const __grid_constant__ TreeMaps maps,
                                                                       const __grid_constant__ TreeP p) {
  constexpr int DB = D / 64;            // 64-element blocks of a head
  constexpr int kBlk = kTile * 128;     // bytes of one block of a 128-row tile
  constexpr int kTB = DB * kBlk;        // bytes of a tile
  constexpr int kThreads = 320;
  constexpr int kSoftWarps = 8;
  // Tensor memory: scores of stream s at 128 s, its output at 256 + 128 s.  A head of 64 leaves room
  // behind the output for the weights, so that the next scores need not wait until the products with
  // the weights are done; a head of 128 has the weights over the scores.
  constexpr bool kApart = D == 64;
  // (declared with the alignment that is sure behind the statically sized part; a stricter one would
  // be taken on trust and fold the rounding below away)
  extern __shared__ __align__(16) uint8_t sm_raw[];
  __shared__ uint64_t kfull[kMaxRing], kempty[kMaxRing], vfull[kMaxRing], vempty[kMaxRing];
  __shared__ uint64_t qfull, qempty, sfull[2], sfree[2], pready[2], pvdone[2], ofree[2], joined, taken, hfull[2], hempty[2], drained;
  __shared__ float2 state[NT == 1 ? kTile : 1];  // one row tile: stream 1's reference maximum and sum of each row
  __shared__ int hdr[2][kHWords];
  __shared__ int q_sel[kSmallB], q_loc[kSmallB], q_n[kSmallB];  // small batches: pooled rows, local rows, drafts
  __shared__ long long warp_sum[kThreads / 32];
  __shared__ long long first_base;
  __shared__ int first_b;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;

  uint8_t* qs = sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u);  // [NT] row tiles (swizzle atoms: 1 KB aligned)
  uint8_t* ks = qs + NT * kTB;            // [ring] key tiles
  uint8_t* vs = ks + p.ring * kTB;        // [ring] value tiles
  int* tab = reinterpret_cast<int*>(vs + p.ring * kTB);  // the query's documents: [k + 1] first key, [k] first row

  if (qs - sm_raw > p.pad) {  // the tiles would not fit where the launch put them
    if (threadIdx.x == 0) raise_dev_error(kDevErrBadIndex);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < p.ring; ++i) {
      mbar_init(&kfull[i], 1);
      mbar_init(&kempty[i], 1);
      mbar_init(&vfull[i], 1);
      mbar_init(&vempty[i], 1);
    }
    mbar_init(&qfull, 1);
    mbar_init(&qempty, 1);
    mbar_init(&drained, 1);
    mbar_init(&joined, 4);
    mbar_init(&taken, 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&sfree[i], 4);
      mbar_init(&pready[i], 4);
      mbar_init(&pvdone[i], 1);
      mbar_init(&ofree[i], 4);
      mbar_init(&hfull[i], 1);
      mbar_init(&hempty[i], kSoftWarps + 1);
    }
    abort_flag = 0;
    first_b = -1;
    fence_mbar_init();
  }
  if (warp == kSoftWarps + 1) {
    tmem_alloc(&tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  for (int i = tid; i < kSmallB; i += kThreads) q_sel[i] = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_enter();

  // ---- the line of tiles: every CTA counts it, for small batches in shared memory; meanwhile the
  // softmax warps clear the value ring (a tile need not fill its slot) ----
  const bool small = p.B <= kSmallB;
  if (warp < kSoftWarps) {
    for (int i = tid; i < p.ring * (kTB / 16); i += 32 * kSoftWarps) reinterpret_cast<uint4*>(vs)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  } else if (small) {
    const int u0 = tid - 32 * kSoftWarps;  // 64 threads
    if (u0 < p.B) {
      q_n[u0] = drafts_of(p, u0);
      q_loc[u0] = local_of(p, u0);
    }
    const int pairs = p.B * p.k;
    for (int i0 = u0; i0 < pairs; i0 += 8 * 64) {  // eight documents of a thread in flight
      int rows[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = i0 + u * 64;
        rows[u] = -1;
        if (i < pairs) {
          const int doc = p.topk_idx[i];
          const bool known = doc >= 0 && doc < p.n_docs;
          if (known) rows[u] = doc_rows(p, doc);
          else raise_dev_error(kDevErrBadIndex);
          if (p.B == 1) {  // the only query's table
            tab[i] = max(rows[u], 0);
            tab[p.k + 1 + i] = known ? p.chunk_off[doc] : 0;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (rows[u] > 0) atomicAdd(&q_sel[p.B == 1 ? 0 : (i0 + u * 64) / p.k], rows[u]);
    }
  }
  __syncthreads();
  auto query = [&](int b, int& sel, int& L, int& n) {
    n = small ? q_n[b] : drafts_of(p, b);
    L = small ? q_loc[b] : local_of(p, b);
    sel = small ? q_sel[b] : p.k ? p.sel[b] : 0;
  };
  auto cost_of = [&](int b) -> long long {
    int sel, L, n;
    query(b, sel, L, n);
    return (long long)blocks_of<NT>(p, n) * tiles_of(sel, L, n);
  };
  // group c of the n_act with work begins at tile floor(c total / n_act)
  const int group = blockIdx.x / p.n_kv, hk = blockIdx.x - group * p.n_kv;
  long long total = 0, w_begin = 0, w_end = 0;
  int n_act = 1;
  auto begin_of = [&](int c) { return min(total, muldiv(total, c, n_act)); };
  auto cut = [&] {
    n_act = (int)max(1ll, min((long long)p.groups, total));
    w_begin = begin_of(group);
    w_end = begin_of(group + 1);
  };
  if (p.B == 1) {  // (only the producer needs it)
    if (warp == kSoftWarps) {
      total = cost_of(0);
      cut();
    }
  } else {
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += cost_of(b);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    long long base = incl - mine;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) base += warp_sum[w];
      total += warp_sum[w];
    }
    cut();
    for (int b = b0; b < b1 && w_begin < w_end; ++b) {
      const long long c = cost_of(b);
      if (base <= w_begin && w_begin < base + c) {
        first_b = b;
        first_base = base;
      }
      base += c;
    }
    __syncthreads();
  }

  if (warp == kSoftWarps) {
    // =======================================================================
    // producer
    // =======================================================================
    uint32_t x = 0;     // tiles loaded
    int k_issued = 0;   // of their key tiles
    int st = 0, ph = 1;  // ring slot of tile x; parity of the phase in which that slot was emptied last
    int n_items = 0;
    bool ok = true;
    long long w = w_begin;
    long long bbase = p.B == 1 ? 0 : first_base;
    int b = p.B == 1 ? 0 : first_b;
    bool fresh = true, listed = false;  // b is new; its documents are in the table
    int L = 0, n = 0, sel = 0, T = 0;
    int *first_key = tab, *first_row = tab + p.k + 1;
    if (lane == 0 && !p.by_item) p.merges[2 * blockIdx.x].x = -1;
    while (ok) {
      const int hb = n_items & 1;
      if (n_items >= 2 && !warp_wait_short(&hempty[hb], ((n_items >> 1) - 1) & 1, &abort_flag)) {
        ok = false;
        break;
      }
      int* h = hdr[hb];
      if (w >= w_end) {
        if (lane == 0) {
          h[kHb] = -1;
          mbar_arrive(&hfull[hb]);
        }
        break;
      }
      for (;;) {
        if (fresh) {
          query(b, sel, L, n);
          T = tiles_of(sel, L, n);
          fresh = listed = false;
        }
        const long long c = (long long)blocks_of<NT>(p, n) * T;
        if (w < bbase + c) break;
        bbase += c;
        ++b;
        fresh = true;
      }
      const int rb = divide(w - bbase, T), lo = (int)(w - bbase - (long long)rb * T);
      const int hi = (int)min((long long)T, lo + (w_end - w));
      const int t0 = rb * NT * p.TT;
      const int Tc = (sel + kTile - 1) / kTile, Tl = (L + kTile - 1) / kTile;
      if (lane == 0) {
        h[kHb] = b;
        h[kHt0] = t0;
        h[kHhk] = hk;
        h[kHsel] = sel;
        h[kHL] = L;
        h[kHn] = n;
        h[kHTc] = Tc;
        h[kHTl] = Tl;
        h[kHlo] = lo;
        h[kHhi] = hi;
        // whole items are written out; a shared one leaves its part: slot 0 of the CTA's first item, 1 of its last
        h[kHslot] = (lo == 0 && hi == T) ? -1 : 2 * (int)blockIdx.x + (n_items > 0);
        mbar_arrive(&hfull[hb]);
      }
      // queries: NT row tiles of TT drafts x G heads
      if (n_items >= 1 && !warp_wait_short(&qempty, (n_items - 1) & 1, &abort_flag)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(&qfull, NT * DB * p.G * p.TT * 128);
        for (int i = 0; i < NT; ++i)
          for (int d = 0; d < DB; ++d)
            tma_load_4d(qs + i * kTB + d * kBlk, &maps.q, &qfull, d * 64, hk * p.G, t0 + i * p.TT, b);
      }
      const bool first = n_items == 0;
      ++n_items;
      bool k_ahead = false;  // the tile's keys have been asked for
      for (int t = lo; t < hi && ok; ++t, ++x) {
        const int c0 = t * kTile, j0 = (t - Tc) * kTile, d0 = (t - Tc - Tl) * kTile;
        const int kind = t < Tc ? 0 : t < Tc + Tl ? 1 : 2;  // pooled rows, local rows, drafts
        int rows, k_rows;   // rows of the tile; rows that its key and value boxes bring
        int v_rows;
        int doc0 = 0;       // kind 0: the first document with keys in the tile
        uint32_t bits = 0;  // kind 2, lane < 16: drafts d0 + 8 lane .. that some draft of the query sees
        if (kind == 0) {
          if (!listed) {  // the query's documents: first key (a running sum) and first pooled row of each
            const int each = (p.k + 31) / 32;
            int sum = 0;
            __syncwarp();
            for (int q = 0; q < each; ++q) {
              const int r = lane * each + q;
              if (r < p.k && p.B == 1) {
                sum += first_key[r];
              } else if (r < p.k) {
                const int doc = p.topk_idx[(size_t)b * p.k + r];
                int n_rows = 0, row0 = 0;
                if (doc >= 0 && doc < p.n_docs) {
                  n_rows = doc_rows(p, doc);
                  row0 = p.chunk_off[doc];
                } else {
                  raise_dev_error(kDevErrBadIndex);
                }
                first_key[r] = n_rows;
                first_row[r] = row0;
                sum += n_rows;
              }
            }
            int in = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const int v = __shfl_up_sync(0xffffffffu, in, o);
              if (lane >= o) in += v;
            }
            int run = in - sum;
            for (int q = 0; q < each; ++q) {
              const int r = lane * each + q;
              if (r < p.k) {
                const int n_rows = first_key[r];
                first_key[r] = run;
                run += n_rows;
              }
            }
            if (lane == 0) first_key[p.k] = sel;
            listed = true;
            __syncwarp();
          }
          rows = min(kTile, sel - c0);
          int z = p.k - 1;
          while (doc0 < z) {
            const int mid = (doc0 + z + 1) >> 1;
            if (first_key[mid] <= c0) doc0 = mid; else z = mid - 1;
          }
          int boxed = 0;
          for (int r = doc0 + lane; r < p.k && first_key[r] < c0 + rows; r += 32) {
            const Cover c = cover_doc(min(first_key[r + 1], c0 + rows) - max(first_key[r], c0));
            boxed += c.size * c.count;
          }
          k_rows = v_rows = __reduce_add_sync(0xffffffffu, boxed);
        } else if (kind == 1) {
          rows = min(kTile, L - j0);
          const Cover c = cover_tail(rows);
          k_rows = kTile;
          v_rows = c.size * c.count;
        } else {
          uint32_t seen[4] = {0, 0, 0, 0};
          for (int r = lane; r < n; r += 32) {
            const int32_t* mk = p.mask + ((size_t)b * p.M + r) * p.W + d0 / 32;
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (d0 / 32 + q < p.W) seen[q] |= (uint32_t)mk[q];
          }
          rows = 0;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            seen[q] = __reduce_or_sync(0xffffffffu, seen[q]);
            const int left = n - d0 - 32 * q;
            if (left < 32) seen[q] &= left > 0 ? (1u << left) - 1 : 0u;
            bits |= (lane >> 2) == q ? seen[q] >> (8 * (lane & 3)) & 0xFFu : 0u;
            rows += __popc(seen[q]);
          }
          k_rows = kTile;
          v_rows = rows;
        }
        const bool k_there = k_ahead;
        // Heads of 128 have a ring of two or three tiles: the next tile's keys, where they are local rows,
        // go before this one's values, whose place is free later (32 queries of 32 drafts over 8K tokens
        // 253 us against 262 on inputs that were not used just before, 204 against 207 on two taken in
        // turns; heads of 64, with six tiles, gain nothing that stands out of their spread).
        k_ahead = D == 128 && t + 1 < hi && t + 1 >= Tc && t + 1 < Tc + Tl;
#pragma unroll 1
        for (int kv = k_there ? 1 : 0; kv < 2; ++kv) {
          if (kv && k_ahead) {
            const int sn = st + 1 == p.ring ? 0 : st + 1, pn = sn == 0 ? ph ^ 1 : ph;
            if (x + 1 >= (uint32_t)p.ring && !warp_wait_short(kempty + sn, pn, &abort_flag)) {
              ok = false;
              break;
            }
            if (lane == 0) mbar_arrive_expect_tx(kfull + sn, kTile * D * 2);
            __syncwarp();
            if (lane < DB)
              tma_load_4d(ks + sn * kTB + lane * kBlk, &maps.k_loc, kfull + sn, lane * 64, hk, j0 + kTile, b);
            ++k_issued;
          }
          uint64_t* fullb = (kv ? vfull : kfull) + st;
          uint8_t* dst = (kv ? vs : ks) + st * kTB;
          if (x >= (uint32_t)p.ring && !warp_wait_short((kv ? vempty : kempty) + st, ph, &abort_flag)) {
            ok = false;
            break;
          }
          // a slot's first tile finds the ring cleared
          if (kv && rows < kTile && x >= (uint32_t)p.ring) clear_rest<DB>(dst, kind == 2 ? bits : first_rows(rows - 8 * lane));
          if (lane == 0) mbar_arrive_expect_tx(fullb, (kv ? v_rows : k_rows) * D * 2);
          __syncwarp();
          if (!kv) ++k_issued;
          if (kind == 0) {  // a lane per (document, box, block of 64 elements)
            constexpr int kPer = 2 * DB;
            for (int r0 = doc0; r0 < p.k && first_key[r0] < c0 + rows; r0 += 32 / kPer) {
              const int r = r0 + lane / kPer, i = lane % kPer / DB, d = lane % DB;
              if (r < p.k && first_key[r] < c0 + rows) {
                const int a = max(first_key[r], c0), run = min(first_key[r + 1], c0 + rows) - a;
                const Cover c = cover_doc(run);
                if (i < c.count) {
                  const int o = i ? run - c.size : 0;
                  tma_load_3d(dst + d * kBlk + (a - c0 + o) * 128, &maps.bar[kv][c.level], fullb, d * 64, hk,
                              first_row[r] + (a - first_key[r]) + o);
                }
              }
            }
          } else if (kv == 0) {
            if (lane < DB)
              tma_load_4d(dst + lane * kBlk, kind == 1 ? &maps.k_loc : &maps.k_draft, fullb, lane * 64, hk,
                          kind == 1 ? j0 : d0, b);
          } else if (kind == 1) {
            const Cover c = cover_tail(rows);
            if (lane < c.count * DB) {
              const int i = lane / DB, d = lane % DB, o = min(i * c.size, rows - c.size);
              tma_load_4d(dst + d * kBlk + o * 128, &maps.v_loc[c.level], fullb, d * 64, hk, j0 + o, b);
            }
          } else {
            const bool whole = bits == 0xFFu;
            if (whole)
              for (int d = 0; d < DB; ++d)
                tma_load_4d(dst + d * kBlk + lane * 1024, &maps.v_draft[1], fullb, d * 64, hk, d0 + 8 * lane, b);
            if (__any_sync(0xffffffffu, bits != 0 && !whole)) {  // groups of 8 with holes, or the last one: row by row
              for (int r = 0; r < 8; ++r)
                if (!whole && (bits >> r & 1))
                  for (int d = 0; d < DB; ++d)
                    tma_load_4d(dst + d * kBlk + lane * 1024 + r * 128, &maps.v_draft[0], fullb, d * 64, hk,
                                d0 + 8 * lane + r, b);
            }
          }
          __syncwarp();
        }
        if (!ok) break;  // this tile's values were not asked for: x counts those that were
        if (++st == p.ring) {
          st = 0;
          ph ^= 1;
        }
        if (t == lo && lane == 0 && (p.by_item ? lo == 0 : first && lo > 0)) {
          // the note for the merge: of a cut item by the CTA that begins it (per item), or by the
          // next group's (per CTA)
          const long long w0 = w - lo;  // tile w is in the group floor(((w + 1) N - 1) / W)
          const int ca = p.by_item ? group : divide((w0 + 1) * n_act - 1, total);
          const int cz = divide((w0 + T) * n_act - 1, total);
          const size_t at = p.by_item ? (size_t)(b * p.n_rb + rb) * p.n_kv + hk : (size_t)blockIdx.x;
          if (p.by_item || ca + 1 == group) {
            p.merges[2 * at + 1] = make_int4(ca, cz, 2 * (ca * p.n_kv + hk) + (begin_of(ca) == w0 ? 0 : 1), 0);
            p.merges[2 * at] = make_int4(ca == cz ? -1 : b, t0, hk, n);
          }
        }
      }
      w += hi - lo;
    }
    if (abort_flag && lane == 0) {  // the copies still in flight land before the CTA exits
      mbar_drain_ring(kfull, p.ring, k_issued - p.ring, k_issued);
      mbar_drain_ring(vfull, p.ring, (int)x - p.ring, (int)x);
      if (n_items) mbar_drain_ring(&qfull, 1, n_items - 1, n_items);
    }
    __syncwarp();
  } else if (warp == kSoftWarps + 1) {
    // =======================================================================
    // MMA issuer
    // =======================================================================
    {
      constexpr uint32_t idesc_s = umma_idesc_bf16(128, 128);
      constexpr uint32_t idesc_o = umma_idesc_bf16(128, D) | kIdescBMnMajor;
      const uint64_t qd = umma_desc_k_sw128(smem_u32(qs)), kd = umma_desc_k_sw128(smem_u32(ks)),
                     vd = umma_desc_mn_sw128(smem_u32(vs), kBlk);
      // ring places of the next key tile to multiply with Q and of the next value tile (slot, parity)
      int ks_st = 0, ks_ph = 0, vs_st = 0, vs_ph = 0;
      uint32_t x = 0;
      bool ok = true;
      auto scores = [&](int i, uint32_t xx) {  // S of row tile i and key tile xx
        if (i == 0 && !warp_wait_short(&kfull[ks_st], ks_ph, &abort_flag)) return false;
        tc_fence_after();
        const uint32_t slot = NT == 1 ? (xx & 1) : i;
        const uint64_t a = qd + (uint64_t)(i * kTB / 16), k = kd + (uint64_t)(ks_st * (kTB / 16));
        if (elect_one()) {
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            const int o = ((s >> 2) * kBlk + (s & 3) * 32) / 16;
            umma_bf16(tmem + slot * 128, a + o, k + o, idesc_s, s > 0);
          }
          umma_commit(&sfull[slot]);
          if (i == NT - 1) umma_commit(&kempty[ks_st]);
        }
        __syncwarp();
        if (i == NT - 1) {
          if (++ks_st == p.ring) {
            ks_st = 0;
            ks_ph ^= 1;
          }
        }
        return true;
      };
      auto weigh = [&](int i, uint32_t xx, bool first) {  // O += P V
        const uint32_t slot = NT == 1 ? (xx & 1) : i;
        if (i == 0 && !warp_wait_short(&vfull[vs_st], vs_ph, &abort_flag)) return false;
        if (!warp_wait_short(&pready[slot], (NT == 1 ? xx >> 1 : xx) & 1, &abort_flag)) return false;
        tc_fence_after();
        const uint64_t v = vd + (uint64_t)(vs_st * (kTB / 16));
        if (elect_one()) {
#pragma unroll
          for (int s = 0; s < kTile / 16; ++s)
            umma_bf16_ts(tmem + 256 + slot * 128, tmem + (kApart ? 320 : 0) + slot * 128 + s * 8, v + s * (2048 / 16),
                         idesc_o, !first || s > 0);
          umma_commit(&pvdone[slot]);
          if (i == NT - 1) umma_commit(&vempty[vs_st]);
        }
        __syncwarp();
        if (i == NT - 1) {
          if (++vs_st == p.ring) {
            vs_st = 0;
            vs_ph ^= 1;
          }
        }
        return true;
      };
      for (int j = 0; ok; ++j) {
        const int hb = j & 1;
        if (!warp_wait_short(&hfull[hb], (j >> 1) & 1, &abort_flag)) break;
        if (hdr[hb][kHb] < 0) break;
        const int T = hdr[hb][kHhi] - hdr[hb][kHlo];
        __syncwarp();
        if (lane == 0) mbar_arrive(&hempty[hb]);
        if (!warp_wait_short(&qfull, j & 1, &abort_flag)) break;
        tc_fence_after();
        // The scores are one step of their stream ahead of the weights: with two row tiles those of the
        // next key tile, with one those of the next key tile but one.
        constexpr int kAhead = NT == 1 ? 2 : 1;
        for (int i = 0; i < NT && ok; ++i) ok = scores(i, x);
        if (NT == 1 && ok && T > 1) ok = scores(0, x + 1);
        if (T <= kAhead && elect_one()) umma_commit(&qempty);  // every product with these queries is issued
        for (int t = 0; t < T && ok; ++t, ++x) {
          for (int i = 0; i < NT && ok; ++i) {
            const uint32_t slot = NT == 1 ? (x & 1) : i;
            const bool more = t + kAhead < T;
            if (kApart && more) {
              ok = warp_wait_short(&sfree[slot], (NT == 1 ? x >> 1 : x) & 1, &abort_flag);
              if (ok) ok = scores(i, x + kAhead);
            }
            if (ok && t == 0 && j > 0) ok = warp_wait_short(&ofree[i], (j - 1) & 1, &abort_flag);
            if (ok) ok = weigh(i, x, t < kAhead);  // the stream's first tile of the item
            if (!kApart && ok && more) ok = scores(i, x + kAhead);
          }
          if (t + kAhead + 1 == T && elect_one()) umma_commit(&qempty);
        }
      }
      __syncwarp();
      if (abort_flag && elect_one()) {  // what was issued ends before the tensor memory is freed
        umma_commit(&drained);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(&drained, 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
        }
      }
    }
    __syncwarp();
  } else {
    // =======================================================================
    // softmax: thread r of a row tile owns row r (draft t0 + r / G, head r % G)
    // =======================================================================
    const int str = warp >> 2;                      // stream
    const int i = NT == 1 ? 0 : str;                // row tile
    const uint32_t lane_base = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
    const int r = (warp & 3) * 32 + lane;
    const uint32_t s_addr = tmem + str * 128 + lane_base, o_addr = tmem + 256 + str * 128 + lane_base;
    // rows behind a query's last block in use belong to no item: zeros
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
      const int t1 = blocks_of<NT>(p, small ? q_n[b] : drafts_of(p, b)) * NT * p.TT;
      if (t1 < p.M) {
        uint4* z = reinterpret_cast<uint4*>(p.out + ((size_t)b * p.M + t1) * p.n_q * D);
        for (int e = tid; e < (p.M - t1) * p.n_q * (D / 8); e += 32 * kSoftWarps) z[e] = make_uint4(0, 0, 0, 0);
      }
    }
    uint32_t x = 0;  // key tiles of the CTA before this item
    uint32_t n = 0;  // tiles of this stream so far: the phase of its barriers
    bool ok = true;
    for (int j = 0; ok; ++j) {
      const int hb = j & 1;
      if (!warp_wait_short(&hfull[hb], (j >> 1) & 1, &abort_flag)) break;
      const int* h = hdr[hb];
      const int b = h[kHb];
      if (b < 0) break;
      const int sel = h[kHsel], L = h[kHL], n_use = h[kHn], Tc = h[kHTc], Tl = h[kHTl], lo = h[kHlo],
                hi = h[kHhi], part = h[kHslot];
      const int rt = r / p.G, g = r - rt * p.G;
      const int t_row = h[kHt0] + i * p.TT + rt;
      const bool in_use = rt < p.TT && t_row < n_use;
      const int32_t* mk = p.mask + ((size_t)b * p.M + (in_use ? t_row : 0)) * p.W;
      float m_ref = -INFINITY, l = 0.f;
      const int step = NT == 1 ? 2 : 1, t_first = NT == 1 ? lo + ((str - (int)x) & 1) : lo;
      for (int t = t_first; t < hi; t += step, ++n) {
        // ---- the keys of the tile that this row sees ----
        uint32_t see[4];
        const bool drafts = t >= Tc + Tl;
        const int left = t < Tc ? sel - t * kTile : drafts ? n_use - (t - Tc - Tl) * kTile : L - (t - Tc) * kTile;
        const int w0 = (t - Tc - Tl) * (kTile / 32);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = left - 32 * q;
          see[q] = c >= 32 ? ~0u : c > 0 ? (1u << c) - 1 : 0u;
          if (drafts) see[q] &= in_use && w0 + q < p.W ? (uint32_t)mk[w0 + q] : 0u;
        }
        const bool all = __all_sync(0xffffffffu, (see[0] & see[1] & see[2] & see[3]) == ~0u);
        if (!warp_wait_short(&sfull[str], n & 1, &abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float m_new = (all ? row_max<false>(s_addr, see) : row_max<true>(s_addr, see)) * p.scale_log2;
        const bool grow = m_new > m_ref + kSlack || (t == t_first && m_new > m_ref);
        const bool need = grow && l > 0.f;
        const bool any = __any_sync(0xffffffffu, need);
        if (any) {  // O holds products with weights of the old reference: rescale
          if (!warp_wait_short(&pvdone[str], (n - 1) & 1, &abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const float f = need ? ex2(m_ref - m_new) : 1.f;
          l *= f;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            uint32_t u[32];
            tmem_ld32(o_addr + c, o);
            tmem_ld_wait_for(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(o[e] * f);
            tmem_st32(o_addr + c, u);
          }
        }
        if (grow) m_ref = m_new;
        const float neg = m_ref == -INFINITY ? 0.f : -m_ref;
        // Weights apart from the scores: the products with the ones before have to be done.  Over the
        // scores: sfull came after them.  (Either way one phase of pvdone is outstanding at a time.)
        if (kApart && t > t_first && !any && !warp_wait_short(&pvdone[str], (n - 1) & 1, &abort_flag)) {
          ok = false;
          break;
        }
        if (kApart) tc_fence_after();
        const uint32_t p_addr = kApart ? o_addr + 64 : s_addr;
        uint64_t* read_bar = kApart ? &sfree[str] : nullptr;
        l += all ? row_weights<false>(s_addr, p_addr, see, p.scale_log2, neg, read_bar)
                 : row_weights<true>(s_addr, p_addr, see, p.scale_log2, neg, read_bar);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pready[str]);
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&hempty[hb]);
      x += hi - lo;
      if (t_first < hi && !warp_wait_short(&pvdone[str], (n - 1) & 1, &abort_flag)) break;
      // the factors of the streams' outputs in this row's (f of a stream without keys is 0, whatever
      // its output holds)
      float f0 = 1.f, f1 = 0.f;
      if (NT == 1) {  // stream 1 hands its state over, stream 0 writes the item
        if (str == 1) {
          if (j > 0 && !warp_wait_short(&taken, (j - 1) & 1, &abort_flag)) break;
          state[r] = make_float2(m_ref, l);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&joined);
          continue;
        }
        if (!warp_wait_short(&joined, j & 1, &abort_flag)) break;
        const float2 z = state[r];
        __syncwarp();
        if (lane == 0) mbar_arrive(&taken);
        const float m0 = m_ref, l0 = l;
        m_ref = fmaxf(m0, z.x);
        f0 = m0 == -INFINITY ? 0.f : ex2(m0 - m_ref);
        f1 = z.x == -INFINITY ? 0.f : ex2(z.x - m_ref);
        l = f0 * l0 + f1 * z.y;
      }
      tc_fence_after();
      const bool some = in_use && l != 0.f;  // a NaN sum is kept
      const bool row_out = rt < p.TT && t_row < p.M;
      if (part < 0) {
        f0 *= 1.f / l;
        f1 *= 1.f / l;
      }
      __nv_bfloat16* out = p.out + (((size_t)b * p.M + t_row) * p.n_q + (size_t)hk * p.G + g) * D;
      float* po = p.part_o + ((size_t)max(part, 0) * (D / 4) * (NT * 128) + i * 128 + r) * 4;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        tmem_ld32(o_addr + c, o);
        if (NT == 1) {
          float o1[32];
          tmem_ld32(o_addr + 128 + c, o1);
          tmem_ld_wait_for(o);
          tmem_ld_wait_for(o1);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = (f0 == 0.f ? 0.f : o[e] * f0) + (f1 == 0.f ? 0.f : o1[e] * f1);
        } else {
          tmem_ld_wait_for(o);
          if (part < 0) {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= f0;
          }
        }
        if (part < 0) {
          if (row_out) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint4 v = make_uint4(0, 0, 0, 0);
              if (some)
                v = make_uint4(pack_bf16x2(o[e], o[e + 1]), pack_bf16x2(o[e + 2], o[e + 3]),
                               pack_bf16x2(o[e + 4], o[e + 5]), pack_bf16x2(o[e + 6], o[e + 7]));
              *reinterpret_cast<uint4*>(out + c + e) = v;
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(po + (size_t)(c + e) * (NT * 128)) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
      if (part >= 0)
        *reinterpret_cast<float2*>(p.part_ml + ((size_t)part * (NT * 128) + i * 128 + r) * 2) = make_float2(m_ref, l);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ofree[i]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kSoftWarps + 1) tmem_dealloc(tmem, kTmemCols);
}

// The items that several CTAs of tree_attend_kernel shared: their parts merged in CTA order.  A CTA
// takes 1024 / D rows of the item noted by one CTA, a thread 4 elements of a row, neighbouring
// threads neighbouring rows (as the parts lie); the parts are read once, kAhead of them in flight,
// with a running maximum.  A note that no call of these sizes leaves (an attention kernel that gave up
// before it wrote it, which is reported) is passed over.
template <int D, int NT, int kAhead>
__global__ void __launch_bounds__(256) tree_combine_kernel(const __grid_constant__ TreeP p) {
  constexpr int kRows = 1024 / D;
  pdl_enter();
  if (p.by_item) {  // an item without drafts in use has no tiles and no note
    const int rb = blockIdx.y / p.n_kv % p.n_rb;
    if (rb * NT * p.TT >= drafts_of(p, blockIdx.y / p.n_kv / p.n_rb)) return;
  }
  const int4 it = p.merges[2 * blockIdx.y], cs = p.merges[2 * blockIdx.y + 1];
  const int b = it.x, n = it.w, c0 = cs.x, c1 = cs.y;
  if (!merge_note_ok({b, it.y, it.z, n, c0, c1, cs.z}, p.B, p.M, p.n_kv, p.groups)) return;
  const int r = blockIdx.x * kRows + (threadIdx.x & (kRows - 1)), e4 = threadIdx.x / kRows;  // row of the block, elements 4 e4 ..
  const int i = r >> 7, rt = (r & 127) / p.G, g = (r & 127) - rt * p.G;
  const int t = it.y + i * p.TT + rt;
  if (rt >= p.TT || t >= p.M) return;
  float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  if (t < n) {
    for (int c = c0; c <= c1; c += kAhead) {
      float2 ml[kAhead];
      float4 o[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        ml[u] = make_float2(-INFINITY, 0.f);
        if (c + u <= c1) {
          const size_t slot = c + u > c0 ? 2 * ((size_t)(c + u) * p.n_kv + it.z) : (size_t)cs.z;
          ml[u] = *reinterpret_cast<const float2*>(p.part_ml + (slot * (NT * 128) + r) * 2);
          o[u] = *reinterpret_cast<const float4*>(p.part_o + ((slot * (D / 4) + e4) * (NT * 128) + r) * 4);
        }
      }
      float mx = m;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) mx = fmaxf(mx, ml[u].x);
      const float mu = mx == -INFINITY ? 0.f : mx;
      const float f0 = m == -INFINITY ? 0.f : ex2(m - mu);
      l *= f0;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] *= f0;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (c + u > c1) break;
        // a part that saw no key has reference -inf (and zeros in O); a NaN reference stays NaN
        const float f = ml[u].x == -INFINITY ? 0.f : ex2(ml[u].x - mu);
        l = fmaf(f, ml[u].y, l);
        acc[0] = fmaf(f, o[u].x, acc[0]);
        acc[1] = fmaf(f, o[u].y, acc[1]);
        acc[2] = fmaf(f, o[u].z, acc[2]);
        acc[3] = fmaf(f, o[u].w, acc[3]);
      }
      m = mx;
    }
  }
  const float inv = 1.f / l;
  uint2 v = make_uint2(0, 0);
  if (l != 0.f) v = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
  *reinterpret_cast<uint2*>(p.out + (((size_t)b * p.M + t) * p.n_q + (size_t)it.z * p.G + g) * D + 4 * e4) = v;
}

// drafts per row tile, row tiles per CTA, row blocks per query
struct TreeShape {
  int TT, NT, n_rb;
};
TreeShape tree_shape(const msa_dims& d, int M) {
  TreeShape s;
  s.TT = 128 / (d.n_q / d.n_kv);
  s.NT = M > s.TT ? 2 : 1;
  s.n_rb = (M + s.NT * s.TT - 1) / (s.NT * s.TT);
  return s;
}

template <int D, int NT>
cudaError_t launch_attend(const TreeMaps& maps, TreeP& p, cudaStream_t s) {
  const int tile = D / 64 * kTile * 128;
  const size_t tables = (size_t)2 * (p.k + 1) * sizeof(int);
  // what aligning the tiles to 1 KB costs: the dynamic part begins behind the system's 1 KB and the
  // statically sized part (the kernel checks that this holds)
  auto kern = tree_attend_kernel<D, NT>;
  static const size_t fixed = [&] {
    cudaFuncAttributes a{};
    return cudaFuncGetAttributes(&a, kern) == cudaSuccess ? (a.sharedSizeBytes + 15) / 16 * 16 : (size_t)0;
  }();
  if (fixed == 0) return cudaErrorUnknown;
  const size_t room = 227 * 1024 - fixed;
  p.pad = (int)((1024 - (1024 + fixed) % 1024) % 1024);
  p.ring = (int)std::min<size_t>(kMaxRing, (room - p.pad - tables - NT * tile) / (2 * tile));
  const size_t smem = p.pad + (size_t)(NT + 2 * p.ring) * tile + tables;
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), (int)room);
  if (e != cudaSuccess) return e;
  const int n_ctas = sm_count();
  p.groups = n_ctas / p.n_kv;
  {
    TraceScope ts(kKTreeAttend, s);
    e = launch_pdl(kern, dim3(n_ctas), dim3(320), smem, s, maps, p);
    if (e != cudaSuccess) return e;
  }
  TraceScope ts(kKTreeCombine, s);
  constexpr int kRows = 1024 / D;
  const int row_groups = NT == 1 ? (p.M * p.G + kRows - 1) / kRows : NT * 128 / kRows;
  // Many items: about two parts each, and many threads; few items: many parts, their loads in flight
  // together.  16 drafts, 32/8 heads of 128, two against sixteen ahead: 1 query over 4K local tokens 22.3 against
  // 18.6 us, over 32K 45.3 against 43.4, 2 over 8K 32.1 against 31.4, 4 over 4K 33.0 against 34.4, 5 36.6 against 39.8,
  // 8 48.8 against 53.8, 32 over 2K 73.3 against 80.8.
  const int n_items = p.B * p.n_rb * p.n_kv;
  auto merge = n_items * 4 > n_ctas ? tree_combine_kernel<D, NT, 2> : tree_combine_kernel<D, NT, 16>;
  return launch_pdl(merge, dim3(row_groups, p.by_item ? n_items : n_ctas), dim3(256), 0, s, p);
}

struct TreeWs {
  int4* merges;
  int32_t* sel;
  float *part_ml, *part_o;
};
size_t tree_carve(const msa_dims& d, int B, int M, void* ws, TreeWs* out) {
  const TreeShape sh = tree_shape(d, M);
  Carver cv(ws);
  TreeWs w;
  w.merges = cv.take<int4>((size_t)2 * sm_count());
  w.sel = cv.take<int32_t>((size_t)B);
  w.part_ml = cv.take<float>((size_t)2 * sm_count() * sh.NT * 128 * 2);
  w.part_o = cv.take<float>((size_t)2 * sm_count() * sh.NT * 128 * d.head_dim);
  if (out) *out = w;
  return cv.size();
}

}  // namespace

msa_status tree_plan_launch(const int32_t* parents, const int32_t* n_draft, const int32_t* loc_len, int B, int M,
                            int pos_offset, int32_t* mask, int32_t* positions, cudaStream_t s) {
  TraceScope ts(kKTreePlan, s);
  MSA_CUDA_CHECK(launch_pdl(tree_plan_kernel, dim3(B), dim3((M + 31) / 32 * 32), 0, s, parents, n_draft, loc_len, M,
                            (M + 31) / 32, pos_offset, mask, positions));
  return MSA_OK;
}

msa_status tree_commit_launch(const msa_dims& d, const void* K_draft, const void* V_draft, const int32_t* path,
                              const int32_t* n_path, int B, int M, int A, void* K_loc, void* V_loc,
                              const int32_t* loc_len, int t_loc_max, int32_t* new_len, cudaStream_t s) {
  TraceScope ts(kKTreeCommit, s);
  const int64_t items = (int64_t)B * A;
  // warps per CTA, one against four: 1024 x 8 rows of 8 heads of 128 8.8 against 6.2 us, 256 x 17 4.8 against
  // 4.4, 64 x 17 2.5 against 2.0; 16 x 9 and 1 x 5 the same 1.5
  const int wpc = items >= 4LL * sm_count() ? 4 : 1;
  MSA_CUDA_CHECK(launch_pdl(tree_commit_kernel, dim3((unsigned)((items + wpc - 1) / wpc)), dim3(32 * wpc), 0, s,
                            static_cast<const uint4*>(K_draft), static_cast<const uint4*>(V_draft), path, n_path, B, M,
                            A, d.n_kv * d.head_dim * 2 / 16, static_cast<uint4*>(K_loc), static_cast<uint4*>(V_loc),
                            loc_len, t_loc_max, new_len));
  return MSA_OK;
}

size_t tree_attend_workspace(const msa_dims& d, int B, int M, int k, int t_loc_max) {
  (void)k, (void)t_loc_max;  // the parts depend on the GPU's SMs, not on the keys
  return tree_carve(d, B, M, nullptr, nullptr);
}

msa_status tree_attend_launch(const msa_dims& d, const TreeAttendCall& c, cudaStream_t s) {
  const TreeShape sh = tree_shape(d, c.M);
  TreeWs w;
  tree_carve(d, c.B, c.M, c.ws, &w);
  TreeP p{};
  p.mask = c.mask;
  p.n_draft = c.n_draft;
  p.loc_len = c.loc_len;
  p.chunk_off = c.chunk_off;
  p.topk_idx = c.topk_idx;
  p.out = static_cast<__nv_bfloat16*>(c.out);
  p.merges = w.merges;
  p.by_item = (int64_t)c.B * sh.n_rb * d.n_kv <= sm_count();
  p.sel = w.sel;
  p.part_o = w.part_o;
  p.part_ml = w.part_ml;
  p.B = c.B;
  p.M = c.M;
  p.W = (c.M + 31) / 32;
  p.n_q = d.n_q;
  p.n_kv = d.n_kv;
  p.G = d.n_q / d.n_kv;
  p.TT = sh.TT;
  p.n_rb = sh.n_rb;
  p.t_loc_max = c.t_loc_max;
  p.n_docs = c.n_docs;
  p.n_chunks = c.n_chunks;
  p.k = c.k;
  p.scale_log2 = (c.scale > 0.f ? c.scale : 1.0f / std::sqrt((float)d.head_dim)) * kLog2e;
  // tensor maps: rows of 64 elements (128 bytes, swizzled); dims (head element, head, row, query)
  TreeMaps maps{};
  const uint64_t row = (uint64_t)d.n_kv * d.head_dim * 2, qrow = (uint64_t)d.n_q * d.head_dim * 2;
  auto map4 = [&](CUtensorMap* m, const void* ptr, uint64_t heads, uint64_t rows, uint64_t pitch, uint32_t box_heads,
                  uint32_t box_rows) {
    const uint64_t dims[4] = {(uint64_t)d.head_dim, heads, rows, (uint64_t)c.B};
    const uint64_t strides[3] = {(uint64_t)d.head_dim * 2, pitch, pitch * rows};
    const uint32_t box[4] = {64, box_heads, box_rows, 1};
    return encode_tensor_map_once(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, ptr, dims, strides, box,
                                  CU_TENSOR_MAP_SWIZZLE_128B);
  };
  auto map3 = [&](CUtensorMap* m, const void* ptr, uint32_t box_rows) {
    const uint64_t dims[3] = {(uint64_t)d.head_dim, (uint64_t)d.n_kv, (uint64_t)c.n_chunks};
    const uint64_t strides[2] = {(uint64_t)d.head_dim * 2, row};
    const uint32_t box[3] = {64, 1, box_rows};
    return encode_tensor_map_once(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, ptr, dims, strides, box,
                                  CU_TENSOR_MAP_SWIZZLE_128B);
  };
  msa_status st = map4(&maps.q, c.q, d.n_q, c.M, qrow, p.G, p.TT);
  for (int i = 0; i < 14 && c.k > 0 && st == MSA_OK; ++i) st = map3(&maps.bar[i / 7][i % 7], i < 7 ? c.K_bar : c.V_bar, 1 << i % 7);
  if (c.t_loc_max > 0) {
    if (st == MSA_OK) st = map4(&maps.k_loc, c.K_loc, d.n_kv, c.t_loc_max, row, 1, kTile);
    for (int i = 0; i < 4 && st == MSA_OK; ++i) st = map4(&maps.v_loc[i], c.V_loc, d.n_kv, c.t_loc_max, row, 1, kTailRows[i]);
  }
  if (st == MSA_OK) st = map4(&maps.k_draft, c.K_draft, d.n_kv, c.M, row, 1, kTile);
  for (int i = 0; i < 2 && st == MSA_OK; ++i) st = map4(&maps.v_draft[i], c.V_draft, d.n_kv, c.M, row, 1, kTailRows[i]);
  if (st != MSA_OK) return st;
  if (c.k > 0 && c.B > kSmallB) {
    TraceScope ts(kKTreeSelect, s);
    MSA_CUDA_CHECK(launch_pdl(tree_select_kernel, dim3((c.B + 7) / 8), dim3(256), 0, s, c.topk_idx, c.chunk_off, c.B,
                              c.k, c.n_docs, c.n_chunks, w.sel));
  }
  cudaError_t e = d.head_dim == 128 ? (sh.NT == 2 ? launch_attend<128, 2>(maps, p, s) : launch_attend<128, 1>(maps, p, s))
                                    : (sh.NT == 2 ? launch_attend<64, 2>(maps, p, s) : launch_attend<64, 1>(maps, p, s));
  if (e != cudaSuccess) return cuda_fail(e, "tree attention launch");
  return MSA_OK;
}

}  // namespace msa
