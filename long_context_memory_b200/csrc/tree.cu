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

namespace msa {

namespace {

constexpr int kMaxDrafts = 256;
constexpr int kMaskWords = kMaxDrafts / 32;
constexpr float kLog2e = 1.4426950408889634f;

// ---------------------------------------------------------------------------
// plan: one CTA per query, one thread per draft.  Pointer doubling: after round r a draft's mask
// holds its 2^r nearest ancestors (itself included) and jump[] the next one up, so a tree of
// depth d takes ceil(log2 d) rounds of shared-memory reads instead of a chain of d dependent ones.
// Bound by latency (launch, two dependent loads, the rounds).
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
// commit: a warp per (query, accepted draft) copies its K and V rows
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
// hold all drafts), so K and V cross HBM once per 256 rows and each key tile of 128 keys costs
//   S = Q K^T   (tcgen05, operands in shared memory, fp32 scores in tensor memory),
//   P = exp2(S c - m)   (one thread per row, scores and weights in registers),
//   O += P V    (tcgen05, P bf16 in tensor memory over S, V in shared memory, O in tensor memory).
// P is rounded to bf16 because the tensor cores take bf16; its sum l is taken before the rounding,
// in fp32.  The reference maximum m of a row moves only when the running maximum passes it by
// 2^kSlack (O is then rescaled in tensor memory; weights stay below 2^kSlack otherwise, far
// inside bf16's and fp32's range), so that a tile normally touches O in the MMA alone.
//
// Keys of a query: its documents' pooled rows in groups of 8 (each document padded to whole
// groups), 16 groups to a tile; the local rows; the drafts.  Work is cut evenly: all tiles of all
// (query, row block, KV head) items in one line, CTA c of N takes tiles c W / N .. (c + 1) W / N, so
// (N = the SMs, or W where there are fewer tiles), so ragged batches and single long queries fill
// the GPU alike; the at most two items that a CTA
// shares with its neighbours leave partial results that tree_combine_kernel merges.
//
// Only value rows that some draft sees are copied (boxes of 128 and 8 rows, and single rows in
// 16-byte pieces where a group of 8 is not whole), into a ring whose V slots start as zeros where
// a first copy does not fill them: whatever stands in the rows behind a sequence, and in drafts
// that nobody sees, never reaches a product.  (Keys come in whole groups: a score that a row does
// not see is replaced, not multiplied.)
//
// Warps: 4 NT softmax warps (a thread per row), one producer (item headers, document tables, TMA),
// one MMA issuer.  One CTA per SM (its ring fills the shared memory).
// ---------------------------------------------------------------------------
constexpr int kTile = 128;        // keys per tile, rows per row tile
constexpr int kMaxRing = 6;
constexpr int kSmallB = 64;       // queries whose tile counts every CTA computes itself
constexpr float kSlack = 8.f;
constexpr int kTmemCols = 512;    // scores 2 x 128, outputs 2 x 128

struct TreeMaps {
  CUtensorMap q;
  CUtensorMap kl128, vl128;               // local cache, 128 rows
  CUtensorMap kl8, vl8, kd8, vd8, kb8, vb8;  // local cache, drafts, pooled rows: 8 rows
};

struct TreeP {
  const int32_t *mask, *n_draft, *loc_len, *chunk_off, *topk_idx;
  const __nv_bfloat16 *V_draft, *V_loc, *V_bar;
  __nv_bfloat16* out;
  int64_t* prefix;   // [B + 1] tiles before each query's first
  int32_t* groups;   // [B] pooled 8-row groups of each query (B > kSmallB)
  float* part_o;     // [2 N][NT * 128][D] unnormalised
  float* part_ml;    // [2 N][NT * 128][2] reference maximum, sum
  int B, M, W, n_q, n_kv, G, TT, n_rb, t_loc_max, n_docs, n_chunks, k, ring;
  float scale_log2;
};

enum { kHb = 0, kHt0, kHhk, kHL, kHn, kHNg, kHTc, kHTl, kHlo, kHhi, kHtab, kHslot, kHWords = 16 };

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
__device__ __forceinline__ int tiles_of(int groups, int L, int n) {
  return (groups + 15) / 16 + (L + kTile - 1) / kTile + (n + kTile - 1) / kTile;
}
// row blocks of a query that hold a draft in use
template <int NT>
__device__ __forceinline__ int blocks_of(const TreeP& p, int n) {
  return (n + NT * p.TT - 1) / (NT * p.TT);
}

// scores that the row does not see become -inf; the largest of the rest
__device__ __forceinline__ float hide_and_max(float (&s)[32], uint32_t see, bool all) {
  if (!all) {
    asm volatile("" : "+r"(see));  // a branch of its own, its tests made where they are used
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (!(see >> e & 1)) s[e] = -INFINITY;
  }
  float m[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
  for (int e = 4; e < 32; ++e) m[e & 3] = fmaxf(m[e & 3], s[e]);
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// weights 2^(s c + neg) of 32 keys to tensor memory as bf16 pairs; returns their sum
__device__ __forceinline__ float weigh_quarter(const float (&s)[32], float c, float neg, uint32_t addr) {
  uint32_t u[16];
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float a = ex2(fmaf(s[2 * e], c, neg)), z = ex2(fmaf(s[2 * e + 1], c, neg));
    sum[e & 3] += a + z;
    u[e] = pack_bf16x2(a, z);
  }
  tmem_st16(addr, u);
  return (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

// each query's pooled groups (large batches only): a warp per query
__global__ void __launch_bounds__(256) tree_groups_kernel(const int32_t* __restrict__ topk_idx,
                                                          const int32_t* __restrict__ chunk_off, int B, int k,
                                                          int n_docs, int n_chunks, int32_t* __restrict__ groups) {
  pdl_enter();
  const int b = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (b >= B) return;
  int g = 0;
  for (int r = lane; r < k; r += 32) {
    const int doc = topk_idx[(size_t)b * k + r];
    if (doc >= 0 && doc < n_docs) g += (max(0, min(chunk_off[doc + 1] - chunk_off[doc], n_chunks)) + 7) / 8;
  }
  g = __reduce_add_sync(0xffffffffu, g);
  if (lane == 0) groups[b] = g;
}

template <int D, int NT>
__global__ void __launch_bounds__(128 * NT + 64, 1) tree_attend_kernel(const __grid_constant__ TreeMaps maps,
                                                                       const __grid_constant__ TreeP p) {
  constexpr int DB = D / 64;            // 64-element blocks of a head
  constexpr int kBlk = kTile * 128;     // bytes of one block of a 128-row tile
  constexpr int kTB = DB * kBlk;        // bytes of a tile
  constexpr int kThreads = 128 * NT + 64;
  constexpr int kSoftWarps = 4 * NT;
  // (declared with the alignment that is sure behind the statically sized part; a stricter one would
  // be taken on trust and fold the rounding below away)
  extern __shared__ __align__(16) uint8_t sm_raw[];
  __shared__ uint64_t kfull[kMaxRing], kempty[kMaxRing], vfull[kMaxRing], vempty[kMaxRing];
  __shared__ uint64_t qfull, qempty, sfull[2], pready[2], pvdone[2], ofree[2], hfull[2], hempty[2], drained;
  __shared__ int hdr[2][kHWords];
  __shared__ int cnt[kSmallB];
  __shared__ long long warp_sum[kThreads / 32];
  __shared__ long long first_base;
  __shared__ int first_b;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;

  uint8_t* qs = sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u);  // [NT] row tiles (swizzle atoms: 1 KB aligned)
  uint8_t* ks = qs + NT * kTB;            // [ring] key tiles
  uint8_t* vs = ks + p.ring * kTB;        // [ring] value tiles
  int* tab = reinterpret_cast<int*>(vs + p.ring * kTB);  // [2][2][k + 1]: first group * 8 + rows % 8; first row

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
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfull[i], 1);
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
  for (int i = tid; i < kSmallB; i += kThreads) cnt[i] = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_enter();

  // ---- the line of tiles: every CTA counts it, CTA 0 leaves it for the merge ----
  const bool small = p.B <= kSmallB;
  if (small && p.k) {
    for (int i = tid; i < p.B * p.k; i += kThreads) {
      const int doc = p.topk_idx[i];
      if (doc >= 0 && doc < p.n_docs)
        atomicAdd(&cnt[i / p.k], (doc_rows(p, doc) + 7) / 8);
      else
        raise_dev_error(kDevErrBadIndex);
    }
    __syncthreads();
  }
  auto cost_of = [&](int b) -> long long {
    const int n = drafts_of(p, b);
    const int g = p.k ? (small ? cnt[b] : p.groups[b]) : 0;
    return (long long)p.n_kv * blocks_of<NT>(p, n) * tiles_of(g, local_of(p, b), n);
  };
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
  long long base = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) base += warp_sum[w];
    total += warp_sum[w];
  }
  const long long n_act = max(1ll, min((long long)gridDim.x, total));  // CTAs with work
  const long long w_begin = min(total, total * blockIdx.x / n_act), w_end = min(total, total * (blockIdx.x + 1) / n_act);
  for (int b = b0; b < b1; ++b) {
    const long long c = cost_of(b);
    if (blockIdx.x == 0) p.prefix[b] = base;
    if (w_begin < w_end && base <= w_begin && w_begin < base + c) {
      first_b = b;
      first_base = base;
    }
    base += c;
  }
  if (blockIdx.x == 0 && tid == 0) p.prefix[p.B] = total;
  __syncthreads();

  if (warp == kSoftWarps) {
    // =======================================================================
    // producer
    // =======================================================================
    uint32_t x = 0;  // tiles loaded
    int n_items = 0, tb = 0;
    bool ok = true;
    long long w = w_begin;
    long long bbase = first_base;
    int b = first_b;
    bool fresh = true;  // b's table is still to be built
    int L = 0, n = 0, Ng = 0;
    const int tstride = p.k + 1;
    while (ok) {
      const int hb = n_items & 1;
      if (n_items >= 2 && !warp_wait(&hempty[hb], ((n_items >> 1) - 1) & 1, &abort_flag)) {
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
      int T = 0;
      for (;;) {
        if (fresh) {
          n = drafts_of(p, b);
          L = local_of(p, b);
          Ng = 0;
          if (p.k) {
            tb ^= 1;
            int* tp = tab + tb * 2 * tstride;
            const int each = (p.k + 31) / 32;
            int sum = 0;
            for (int q = 0; q < each; ++q) {
              const int r = lane * each + q;
              if (r < p.k) {
                const int doc = p.topk_idx[(size_t)b * p.k + r];
                int rows = 0, row0 = 0;
                if (doc >= 0 && doc < p.n_docs) {
                  rows = doc_rows(p, doc);
                  row0 = p.chunk_off[doc];
                } else {
                  raise_dev_error(kDevErrBadIndex);
                }
                tp[r] = rows;
                tp[tstride + r] = row0;
                sum += (rows + 7) / 8;
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
                const int rows = tp[r];
                tp[r] = run * 8 + (rows & 7);
                run += (rows + 7) / 8;
              }
            }
            Ng = __shfl_sync(0xffffffffu, in, 31);
            if (lane == 0) tp[p.k] = Ng * 8;
            __syncwarp();
          }
          fresh = false;
        }
        T = tiles_of(Ng, L, n);
        const long long c = (long long)p.n_kv * blocks_of<NT>(p, n) * T;
        if (w < bbase + c) break;
        bbase += c;
        ++b;
        fresh = true;
      }
      const long long off = w - bbase;
      const int item = (int)(off / T), lo = (int)(off - (long long)item * T);
      const int hi = (int)min((long long)T, lo + (w_end - w));
      const int rb = item / p.n_kv, hk = item - rb * p.n_kv;
      const int t0 = rb * NT * p.TT;
      const int Tc = (Ng + 15) / 16, Tl = (L + kTile - 1) / kTile;
      if (lane == 0) {
        h[kHb] = b;
        h[kHt0] = t0;
        h[kHhk] = hk;
        h[kHL] = L;
        h[kHn] = n;
        h[kHNg] = Ng;
        h[kHTc] = Tc;
        h[kHTl] = Tl;
        h[kHlo] = lo;
        h[kHhi] = hi;
        h[kHtab] = tb;
        // whole items are written out; a shared one leaves its part: slot 0 of the CTA's first item, 1 of its last
        h[kHslot] = (lo == 0 && hi == T) ? -1 : 2 * (int)blockIdx.x + (n_items > 0);
        mbar_arrive(&hfull[hb]);
      }
      // queries: NT row tiles of TT drafts x G heads
      if (n_items >= 1 && !warp_wait(&qempty, (n_items - 1) & 1, &abort_flag)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(&qfull, NT * DB * p.G * p.TT * 128);
        for (int i = 0; i < NT; ++i)
          for (int d = 0; d < DB; ++d)
            tma_load_4d(qs + i * kTB + d * kBlk, &maps.q, &qfull, d * 64, hk * p.G, t0 + i * p.TT, b);
      }
      ++n_items;
      const int* tp = tab + tb * 2 * tstride;
      for (int t = lo; t < hi && ok; ++t, ++x) {
        const uint32_t st = x % p.ring, ph = (x / p.ring - 1) & 1;
        // the tile as 16 groups of 8 rows: lane < 16 holds its group's first row and the rows to copy
        const CUtensorMap *mk8, *mv8;
        const __nv_bfloat16* vsrc;  // the value rows' tensor at row 0 of this query
        int g_row = 0;
        uint32_t g_bits = 0;
        bool full = false;  // 128 consecutive rows: one box
        const int j0 = (t - Tc) * kTile, d0 = (t - Tc - Tl) * kTile;
        if (t < Tc) {
          mk8 = &maps.kb8;
          mv8 = &maps.vb8;
          vsrc = p.V_bar;
          const int g = t * 16 + lane;
          if (lane < 16 && g < Ng) {
            int a = 0, z = p.k - 1;  // the last document whose first group is at or before g
            while (a < z) {
              const int mid = (a + z + 1) >> 1;
              if ((tp[mid] >> 3) <= g) a = mid; else z = mid - 1;
            }
            const int g0 = tp[a] >> 3, g1 = tp[a + 1] >> 3, rest = tp[a] & 7;
            g_row = tp[tstride + a] + (g - g0) * 8;
            g_bits = g == g1 - 1 && rest ? (1u << rest) - 1 : 0xFFu;
          }
        } else if (t < Tc + Tl) {
          mk8 = &maps.kl8;
          mv8 = &maps.vl8;
          vsrc = p.V_loc + (size_t)b * p.t_loc_max * p.n_kv * D;
          full = L - j0 >= kTile;
          g_row = j0 + 8 * lane;
          if (lane < 16) g_bits = (1u << max(0, min(8, L - g_row))) - 1;
        } else {
          mk8 = &maps.kd8;
          mv8 = &maps.vd8;
          vsrc = p.V_draft + (size_t)b * p.M * p.n_kv * D;
          g_row = d0 + 8 * lane;
          uint32_t seen[4] = {0, 0, 0, 0};  // drafts that some draft of the query sees
          for (int r = lane; r < n; r += 32) {
            const int32_t* mk = p.mask + ((size_t)b * p.M + r) * p.W + d0 / 32;
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (d0 / 32 + q < p.W) seen[q] |= (uint32_t)mk[q];
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            seen[q] = __reduce_or_sync(0xffffffffu, seen[q]);
            const int left = n - d0 - 32 * q;
            if (left < 32) seen[q] &= left > 0 ? (1u << left) - 1 : 0u;
            g_bits |= (lane >> 2) == q ? seen[q] >> (8 * (lane & 3)) & 0xFFu : 0u;
          }
        }
        const int n_rows = __reduce_add_sync(0xffffffffu, __popc(g_bits));
        const uint32_t broken = __ballot_sync(0xffffffffu, g_bits != 0 && g_bits != 0xFFu);
        const int n_groups = __popc(__ballot_sync(0xffffffffu, g_bits != 0));
        for (int kv = 0; kv < 2; ++kv) {
          uint64_t* fullb = (kv ? vfull : kfull) + st;
          uint8_t* dst = (kv ? vs : ks) + st * kTB;
          if (x >= (uint32_t)p.ring && !warp_wait((kv ? vempty : kempty) + st, ph, &abort_flag)) {
            ok = false;
            break;
          }
          if (kv && x < (uint32_t)p.ring && n_rows < kTile) {  // a slot's first use that leaves rows out
            for (int i = lane; i < kTB / 16; i += 32) reinterpret_cast<uint4*>(dst)[i] = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive_expect_tx(fullb, (kv ? n_rows : 8 * n_groups) * D * 2);
          __syncwarp();
          if (full) {
            if (lane < DB)
              tma_load_4d(dst + lane * kBlk, kv ? &maps.vl128 : &maps.kl128, fullb, lane * 64, hk, j0, b);
          } else {
            if (kv ? g_bits == 0xFFu : g_bits != 0) {
              const CUtensorMap* m = kv ? mv8 : mk8;
              for (int d = 0; d < DB; ++d) {
                uint8_t* to = dst + d * kBlk + lane * 1024;
                if (t < Tc)
                  tma_load_3d(to, m, fullb, d * 64, hk, g_row);
                else
                  tma_load_4d(to, m, fullb, d * 64, hk, g_row, b);
              }
            }
            for (uint32_t left = kv ? broken : 0u; left; left &= left - 1) {
              const int src = __ffs(left) - 1;
              const uint32_t bits = __shfl_sync(0xffffffffu, g_bits, src);
              const int row = __shfl_sync(0xffffffffu, g_row, src);
              const __nv_bfloat16* from = vsrc + ((size_t)row * p.n_kv + hk) * D;
#pragma unroll
              for (int u = lane; u < 64 * DB; u += 32) {  // 8 rows x 8 DB pieces, at their swizzled places
                const int r = u / (8 * DB), c = u % (8 * DB);
                if (bits >> r & 1)
                  bulk_load(dst + (c >> 3) * kBlk + (src * 8 + r) * 128 + (((c & 7) ^ r) << 4),
                            from + (size_t)r * p.n_kv * D + c * 8, 16, fullb);
              }
            }
          }
          __syncwarp();
        }
      }
      w += hi - lo;
    }
    if (abort_flag && lane == 0) {  // the copies still in flight land before the CTA exits
      mbar_drain_ring(kfull, p.ring, (int)x - p.ring, (int)x + 1);
      mbar_drain_ring(vfull, p.ring, (int)x - p.ring, (int)x);
      if (n_items) mbar_drain_ring(&qfull, 1, n_items - 1, n_items);
    }
    __syncwarp();
  } else if (warp == kSoftWarps + 1) {
    // =======================================================================
    // MMA issuer
    // =======================================================================
    if (lane == 0) {
      constexpr uint32_t idesc_s = umma_idesc_bf16(128, 128);
      constexpr uint32_t idesc_o = umma_idesc_bf16(128, D) | kIdescBMnMajor;
      const uint32_t qa = smem_u32(qs), ka = smem_u32(ks), va = smem_u32(vs);
      uint32_t x = 0;
      bool ok = true;
      auto scores = [&](int i, uint32_t xx, bool last_reader) {  // S of row tile i and key tile xx
        const uint32_t st = xx % p.ring;
        if (!mbar_wait(&kfull[st], (xx / p.ring) & 1, &abort_flag)) return false;
        tc_fence_after();
        const uint32_t slot = NT == 1 ? (xx & 1) : i;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint32_t o = (s >> 2) * kBlk + (s & 3) * 32;
          umma_bf16(tmem + slot * 128, umma_desc_k_sw128(qa + i * kTB + o), umma_desc_k_sw128(ka + st * kTB + o), idesc_s,
                    s > 0);
        }
        umma_commit(&sfull[slot]);
        if (last_reader) umma_commit(&kempty[st]);
        return true;
      };
      auto weigh = [&](int i, uint32_t xx, bool first, bool last_reader) {  // O += P V
        const uint32_t st = xx % p.ring;
        const uint32_t slot = NT == 1 ? (xx & 1) : i;
        if (!mbar_wait(&pready[slot], (NT == 1 ? xx >> 1 : xx) & 1, &abort_flag)) return false;
        if (!mbar_wait(&vfull[st], (xx / p.ring) & 1, &abort_flag)) return false;
        tc_fence_after();
#pragma unroll
        for (int s = 0; s < kTile / 16; ++s)
          umma_bf16_ts(tmem + 256 + i * 128, tmem + slot * 128 + s * 8, umma_desc_mn_sw128(va + st * kTB + s * 2048, kBlk),
                       idesc_o, !first || s > 0);
        umma_commit(&pvdone[i]);
        if (last_reader) umma_commit(&vempty[st]);
        return true;
      };
      for (int j = 0; ok; ++j) {
        const int hb = j & 1;
        if (!mbar_wait(&hfull[hb], (j >> 1) & 1, &abort_flag)) break;
        if (hdr[hb][kHb] < 0) break;
        const int T = hdr[hb][kHhi] - hdr[hb][kHlo];
        mbar_arrive(&hempty[hb]);
        if (!mbar_wait(&qfull, j & 1, &abort_flag)) break;
        tc_fence_after();
        for (int i = 0; i < NT && ok; ++i) ok = scores(i, x, i == NT - 1);
        for (int t = 0; t < T && ok; ++t, ++x) {
          if (NT == 1 && t + 1 < T) ok = scores(0, x + 1, true);
          if (t + 1 == T) umma_commit(&qempty);  // every product with these queries is issued (NT 1), or is below
          for (int i = 0; i < NT && ok; ++i) {
            if (t == 0 && j > 0) ok = mbar_wait(&ofree[i], (j - 1) & 1, &abort_flag);
            if (ok) ok = weigh(i, x, t == 0, i == NT - 1);
            if (NT == 2 && ok && t + 1 < T) ok = scores(i, x + 1, i == 1);
          }
        }
      }
      if (abort_flag) {  // what was issued ends before the tensor memory is freed
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
    const int i = warp >> 2;                        // row tile
    const uint32_t lane_base = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
    const int r = (warp & 3) * 32 + lane;
    const uint32_t o_addr = tmem + 256 + i * 128 + lane_base;
    uint32_t x = 0;
    bool ok = true;
    for (int j = 0; ok; ++j) {
      const int hb = j & 1;
      if (!warp_wait(&hfull[hb], (j >> 1) & 1, &abort_flag)) break;
      const int* h = hdr[hb];
      const int b = h[kHb];
      if (b < 0) break;
      const int hk = h[kHhk], L = h[kHL], n = h[kHn], Ng = h[kHNg], Tc = h[kHTc], Tl = h[kHTl], lo = h[kHlo],
                hi = h[kHhi], part = h[kHslot];
      const int* tp = tab + h[kHtab] * 2 * (p.k + 1);
      const int rt = r / p.G, g = r - rt * p.G;
      const int t_row = h[kHt0] + i * p.TT + rt;
      const bool in_use = rt < p.TT && t_row < n;
      const int32_t* mk = p.mask + ((size_t)b * p.M + (in_use ? t_row : 0)) * p.W;
      float m_ref = -INFINITY, l = 0.f;
      for (int t = lo; t < hi; ++t, ++x) {
        // ---- the keys of the tile that this row sees ----
        uint32_t see[4];
        if (t < Tc) {
          uint32_t bits = 0;
          const int gi = t * 16 + lane;
          if (lane < 16 && gi < Ng) {
            int a = 0, z = p.k - 1;
            while (a < z) {
              const int mid = (a + z + 1) >> 1;
              if ((tp[mid] >> 3) <= gi) a = mid; else z = mid - 1;
            }
            const int g1 = tp[a + 1] >> 3, rest = tp[a] & 7;
            bits = (gi == g1 - 1 && rest ? (1u << rest) - 1 : 0xFFu) << (8 * (lane & 3));
          }
          bits |= __shfl_xor_sync(0xffffffffu, bits, 1);
          bits |= __shfl_xor_sync(0xffffffffu, bits, 2);
#pragma unroll
          for (int q = 0; q < 4; ++q) see[q] = __shfl_sync(0xffffffffu, bits, 4 * q);
        } else {
          const bool loc = t < Tc + Tl;
          const int d0 = loc ? (t - Tc) * kTile : (t - Tc - Tl) * kTile;
          const int left = (loc ? L : n) - d0;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int c = left - 32 * q;
            see[q] = c >= 32 ? ~0u : c > 0 ? (1u << c) - 1 : 0u;
            if (!loc) see[q] &= in_use && d0 / 32 + q < p.W ? (uint32_t)mk[d0 / 32 + q] : 0u;
          }
        }
        const bool all = __all_sync(0xffffffffu, (see[0] & see[1] & see[2] & see[3]) == ~0u);
        const uint32_t slot = NT == 1 ? (x & 1) : i;
        const uint32_t s_addr = tmem + slot * 128 + lane_base;
        if (!warp_wait(&sfull[slot], (NT == 1 ? x >> 1 : x) & 1, &abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // the scores in quarters of 32 keys, twice: for the maximum, then for the weights, which take
        // the columns of quarters already read
        float sa[32], sb[32];
        float m_new;
        tmem_ld32(s_addr, sa);
        tmem_ld32(s_addr + 32, sb);
        tmem_ld_wait_for(sa);
        tmem_ld_wait_for(sb);
        m_new = fmaxf(hide_and_max(sa, see[0], all), hide_and_max(sb, see[1], all));
        tmem_ld32(s_addr + 64, sa);
        tmem_ld32(s_addr + 96, sb);
        tmem_ld_wait_for(sa);
        tmem_ld_wait_for(sb);
        m_new = fmaxf(m_new, fmaxf(hide_and_max(sa, see[2], all), hide_and_max(sb, see[3], all))) * p.scale_log2;
        tmem_ld32(s_addr, sa);  // in flight while the reference is settled
        const bool grow = m_new > m_ref + kSlack || (t == lo && m_new > m_ref);
        const bool need = grow && l > 0.f;
        const bool any = __any_sync(0xffffffffu, need);
        if (any) {  // O holds products with weights of the old reference: rescale
          if (!warp_wait(&pvdone[i], (x - 1) & 1, &abort_flag)) {
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
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float(&cur)[32] = q & 1 ? sb : sa;
          tmem_ld_wait_for(cur);
          if (q < 3) tmem_ld32(s_addr + 32 * (q + 1), q & 1 ? sa : sb);
          if (!all) hide_and_max(cur, see[q], false);
          l += weigh_quarter(cur, p.scale_log2, neg, s_addr + 16 * q);
        }
        tmem_st_wait();
        // the products of the tile before have ended when those of this one may start: one phase of
        // pvdone is outstanding at a time
        if (t > lo && !any && !warp_wait(&pvdone[i], (x - 1) & 1, &abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pready[slot]);
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&hempty[hb]);
      if (!warp_wait(&pvdone[i], (x - 1) & 1, &abort_flag)) break;
      tc_fence_after();
      const bool some = in_use && l != 0.f;  // a NaN sum is kept
      const bool row_out = rt < p.TT && t_row < p.M;
      const float inv = 1.f / l;
      __nv_bfloat16* out = p.out + (((size_t)b * p.M + t_row) * p.n_q + (size_t)hk * p.G + g) * D;
      float* po = p.part_o + ((size_t)max(part, 0) * (NT * 128) + i * 128 + r) * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        tmem_ld32(o_addr + c, o);
        tmem_ld_wait_for(o);
        if (part < 0) {
          if (row_out) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint4 v = make_uint4(0, 0, 0, 0);
              if (some)
                v = make_uint4(pack_bf16x2(o[e] * inv, o[e + 1] * inv), pack_bf16x2(o[e + 2] * inv, o[e + 3] * inv),
                               pack_bf16x2(o[e + 4] * inv, o[e + 5] * inv), pack_bf16x2(o[e + 6] * inv, o[e + 7] * inv));
              *reinterpret_cast<uint4*>(out + c + e) = v;
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(po + c + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
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

// The rows that tree_attend_kernel did not write itself: shared items' parts merged in CTA order,
// zeros where a query has no drafts in use or no keys.  A warp per (query, draft, head).
template <int D, int NT>
__global__ void __launch_bounds__(256) tree_combine_kernel(const __grid_constant__ TreeP p, int grid) {
  constexpr int E = D / 32;
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= (int64_t)p.B * p.M * p.n_q) return;
  const int head = (int)(row % p.n_q), t = (int)(row / p.n_q % p.M), b = (int)(row / p.n_q / p.M);
  const int hk = head / p.G, g = head - hk * p.G;
  const int n = drafts_of(p, b);
  const long long base = p.prefix[b], cost = p.prefix[b + 1] - base, W = p.prefix[p.B];
  const long long n_ctas = min((long long)grid, W);
  const int rb = t / (NT * p.TT), blocks = blocks_of<NT>(p, n);
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  float l = 0.f;
  if (rb < blocks && cost > 0) {
    const long long T = cost / ((long long)p.n_kv * blocks);
    const long long w0 = base + ((long long)rb * p.n_kv + hk) * T, w1 = w0 + T - 1;  // the item's tiles
    // CTA c begins at floor(c W / N): tile w is in the CTA floor(((w + 1) N - 1) / W)
    const int c0 = (int)(((w0 + 1) * n_ctas - 1) / W), c1 = (int)(((w1 + 1) * n_ctas - 1) / W);
    if (c0 == c1) return;  // written
    if (t < n) {
      const int tr = t - rb * NT * p.TT, i = tr / p.TT;
      const int r = i * 128 + (tr - i * p.TT) * p.G + g;
      auto part = [&](int c) -> size_t {
        const bool first = c > c0 || W * c / n_ctas == w0;
        return (size_t)(2 * c + (first ? 0 : 1)) * (NT * 128) + r;
      };
      float m = -INFINITY;
      for (int c = c0 + lane; c <= c1; c += 32) m = fmaxf(m, p.part_ml[part(c) * 2]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll 4
      for (int c = c0; c <= c1; ++c) {
        const size_t pr = part(c);
        const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + pr * 2);
        // an empty part (no key seen) has weight 0 whatever its row of O holds
        const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - mu);
        l = fmaf(f, ml.y, l);
        float v[E];
        if constexpr (E == 4) {
          const float4 x4 = *reinterpret_cast<const float4*>(p.part_o + pr * D + lane * 4);
          v[0] = x4.x; v[1] = x4.y; v[2] = x4.z; v[3] = x4.w;
        } else {
          const float2 x2 = *reinterpret_cast<const float2*>(p.part_o + pr * D + lane * 2);
          v[0] = x2.x; v[1] = x2.y;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(f, v[e], acc[e]);
      }
    }
  }
  const float inv = 1.f / l;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(p.out + row * D + lane * E + e) =
        l > 0.f || l != l ? pack_bf16x2(acc[e] * inv, acc[e + 1] * inv) : 0u;
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
  const size_t tables = (size_t)4 * (p.k + 1) * sizeof(int);
  constexpr size_t kDyn = 227 * 1024 - 832;  // less the statically sized part
  p.ring = (int)std::min<size_t>(kMaxRing, (kDyn - 1024 - tables - NT * tile) / (2 * tile));
  const size_t smem = 1024 + (size_t)(NT + 2 * p.ring) * tile + tables;
  auto kern = tree_attend_kernel<D, NT>;
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), (int)kDyn);
  if (e != cudaSuccess) return e;
  const int n_ctas = sm_count();
  {
    TraceScope ts(kKTreeAttend, s);
    e = launch_pdl(kern, dim3(n_ctas), dim3(128 * NT + 64), smem, s, maps, p);
    if (e != cudaSuccess) return e;
  }
  TraceScope ts(kKTreeCombine, s);
  const int64_t rows = (int64_t)p.B * p.M * p.n_q;
  return launch_pdl(tree_combine_kernel<D, NT>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, s, p, n_ctas);
}

struct TreeWs {
  int64_t* prefix;
  int32_t* groups;
  float *part_ml, *part_o;
};
size_t tree_carve(const msa_dims& d, int B, int M, void* ws, TreeWs* out) {
  const TreeShape sh = tree_shape(d, M);
  Carver cv(ws);
  TreeWs w;
  w.prefix = cv.take<int64_t>((size_t)B + 1);
  w.groups = cv.take<int32_t>((size_t)B);
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
  p.V_draft = static_cast<const __nv_bfloat16*>(c.V_draft);
  p.V_loc = static_cast<const __nv_bfloat16*>(c.V_loc);
  p.V_bar = static_cast<const __nv_bfloat16*>(c.V_bar);
  p.out = static_cast<__nv_bfloat16*>(c.out);
  p.prefix = w.prefix;
  p.groups = w.groups;
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
  if (st == MSA_OK) st = map4(&maps.kd8, c.K_draft, d.n_kv, c.M, row, 1, 8);
  if (st == MSA_OK) st = map4(&maps.vd8, c.V_draft, d.n_kv, c.M, row, 1, 8);
  if (c.t_loc_max > 0) {
    if (st == MSA_OK) st = map4(&maps.kl128, c.K_loc, d.n_kv, c.t_loc_max, row, 1, kTile);
    if (st == MSA_OK) st = map4(&maps.vl128, c.V_loc, d.n_kv, c.t_loc_max, row, 1, kTile);
    if (st == MSA_OK) st = map4(&maps.kl8, c.K_loc, d.n_kv, c.t_loc_max, row, 1, 8);
    if (st == MSA_OK) st = map4(&maps.vl8, c.V_loc, d.n_kv, c.t_loc_max, row, 1, 8);
  }
  if (c.k > 0) {
    if (st == MSA_OK) st = map3(&maps.kb8, c.K_bar, 8);
    if (st == MSA_OK) st = map3(&maps.vb8, c.V_bar, 8);
  }
  if (st != MSA_OK) return st;
  if (c.k > 0 && c.B > kSmallB) {
    TraceScope ts(kKTreePlan, s);
    MSA_CUDA_CHECK(launch_pdl(tree_groups_kernel, dim3((c.B + 7) / 8), dim3(256), 0, s, c.topk_idx, c.chunk_off, c.B,
                              c.k, c.n_docs, c.n_chunks, w.groups));
  }
  cudaError_t e = d.head_dim == 128 ? (sh.NT == 2 ? launch_attend<128, 2>(maps, p, s) : launch_attend<128, 1>(maps, p, s))
                                    : (sh.NT == 2 ? launch_attend<64, 2>(maps, p, s) : launch_attend<64, 1>(maps, p, s));
  if (e != cudaSuccess) return cuda_fail(e, "tree attention launch");
  return MSA_OK;
}

}  // namespace msa
