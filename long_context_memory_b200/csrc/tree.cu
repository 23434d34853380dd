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
// attention: a warp per (query, draft, query head), its lanes D / 32 dims each, one key at a time
// with a running maximum and sum
// ---------------------------------------------------------------------------
struct TreeP {
  const __nv_bfloat16 *q, *K_draft, *V_draft, *K_loc, *V_loc, *K_bar, *V_bar;
  const int32_t *mask, *n_draft, *loc_len, *chunk_off, *topk_idx;
  __nv_bfloat16* out;
  int B, M, W, n_q, n_kv, t_loc_max, n_docs, n_chunks, k;
  float scale_log2;
};

template <int D>
__global__ void __launch_bounds__(256) tree_attend_warp_kernel(const TreeP p) {
  constexpr int E = D / 32;
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= (int64_t)p.B * p.M * p.n_q) return;
  const int h = (int)(row % p.n_q), t = (int)(row / p.n_q % p.M), b = (int)(row / p.n_q / p.M);
  const int hk = h / (p.n_q / p.n_kv);
  const int n = p.n_draft ? max(0, min(p.n_draft[b], p.M)) : p.M;
  const int L = max(0, min(p.loc_len[b], p.t_loc_max));
  float q[E], acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(p.q[row * D + lane * E + e]) * p.scale_log2;
    acc[e] = 0.f;
  }
  auto key = [&](const __nv_bfloat16* K, const __nv_bfloat16* V, size_t r) {
    const size_t off = (r * p.n_kv + hk) * D + lane * E;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], __bfloat162float(K[off + e]), s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float m_new = fmaxf(m, s), m_use = m_new == -INFINITY ? 0.f : m_new;
    const float a = exp2f(m - m_use), w = exp2f(s - m_use);
    m = m_new;
    l = l * a + w;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * a + w * __bfloat162float(V[off + e]);
  };
  if (t < n) {
    for (int r = 0; r < p.k; ++r) {
      const int doc = p.topk_idx[(size_t)b * p.k + r];
      if (doc < 0 || doc >= p.n_docs) {
        if (lane == 0) raise_dev_error(kDevErrBadIndex);
        continue;
      }
      const int c1 = min(p.chunk_off[doc + 1], p.n_chunks);
      for (int c = max(0, p.chunk_off[doc]); c < c1; ++c) key(p.K_bar, p.V_bar, c);
    }
    for (int j = 0; j < L; ++j) key(p.K_loc, p.V_loc, (size_t)b * p.t_loc_max + j);
    const int32_t* mk = p.mask + ((size_t)b * p.M + t) * p.W;
    for (int j = 0; j < n; ++j)
      if (mk[j >> 5] >> (j & 31) & 1) key(p.K_draft, p.V_draft, (size_t)b * p.M + j);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) p.out[row * D + lane * E + e] = __float2bfloat16_rn(l > 0.f ? acc[e] / l : 0.f);
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
  (void)d, (void)B, (void)M, (void)k, (void)t_loc_max;
  return 256;
}

msa_status tree_attend_launch(const msa_dims& d, const TreeAttendCall& c, cudaStream_t s) {
  TraceScope ts(kKTreeAttend, s);
  TreeP p{};
  using BF = __nv_bfloat16;
  p.q = static_cast<const BF*>(c.q);
  p.K_draft = static_cast<const BF*>(c.K_draft);
  p.V_draft = static_cast<const BF*>(c.V_draft);
  p.K_loc = static_cast<const BF*>(c.K_loc);
  p.V_loc = static_cast<const BF*>(c.V_loc);
  p.K_bar = static_cast<const BF*>(c.K_bar);
  p.V_bar = static_cast<const BF*>(c.V_bar);
  p.mask = c.mask;
  p.n_draft = c.n_draft;
  p.loc_len = c.loc_len;
  p.chunk_off = c.chunk_off;
  p.topk_idx = c.topk_idx;
  p.out = static_cast<BF*>(c.out);
  p.B = c.B;
  p.M = c.M;
  p.W = (c.M + 31) / 32;
  p.n_q = d.n_q;
  p.n_kv = d.n_kv;
  p.t_loc_max = c.t_loc_max;
  p.n_docs = c.n_docs;
  p.n_chunks = c.n_chunks;
  p.k = c.k;
  p.scale_log2 = (c.scale > 0.f ? c.scale : 1.0f / std::sqrt((float)d.head_dim)) * kLog2e;
  const int64_t rows = (int64_t)c.B * c.M * d.n_q;
  auto kern = d.head_dim == 128 ? tree_attend_warp_kernel<128> : tree_attend_warp_kernel<64>;
  MSA_CUDA_CHECK(launch_pdl(kern, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, s, p));
  return MSA_OK;
}

}  // namespace msa
