// Rotary positions of query and key heads in the backbone's layout and frequency scaling, and the
// per-head RMS norms with the rotation in the same pass: forward, the decode step's form that
// writes the local cache, and the gradients.
//
//   rotation  (a, b) -> m (a cos - b sin, b cos + a sin); its gradient is the transpose (sin -> -sin)
//   norm      n = x r, r = 1 / sqrt(mean(x^2) + eps); y = Rot(n (w_off + w))
//   gradient  z = Rot^T(dy), u = z (w_off + w): dx = r (u - n mean(u n)), dw = sum z n
//
// All of them read each head once and write it once, a few dozen operations per element: bound by
// HBM at the large sizes and by the launch at the small ones.
//
// Work split.  A head is taken by L lanes (a power of two, 32 / L heads per warp at once); a lane
// holds one unit of two V-element vectors that contain whole rotation pairs, so that the rotation
// needs no exchange between lanes and the norm is a shuffle over the L lanes:
//   half         unit u: elements uV .. and R/2 + uV .. (pairs across the two vectors), and past
//                the rotated part two consecutive vectors;
//   interleaved  unit u: elements 2uV .. 2uV + 2V - 1 (pairs inside the vectors).
// Either way unit u turns the pairs uV .. uV + V - 1.  A warp takes one row (or a share of its
// heads when there are few rows): its lanes compute their V cosines and sines once and keep them in
// registers over the row's heads.  V is the widest of 16 bytes, 4 elements and 1 element that
// divides rot_dim / 2, head_dim, every stride and the pointers' alignment.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "common.cuh"
#include "internal.h"

namespace msa {

namespace {

constexpr int kMaxPairs = 128;  // rot_dim / 2 of the largest head

struct HeadsP {
  const void* in;
  void* out;
  const void* w;  // norm weight [D] or null
  const void* g;  // gradient of the output (backward)
  int64_t in_row, in_head, out_row, out_head, g_row, g_head;
  int heads;
  int its;  // warp iterations over the heads: ceil(heads / (32 / L))
};

struct RotP {
  HeadsP h[3];  // query heads, key heads, value heads (append: copied)
  int64_t rows;
  const int32_t* pos;
  const int32_t* slots;  // append: cache slot of each row
  int64_t rows_per_query;
  int t_loc_max;
  int D, half, units, L, logL, interleaved, parts, its;
  float mag, sign;  // sign: -1 for the transposed rotation
  float w_off, eps, inv_d;
  float* dw_part;  // backward: [CTA][2][D] weight-gradient partials, or null
  uint64_t turns[kMaxPairs];
};

template <int BYTES>
struct Raw;
template <>
struct Raw<16> { using t = uint4; };
template <>
struct Raw<8> { using t = uint2; };
template <>
struct Raw<4> { using t = uint32_t; };
template <>
struct Raw<2> { using t = uint16_t; };

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

template <typename T, int V>
struct Vec {
  using R = typename Raw<(int)sizeof(T) * V>::t;
  __device__ static __forceinline__ R zero() {
    R r;
    memset(&r, 0, sizeof(R));
    return r;
  }
  __device__ static __forceinline__ R load(const T* p) { return *reinterpret_cast<const R*>(p); }
  __device__ static __forceinline__ void store(T* p, R r) { *reinterpret_cast<R*>(p) = r; }
  __device__ static __forceinline__ void unpack(const R& r, float* x) {
    T t[V];
    memcpy(t, &r, sizeof(R));
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = to_f32(t[e]);
  }
  __device__ static __forceinline__ R pack(const float* x) {
    T t[V];
#pragma unroll
    for (int e = 0; e < V; ++e) t[e] = from_f32<T>(x[e]);
    R r;
    memcpy(&r, t, sizeof(R));
    return r;
  }
};

// cos and sin of pos * theta from theta as a 64-bit fraction of a turn: the product wraps to the
// exact fraction of a turn, which is split into the nearest quarter turn and a rest within an
// eighth of a turn, so that the rest's rounding to fp32 costs 2^-24 of a small angle
__device__ __forceinline__ void turn_cos_sin(uint64_t turns, int64_t pos, float mag, float& c, float& s) {
  const uint32_t u = (uint32_t)(((uint64_t)pos * turns) >> 32);
  const uint32_t quarter = (u + 0x20000000u) >> 30;
  const int32_t rest = (int32_t)(u - (quarter << 30));  // turns * 2^32 in [-2^29, 2^29)
  float sn, cs;
  sincospif((float)rest * 4.656612873077392578125e-10f, &sn, &cs);  // 2^-31: half turns
  const float c0 = (quarter & 1) ? -sn : cs, s0 = (quarter & 1) ? cs : sn;
  const float m = (quarter & 2) ? -mag : mag;
  c = c0 * m;
  s = s0 * m;
}

// a lane's place in a head
struct Unit {
  int a, b;              // element offsets of its two vectors
  bool va, vb, ra, rb;   // inside the head; rotated
};
template <int V>
__device__ __forceinline__ Unit unit_of(const RotP& p, int u) {
  Unit t;
  const bool in = u < p.units;
  if (p.interleaved) {
    t.a = 2 * V * u;
    t.b = t.a + V;
    t.ra = t.a < 2 * p.half;
    t.rb = t.b < 2 * p.half;
  } else {
    const int nr = p.half / V;
    t.ra = t.rb = u < nr;
    t.a = t.ra ? u * V : 2 * p.half + 2 * V * (u - nr);
    t.b = t.ra ? p.half + u * V : t.a + V;
  }
  t.va = in && t.a < p.D;
  t.vb = in && t.b < p.D;
  return t;
}

// rotate one unit in registers: x[0 .. V-1] the first vector, x[V .. 2V-1] the second
template <int V>
__device__ __forceinline__ void rotate_unit(const RotP& p, const Unit& t, const float* c, const float* s, float* x) {
  if (p.interleaved) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const bool r = (2 * e < V || V == 1) ? t.ra : t.rb;
      const float a = x[2 * e], b = x[2 * e + 1];
      if (r) {
        x[2 * e] = a * c[e] - b * s[e];
        x[2 * e + 1] = b * c[e] + a * s[e];
      }
    }
  } else if (t.ra) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float a = x[e], b = x[V + e];
      x[e] = a * c[e] - b * s[e];
      x[V + e] = b * c[e] + a * s[e];
    }
  }
}

template <int V, int J>
__device__ __forceinline__ void row_angles(const RotP& p, const uint64_t* turns, int sub, int64_t pos, float (*c)[V],
                                           float (*s)[V]) {
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int i = (sub + j * p.L) * V + e;
      c[j][e] = 1.f;
      s[j][e] = 0.f;
      if (i < p.half) turn_cos_sin(turns[i], pos, p.mag, c[j][e], s[j][e]);
      s[j][e] *= p.sign;
    }
}

// Rotation (NORM false) or norm and rotation of the query and key heads; append: keys and values
// into the cache.  A warp takes share `part` of a row's iterations (32 / L heads each).
template <typename T, int V, int J, bool NORM>
__global__ void __launch_bounds__(256) rotate_kernel(const __grid_constant__ RotP p) {
  constexpr int U = J == 1 ? 4 : 1;  // iterations whose loads are in flight together
  using X = Vec<T, V>;
  __shared__ uint64_t turns[kMaxPairs];
  for (int i = threadIdx.x; i < p.half; i += blockDim.x) turns[i] = p.turns[i];
  __syncthreads();
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int64_t row = item / p.parts;
  const int part = (int)(item - row * p.parts);
  if (row >= p.rows) return;
  const int sub = lane & (p.L - 1), grp = lane >> p.logL, gpw = 32 >> p.logL;
  float c[J][V], s[J][V];
  row_angles<V, J>(p, turns, sub, p.pos[row], c, s);
  int64_t cache_row = -1;
  if (p.slots) {
    const int slot = p.slots[row];
    if (slot >= 0 && slot < p.t_loc_max)
      cache_row = (row / p.rows_per_query) * p.t_loc_max + slot;
    else if (slot != -1 && lane == 0)
      raise_dev_error(kDevErrBadIndex);
  }
  const int it0 = (int)((int64_t)part * p.its / p.parts), it1 = (int)((int64_t)(part + 1) * p.its / p.parts);
  for (int base = it0; base < it1; base += U) {
    typename X::R a[U][J], b[U][J];
    T* dst[U];
    int cls[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      int it = base + u, k = 0;
      dst[u] = nullptr;
      if (it >= p.h[0].its) {
        it -= p.h[0].its;
        k = 1;
        if (it >= p.h[1].its) {
          it -= p.h[1].its;
          k = 2;
        }
      }
      cls[u] = k;
      const HeadsP& h = p.h[k];
      const int head = it * gpw + grp;
      const bool on = base + u < it1 && head < h.heads && (!p.slots || k == 0 || cache_row >= 0);
      const T* src = static_cast<const T*>(h.in) + row * h.in_row + (int64_t)head * h.in_head;
      if (on) {
        if (p.slots && k > 0)
          dst[u] = static_cast<T*>(h.out) + (cache_row * h.heads + head) * p.D;
        else
          dst[u] = static_cast<T*>(h.out) + row * h.out_row + (int64_t)head * h.out_head;
      }
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const Unit t = unit_of<V>(p, sub + j * p.L);
        a[u][j] = on && t.va ? X::load(src + t.a) : X::zero();
        b[u][j] = on && t.vb ? X::load(src + t.b) : X::zero();
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (base + u >= it1) break;  // warp-uniform
      const int k = cls[u];
      if (k == 2) {  // values: copied
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const Unit t = unit_of<V>(p, sub + j * p.L);
          if (dst[u] && t.va) X::store(dst[u] + t.a, a[u][j]);
          if (dst[u] && t.vb) X::store(dst[u] + t.b, b[u][j]);
        }
        continue;
      }
      float x[J][2 * V];
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        X::unpack(a[u][j], x[j]);
        X::unpack(b[u][j], x[j] + V);
        if (NORM) {
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) ss = fmaf(x[j][e], x[j][e], ss);
        }
      }
      float inv = 1.f;
      if (NORM) {
        for (int o = p.L >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        inv = __frsqrt_rn(fmaf(ss, p.inv_d, p.eps));
      }
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const Unit t = unit_of<V>(p, sub + j * p.L);
        if (NORM) {
          const T* w = static_cast<const T*>(p.h[k].w);
          float wf[2 * V];
          if (w) {
            X::unpack(t.va ? X::load(w + t.a) : X::zero(), wf);
            X::unpack(t.vb ? X::load(w + t.b) : X::zero(), wf + V);
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) x[j][e] = x[j][e] * inv * (p.w_off + wf[e]);
          } else {
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) x[j][e] *= inv;
          }
        }
        rotate_unit<V>(p, t, c[j], s[j], x[j]);
        if (dst[u] && t.va) X::store(dst[u] + t.a, X::pack(x[j]));
        if (dst[u] && t.vb) X::store(dst[u] + t.b, X::pack(x[j] + V));
      }
    }
  }
}

// Gradients of the norms: persistent warps take (row, share) items in a fixed order and keep the
// weight gradients of their lanes' elements in registers; a CTA sums its warps in order and writes
// one partial per weight.
template <typename T, int V, int J>
__global__ void __launch_bounds__(256) norm_grad_kernel(const __grid_constant__ RotP p) {
  constexpr int U = J == 1 ? 2 : 1;
  using X = Vec<T, V>;
  extern __shared__ float red[];  // [warps][2][D]
  __shared__ uint64_t turns[kMaxPairs];
  for (int i = threadIdx.x; i < p.half; i += blockDim.x) turns[i] = p.turns[i];
  __syncthreads();
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
  const int sub = lane & (p.L - 1), grp = lane >> p.logL, gpw = 32 >> p.logL;
  float dw[2][J][2 * V];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) dw[k][j][e] = 0.f;
  const int64_t n_items = p.rows * p.parts, stride = (int64_t)gridDim.x * n_warps;
  for (int64_t item = (int64_t)blockIdx.x * n_warps + warp; item < n_items; item += stride) {
    const int64_t row = item / p.parts;
    const int part = (int)(item - row * p.parts);
    float c[J][V], s[J][V];
    row_angles<V, J>(p, turns, sub, p.pos[row], c, s);
    const int it0 = (int)((int64_t)part * p.its / p.parts), it1 = (int)((int64_t)(part + 1) * p.its / p.parts);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const HeadsP& h = p.h[k];
      const int first = k ? p.h[0].its : 0;
      const int lo = max(it0 - first, 0), hi = min(it1 - first, h.its);
      const T* w = static_cast<const T*>(h.w);
      for (int base = lo; base < hi; base += U) {
        typename X::R xa[U][J], xb[U][J], ga[U][J], gb[U][J];
        bool on[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int head = (base + u) * gpw + grp;
          on[u] = base + u < hi && head < h.heads;
          const T* src = static_cast<const T*>(h.in) + row * h.in_row + (int64_t)head * h.in_head;
          const T* grd = static_cast<const T*>(h.g) + row * h.g_row + (int64_t)head * h.g_head;
#pragma unroll
          for (int j = 0; j < J; ++j) {
            const Unit t = unit_of<V>(p, sub + j * p.L);
            xa[u][j] = on[u] && t.va ? X::load(src + t.a) : X::zero();
            xb[u][j] = on[u] && t.vb ? X::load(src + t.b) : X::zero();
            ga[u][j] = on[u] && t.va ? X::load(grd + t.a) : X::zero();
            gb[u][j] = on[u] && t.vb ? X::load(grd + t.b) : X::zero();
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (base + u >= hi) break;  // warp-uniform
          float x[J][2 * V], z[J][2 * V], wf[J][2 * V];
          float ss = 0.f, dot = 0.f;
#pragma unroll
          for (int j = 0; j < J; ++j) {
            const Unit t = unit_of<V>(p, sub + j * p.L);
            X::unpack(xa[u][j], x[j]);
            X::unpack(xb[u][j], x[j] + V);
            X::unpack(ga[u][j], z[j]);
            X::unpack(gb[u][j], z[j] + V);
            rotate_unit<V>(p, t, c[j], s[j], z[j]);
            if (w) {
              X::unpack(t.va ? X::load(w + t.a) : X::zero(), wf[j]);
              X::unpack(t.vb ? X::load(w + t.b) : X::zero(), wf[j] + V);
            }
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) {
              wf[j][e] = w ? p.w_off + wf[j][e] : 1.f;
              ss = fmaf(x[j][e], x[j][e], ss);
              dot = fmaf(z[j][e] * wf[j][e], x[j][e], dot);
            }
          }
          for (int o = p.L >> 1; o > 0; o >>= 1) {
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
            dot += __shfl_xor_sync(0xffffffffu, dot, o);
          }
          // lanes without a head add nothing to the weight sums (eps may be 0)
          const float inv = on[u] ? __frsqrt_rn(fmaf(ss, p.inv_d, p.eps)) : 0.f;
          const float mean = dot * inv * p.inv_d;  // mean of u n
          T* dst = static_cast<T*>(h.out) + row * h.out_row + (int64_t)((base + u) * gpw + grp) * h.out_head;
#pragma unroll
          for (int j = 0; j < J; ++j) {
            const Unit t = unit_of<V>(p, sub + j * p.L);
            float dx[2 * V];
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) {
              const float n = x[j][e] * inv;
              dw[k][j][e] = fmaf(z[j][e], n, dw[k][j][e]);
              dx[e] = inv * (z[j][e] * wf[j][e] - n * mean);
            }
            if (on[u] && t.va) X::store(dst + t.a, X::pack(dx));
            if (on[u] && t.vb) X::store(dst + t.b, X::pack(dx + V));
          }
        }
      }
    }
  }
  if (!p.dw_part) return;
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const Unit t = unit_of<V>(p, sub + j * p.L);
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) {
        float v = dw[k][j][e];
        for (int o = 16; o >= p.L; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);  // the warp's heads
        if (grp == 0 && (e < V ? t.va : t.vb)) red[(warp * 2 + k) * p.D + (e < V ? t.a + e : t.b + e - V)] = v;
      }
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * p.D; i += blockDim.x) {
    float v = 0.f;
    for (int w = 0; w < n_warps; ++w) v += red[w * 2 * p.D + i];
    p.dw_part[(int64_t)blockIdx.x * 2 * p.D + i] = v;
  }
}

// the CTAs' partials summed in a fixed order: 32 columns per CTA, 8 warps over the partials
__global__ void __launch_bounds__(256) norm_grad_sum_kernel(const float* __restrict__ part, int n_part, int D,
                                                            float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ float red[8][32];
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (i < 2 * D) {
#pragma unroll 8
    for (int c = warp; c < n_part; c += 8) v += part[(int64_t)c * 2 * D + i];
  }
  red[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && i < 2 * D) {
#pragma unroll
    for (int w = 1; w < 8; ++w) v += red[w][lane];
    if (i < D) {
      if (dwq) dwq[i] = v;
    } else if (dwk) {
      dwk[i - D] = v;
    }
  }
}

bool vec_ok(const void* ptr, int64_t s0, int64_t s1, int v, int size) {
  return reinterpret_cast<uintptr_t>(ptr) % (size_t)(v * size) == 0 && s0 % v == 0 && s1 % v == 0;
}

// CTAs of the gradient kernel: two per SM (its registers allow two), fewer for few rows; the
// workspace holds one partial per CTA
int grad_ctas(int64_t rows, int its) {
  const int64_t warps = rows * std::max(1, its);
  return (int)std::max<int64_t>(1, std::min<int64_t>((warps + 7) / 8, 2 * sm_count()));
}

template <typename T, int V, int J>
cudaError_t launch_forward(const RotP& p, bool norm, cudaStream_t s) {
  const int64_t warps = p.rows * p.parts;
  // few warps: a small CTA on each of many SMs; many: 8 warps per CTA
  const int wpc = warps >= 8LL * sm_count() ? 8 : (int)std::max<int64_t>(1, warps / sm_count());
  const dim3 grid((unsigned)((warps + wpc - 1) / wpc));
  return norm ? launch_pdl(rotate_kernel<T, V, J, true>, grid, dim3(32 * wpc), 0, s, p)
              : launch_pdl(rotate_kernel<T, V, J, false>, grid, dim3(32 * wpc), 0, s, p);
}

template <typename T, int V, int J>
cudaError_t launch_backward(const RotP& p, int ctas, cudaStream_t s) {
  const size_t sm = 8 * 2 * (size_t)p.D * sizeof(float);
  return launch_pdl(norm_grad_kernel<T, V, J>, dim3(ctas), dim3(256), sm, s, p);
}

template <typename T>
cudaError_t launch_typed(const RotP& p, int v, int mode, int ctas, cudaStream_t s) {
  constexpr int W = 16 / (int)sizeof(T);
  if (v == W) return mode == 2 ? launch_backward<T, W, 1>(p, ctas, s) : launch_forward<T, W, 1>(p, mode == 1, s);
  if (sizeof(T) == 2 && v == 4)
    return mode == 2 ? launch_backward<T, 4, 1>(p, ctas, s) : launch_forward<T, 4, 1>(p, mode == 1, s);
  return mode == 2 ? launch_backward<T, 1, 4>(p, ctas, s) : launch_forward<T, 1, 4>(p, mode == 1, s);
}

int elem_size(msa_dtype t) { return t == MSA_FP32 ? 4 : 2; }

}  // namespace

// theta'_i / (2 pi) of every pair as 64-bit binary fractions; the last rotary of this host thread
// is kept (a decode loop asks for the same one every step)
void rotary_turns(const msa_rotary& r, uint64_t* f) {
  thread_local msa_rotary c_key;
  thread_local uint64_t c_f[kMaxPairs];
  thread_local bool c_set = false;
  const int half = r.rot_dim / 2;
  if (!c_set || std::memcmp(&c_key, &r, sizeof(r)) != 0) {
    const long double two_pi = 6.283185307179586476925286766559005768L;
    const long double R = r.rot_dim, s = r.factor;
    long double lb = logl((long double)r.base);
    if (r.scaling == MSA_SCALING_NTK && r.rot_dim > 2) lb += logl(s) * R / (R - 2.0L);
    long double first = 0, last = 0;
    if (r.scaling == MSA_SCALING_YARN) {
      auto at = [&](long double t) { return R * logl((long double)r.orig_len / (two_pi * t)) / (2.0L * lb); };
      first = std::max(floorl(at(r.high)), 0.0L);
      last = std::min(ceill(at(r.low)), R - 1.0L);
    }
    for (int i = 0; i < half; ++i) {
      long double th = expl(-2.0L * i / R * lb);
      if (r.scaling == MSA_SCALING_LINEAR) th /= s;
      if (r.scaling == MSA_SCALING_PARTS) {
        const long double t = r.orig_len * th / two_pi;
        const long double g = std::min(1.0L, std::max(0.0L, (t - r.low) / ((long double)r.high - r.low)));
        th = (1.0L - g) * th / s + g * th;
      }
      if (r.scaling == MSA_SCALING_YARN) {
        const long double span = last > first ? last - first : 0.001L;
        const long double g = 1.0L - std::min(1.0L, std::max(0.0L, (i - first) / span));
        th = (1.0L - g) * th / s + g * th;
      }
      c_f[i] = (uint64_t)ldexpl(th / two_pi, 64);  // th <= 1: below one turn
    }
    std::memcpy(&c_key, &r, sizeof(r));
    c_set = true;
  }
  for (int i = 0; i < half; ++i) f[i] = c_f[i];
}

size_t norm_grad_workspace(const msa_rotary& r, int64_t rows, int n_heads) {
  // an upper bound on the CTAs whatever the vector width: every head an iteration of its own
  return ((size_t)grad_ctas(rows, n_heads) * 2 * r.head_dim * sizeof(float) + 255) & ~size_t(255);
}

msa_status rotary_launch(const msa_rotary& r, msa_dtype dtype, const RotaryCall& c, cudaStream_t s) {
  RotP p{};
  const int size = elem_size(dtype);
  p.rows = c.rows;
  p.pos = c.positions;
  p.slots = c.slots;
  p.rows_per_query = c.rows_per_query;
  p.t_loc_max = c.t_loc_max;
  p.D = r.head_dim;
  p.half = r.rot_dim / 2;
  p.interleaved = r.layout == MSA_LAYOUT_INTERLEAVED;
  p.mag = (float)r.magnitude;
  p.sign = c.mode == 2 || c.grad ? -1.f : 1.f;
  p.w_off = c.weight_offset;
  p.eps = c.eps;
  p.inv_d = 1.0f / (float)r.head_dim;
  rotary_turns(r, p.turns);
  const msa_heads* in[3] = {c.q, c.k, c.v};
  const msa_heads* gr[2] = {c.dq, c.dk};
  const void* w[3] = {c.q_weight, c.k_weight, nullptr};
  int v = 16 / size;
  for (;; v = v == 8 ? 4 : 1) {  // the widest vector that fits everything
    if (v == 1) break;
    bool ok = p.D % v == 0 && p.half % (p.interleaved ? v / 2 : v) == 0;
    for (int i = 0; i < 3 && ok; ++i) {
      if (!in[i]) continue;
      ok = vec_ok(in[i]->in, in[i]->in_row, in[i]->in_head, v, size) && (!w[i] || vec_ok(w[i], 0, 0, v, size));
      if (c.slots && i > 0)
        ok = ok && vec_ok(i == 1 ? c.K_loc : c.V_loc, 0, 0, v, size);
      else if (c.mode != 2)
        ok = ok && vec_ok(in[i]->out, in[i]->out_row, in[i]->out_head, v, size);
      if (c.mode == 2)
        ok = ok && vec_ok(gr[i]->in, gr[i]->in_row, gr[i]->in_head, v, size) &&
             vec_ok(gr[i]->out, gr[i]->out_row, gr[i]->out_head, v, size);
    }
    if (ok) break;
  }
  p.units = p.interleaved ? (p.D + 2 * v - 1) / (2 * v) : p.half / v + (p.D - 2 * p.half + 2 * v - 1) / (2 * v);
  p.L = 1;
  p.logL = 0;
  while (p.L < 32 && p.L < p.units) {
    p.L *= 2;
    ++p.logL;
  }
  const int gpw = 32 / p.L;
  for (int i = 0; i < 3; ++i) {
    if (!in[i]) continue;
    HeadsP& h = p.h[i];
    h.in = in[i]->in;
    h.in_row = in[i]->in_row;
    h.in_head = in[i]->in_head;
    h.heads = in[i]->heads;
    h.w = w[i];
    h.its = (h.heads + gpw - 1) / gpw;
    const msa_heads* o = c.mode == 2 ? gr[i] : in[i];
    h.out = c.slots && i > 0 ? (i == 1 ? c.K_loc : c.V_loc) : o->out;
    h.out_row = o->out_row;
    h.out_head = o->out_head;
    if (c.mode == 2) {
      h.g = gr[i]->in;
      h.g_row = gr[i]->in_row;
      h.g_head = gr[i]->in_head;
    }
    p.its += h.its;
  }
  // shares of a row: enough warps for every SM when there are few rows
  const int64_t want = 16LL * sm_count();
  p.parts = (int)std::max<int64_t>(1, std::min<int64_t>(p.its, (want + p.rows - 1) / std::max<int64_t>(1, p.rows)));
  int ctas = 0;
  if (c.mode == 2) {
    ctas = grad_ctas(p.rows, p.parts);
    p.dw_part = c.dq_weight || c.dk_weight ? static_cast<float*>(c.ws) : nullptr;
  }
  {
    TraceScope ts(c.mode == 0 ? kKRotate : c.mode == 1 ? kKHeadNorm : kKHeadNormGrad, s);
    cudaError_t e = dtype == MSA_BF16   ? launch_typed<__nv_bfloat16>(p, v, c.mode, ctas, s)
                    : dtype == MSA_FP16 ? launch_typed<__half>(p, v, c.mode, ctas, s)
                                        : launch_typed<float>(p, v, c.mode, ctas, s);
    if (e != cudaSuccess) return cuda_fail(e, "rotary launch");
  }
  if (p.dw_part) {
    TraceScope ts(kKHeadNormSum, s);
    MSA_CUDA_CHECK(launch_pdl(norm_grad_sum_kernel, dim3((2 * p.D + 31) / 32), dim3(256), 0, s,
                              (const float*)p.dw_part, ctas, p.D, c.dq_weight, c.dk_weight));
  }
  return MSA_OK;
}

}  // namespace msa
