// Rotary positions of query and key heads in the backbone's layout and frequency scaling, and the
// per-head RMS norms with the rotation in the same pass: forward, the decode step's form that
// writes the local cache, and the gradients.
//
//   rotation  (a, b) -> m (a cos - b sin, b cos + a sin); its gradient is the transpose (sin -> -sin)
//   norm      n = x r, r = 1 / sqrt(mean(x^2) + eps); y = Rot(n (w_off + w))
//   gradient  z = Rot^T(dy), u = z (w_off + w): dx = r (u - n mean(u n)), dw = sum z n
//
// All of them read each head once and write it once, a few dozen operations per element: bound by
// HBM at the large sizes and by the launch at the small ones.  Measured: the transposed rotation of
// 8193 rows of 40 fp32 heads of 128 (336 MB) 64.6 us, 5.2 TB/s; norm and rotation of 16384 rows of 40
// bf16 heads of 128 (336 MB) 70 us, 4.8 TB/s (a plain copy of the same bytes: 53 us, 6.3 TB/s; here the
// issue slots are 53% busy as well); the gradients of 8191 rows of 40 fp16 heads of 96 (189 MB) 62 us, 3.1
// TB/s, bound by the arithmetic of a head group and its dependences; one row 2.8 us, a decode step of 16
// rows with its cache 3.4 us on the device, of which the launch is most.
//
// Work split.  A head is taken by L lanes (a power of two, 32 / L heads per warp at once); a lane
// holds one unit of two V-element vectors that contain whole rotation pairs, so that the rotation
// needs no exchange between lanes and the norm is a shuffle over the L lanes:
//   half         unit u: elements uV .. and R/2 + uV .. (pairs across the two vectors), and past
//                the rotated part two consecutive vectors;
//   interleaved  unit u: elements 2uV .. 2uV + 2V - 1 (pairs inside the vectors).
// Either way unit u turns the pairs uV .. uV + V - 1.  A warp takes one row (or a share of its
// heads when there are few rows): its lanes compute the row's cosines and sines once for all its
// heads.  V is the widest of 16 bytes, 4 elements and 1 element that
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

constexpr int kRotCtas = 2, kRotBatch = 2;    // CTAs per SM, iterations whose loads are in flight together
constexpr int kGradCtas = 2, kGradBatch = 2;  // (the gradients')
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
  int D, half, units, L, logL, interleaved, parts, its, classes;
  int full;  // every element is turned (rot_dim == head_dim)
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
};

// A lane's unit (two vectors a, b of V elements) as V pairs of fp32.  PAIRED: pair e holds the two
// elements that are turned together (interleaved layout, or single elements); else pairs 0 .. V/2 - 1
// are the first vector's neighbours and the others the second's, and pair e is turned with e + V/2.
__device__ __forceinline__ uint64_t wide2(uint32_t w, __nv_bfloat16) {
  return pack_f32x2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint64_t wide2(uint32_t w, __half) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pack_f32x2(f.x, f.y);
}
__device__ __forceinline__ uint32_t narrow2(uint64_t v, __nv_bfloat16) {
  const float2 f = unpack_f32x2(v);
  return pack_bf16x2(f.x, f.y);
}
__device__ __forceinline__ uint32_t narrow2(uint64_t v, __half) {
  const float2 f = unpack_f32x2(v);
  const __half2 h = __floats2half2_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T, int V>
__device__ __forceinline__ void widen(const typename Vec<T, V>::R& a, const typename Vec<T, V>::R& b, uint64_t (&x)[V]) {
  if constexpr (V == 1) {
    T ta, tb;
    memcpy(&ta, &a, sizeof(T));
    memcpy(&tb, &b, sizeof(T));
    x[0] = pack_f32x2(to_f32(ta), to_f32(tb));
  } else if constexpr (sizeof(T) == 4) {
    float fa[V], fb[V];
    memcpy(fa, &a, sizeof(fa));
    memcpy(fb, &b, sizeof(fb));
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      x[e] = pack_f32x2(fa[2 * e], fa[2 * e + 1]);
      x[V / 2 + e] = pack_f32x2(fb[2 * e], fb[2 * e + 1]);
    }
  } else {
    uint32_t wa[V / 2], wb[V / 2];
    memcpy(wa, &a, sizeof(wa));
    memcpy(wb, &b, sizeof(wb));
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      x[e] = wide2(wa[e], T());
      x[V / 2 + e] = wide2(wb[e], T());
    }
  }
}
template <typename T, int V>
__device__ __forceinline__ void narrow(const uint64_t (&x)[V], typename Vec<T, V>::R& a, typename Vec<T, V>::R& b) {
  if constexpr (V == 1) {
    const float2 f = unpack_f32x2(x[0]);
    const T ta = from_f32<T>(f.x), tb = from_f32<T>(f.y);
    memcpy(&a, &ta, sizeof(T));
    memcpy(&b, &tb, sizeof(T));
  } else if constexpr (sizeof(T) == 4) {
    float2 fa[V / 2], fb[V / 2];
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      fa[e] = unpack_f32x2(x[e]);
      fb[e] = unpack_f32x2(x[V / 2 + e]);
    }
    memcpy(&a, fa, sizeof(fa));
    memcpy(&b, fb, sizeof(fb));
  } else {
    uint32_t wa[V / 2], wb[V / 2];
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      wa[e] = narrow2(x[e], T());
      wb[e] = narrow2(x[V / 2 + e], T());
    }
    memcpy(&a, wa, sizeof(wa));
    memcpy(&b, wb, sizeof(wb));
  }
}
__device__ __forceinline__ uint64_t swap_f32x2(uint64_t v) {
  const float2 f = unpack_f32x2(v);
  return pack_f32x2(f.y, f.x);
}

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

// The factors that turn a unit: PAIRED: y_e = x_e p_e + swap(x_e) q_e with p = (c, c), q = (-s, s);
// else y_e = x_e p_e + x_{e+V/2} q_e and y_{e+V/2} = x_{e+V/2} p_{e+V/2} + x_e q_{e+V/2} with
// p = c, q = -s then s.  (A unit turns the pairs u V .. u V + V - 1.)
template <int V, bool PAIRED>
__device__ __forceinline__ void unit_factors(const float2* ang, int i0, int half, uint64_t (&p)[V], uint64_t (&q)[V]) {
  auto at = [&](int i) { return i < half ? ang[i] : make_float2(1.f, 0.f); };
  if constexpr (PAIRED) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float2 cs = at(i0 + e);
      p[e] = pack_f32x2(cs.x, cs.x);
      q[e] = pack_f32x2(-cs.y, cs.y);
    }
  } else {
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      const float2 u = at(i0 + 2 * e), v = at(i0 + 2 * e + 1);
      p[e] = p[V / 2 + e] = pack_f32x2(u.x, v.x);
      q[e] = pack_f32x2(-u.y, -v.y);
      q[V / 2 + e] = pack_f32x2(u.y, v.y);
    }
  }
}
template <int V, bool PAIRED>
__device__ __forceinline__ uint64_t partner(const uint64_t (&x)[V], int e) {
  if constexpr (PAIRED) return swap_f32x2(x[e]);
  return x[e < V / 2 ? e + V / 2 : e - V / 2];
}
// is pair e of the unit turned (else its elements only take their weights)
template <int V, bool PAIRED, bool INTER>
__device__ __forceinline__ bool turned(const Unit& t, int e) {
  return !INTER || V == 1 || 2 * e < V ? t.ra : t.rb;
}

// A row's cosines and sines: the warp's lanes compute each pair's once, `ang` (shared memory of the
// warp) hands them out
__device__ __forceinline__ void row_angles(const RotP& p, const uint64_t* turns, int64_t pos, float2* ang, int lane) {
  __syncwarp();
  for (int i = lane; i < p.half; i += 32) {
    float c, s;
    turn_cos_sin(turns[i], pos, p.mag, c, s);
    ang[i] = make_float2(c, s * p.sign);
  }
  __syncwarp();
}

// Rotation (NORM false) or norm and rotation of the query and key heads; append: keys and values
// into the cache.  Persistent warps, each a row (or share `part` of its iterations of 32 / L heads) at
// a time.  The weights are folded into the rotation's factors, which stay in registers over the heads
// of a class: y = (x (w p) + x' (w' q)) r; two elements per instruction throughout.
template <typename T, int V, int J, bool NORM, bool INTER>
__global__ void __launch_bounds__(256, kRotCtas) rotate_kernel(const __grid_constant__ RotP p) {
  constexpr int U = J == 1 ? kRotBatch : 1;  // iterations whose loads are in flight together
  constexpr bool PAIRED = INTER || V == 1;
  using X = Vec<T, V>;
  __shared__ uint64_t turns[kMaxPairs];
  __shared__ float2 angles[8][kMaxPairs];
  for (int i = threadIdx.x; i < p.half; i += blockDim.x) turns[i] = p.turns[i];
  __syncthreads();
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane & (p.L - 1), grp = lane >> p.logL, gpw = 32 >> p.logL;
  Unit un[J];
#pragma unroll
  for (int j = 0; j < J; ++j) un[j] = unit_of<V>(p, sub + j * p.L);
  // A cursor runs over the warp's batches of U iterations: rows (or shares of rows), their classes of
  // heads, the iterations of a class.  The next batch's loads are in flight while one is worked on.
  const int64_t n_items = p.rows * p.parts, stride = (int64_t)gridDim.x * (blockDim.x >> 5);
  struct Cursor {
    int64_t item, row;
    int k, base, hi, pos, slot;
  };
  auto enter_class = [&](Cursor& c, int k, int64_t part) {  // the share's first class from k on with iterations
    const int it0 = p.parts == 1 ? 0 : (int)(part * p.its / p.parts);
    const int it1 = p.parts == 1 ? p.its : (int)((part + 1) * p.its / p.parts);
    for (; k < p.classes; ++k) {
      const int first = k == 0 ? 0 : k == 1 ? p.h[0].its : p.h[0].its + p.h[1].its;
      c.k = k;
      c.base = max(it0 - first, 0);
      c.hi = min(it1 - first, p.h[k].its);
      if (c.base < c.hi) return true;
    }
    return false;
  };
  auto enter_item = [&](Cursor& c) {  // a share has at least one iteration
    if (c.item >= n_items) return;
    c.row = p.parts == 1 ? c.item : c.item / p.parts;
    c.pos = p.pos[c.row];
    c.slot = p.slots ? p.slots[c.row] : 0;
    enter_class(c, 0, c.item - c.row * p.parts);
  };
  auto advance = [&](Cursor& c) {
    c.base += U;
    if (c.base < c.hi || enter_class(c, c.k + 1, c.item - c.row * p.parts)) return;
    c.item += stride;
    enter_item(c);
  };
  auto fetch = [&](const Cursor& c, typename X::R (&a)[U][J], typename X::R (&b)[U][J]) {
    if (c.item >= n_items) return;
    const HeadsP& h = p.h[c.k];
    const T* hp = static_cast<const T*>(h.in) + c.row * h.in_row + (int64_t)(c.base * gpw + grp) * h.in_head;
    const int64_t step = gpw * h.in_head;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool on = c.base + u < c.hi && (c.base + u) * gpw + grp < h.heads;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        a[u][j] = on && un[j].va ? X::load(hp + un[j].a) : X::zero();
        b[u][j] = on && un[j].vb ? X::load(hp + un[j].b) : X::zero();
      }
      hp += step;
    }
  };
  Cursor cur;
  cur.item = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp;
  enter_item(cur);
  typename X::R a[U][J], b[U][J];
  fetch(cur, a, b);
  int64_t angles_of = -1, factors_of = -1;  // row of `angles`; row * 4 + class of the factors
  uint64_t fp[J][V], fq[J][V];
  while (cur.item < n_items) {
    Cursor nxt = cur;
    advance(nxt);
    typename X::R na[U][J], nb[U][J];
    fetch(nxt, na, nb);
    const int k = cur.k;
    const HeadsP& h = p.h[k];
    const bool cached = p.slots && k > 0;
    if (angles_of != cur.row) {
      row_angles(p, turns, cur.pos, angles[warp], lane);
      angles_of = cur.row;
      if (p.slots && cur.slot != -1 && (cur.slot < 0 || cur.slot >= p.t_loc_max) && lane == 0) raise_dev_error(kDevErrBadIndex);
    }
    if (k < 2 && factors_of != cur.row * 4 + k) {
      factors_of = cur.row * 4 + k;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        unit_factors<V, PAIRED>(angles[warp], (sub + j * p.L) * V, p.half, fp[j], fq[j]);
        if (NORM && h.w) {
          const T* wp = static_cast<const T*>(h.w);
          uint64_t w[V];
          widen<T, V>(un[j].va ? X::load(wp + un[j].a) : X::zero(), un[j].vb ? X::load(wp + un[j].b) : X::zero(), w);
          const uint64_t off = pack_f32x2(p.w_off, p.w_off);
#pragma unroll
          for (int e = 0; e < V; ++e) w[e] = add_f32x2(w[e], off);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            fp[j][e] = mul_f32x2(fp[j][e], w[e]);
            fq[j][e] = mul_f32x2(fq[j][e], partner<V, PAIRED>(w, e));
          }
        }
      }
    }
    const bool live = !cached || (cur.slot >= 0 && cur.slot < p.t_loc_max);
    const int64_t out_head = cached ? p.D : h.out_head;
    T* op = static_cast<T*>(h.out) + (int64_t)(cur.base * gpw + grp) * out_head +
            (cached ? (cur.row / p.rows_per_query * p.t_loc_max + cur.slot) * h.heads * p.D : cur.row * h.out_row);
    const int64_t step = gpw * out_head;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (cur.base + u >= cur.hi) break;  // warp-uniform
      if (k < 2) {
        uint64_t x[J][V], ss2 = 0;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          widen<T, V>(a[u][j], b[u][j], x[j]);
          if (NORM) {
#pragma unroll
            for (int e = 0; e < V; ++e) ss2 = fma_f32x2(x[j][e], x[j][e], ss2);
          }
        }
        uint64_t inv2 = 0;
        if (NORM) {
          const float2 s2 = unpack_f32x2(ss2);
          float ss = s2.x + s2.y;
          for (int o = p.L >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float inv = rsqrtf(fmaf(ss, p.inv_d, p.eps));
          inv2 = pack_f32x2(inv, inv);
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
          uint64_t y[V];
          if (p.full) {
#pragma unroll
            for (int e = 0; e < V; ++e)
              y[e] = fma_f32x2(partner<V, PAIRED>(x[j], e), fq[j][e], mul_f32x2(x[j][e], fp[j][e]));
          } else {  // what is not turned is not multiplied by a zero sine: the other may be infinite
#pragma unroll
            for (int e = 0; e < V; ++e)
              if (turned<V, PAIRED, INTER>(un[j], e))
                y[e] = fma_f32x2(partner<V, PAIRED>(x[j], e), fq[j][e], mul_f32x2(x[j][e], fp[j][e]));
              else
                y[e] = NORM ? mul_f32x2(x[j][e], fp[j][e]) : x[j][e];
          }
          if (NORM) {
#pragma unroll
            for (int e = 0; e < V; ++e) y[e] = mul_f32x2(y[e], inv2);
          }
          narrow<T, V>(y, a[u][j], b[u][j]);
        }
      }
      const bool on = (cur.base + u) * gpw + grp < h.heads && live;
#pragma unroll
      for (int j = 0; j < J; ++j) {  // (the values of an append are stored as they came)
        if (on && un[j].va) X::store(op + un[j].a, a[u][j]);
        if (on && un[j].vb) X::store(op + un[j].b, b[u][j]);
      }
      op += step;
    }
    cur = nxt;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < J; ++j) {
        a[u][j] = na[u][j];
        b[u][j] = nb[u][j];
      }
  }
}

// Gradients of the norms: persistent warps take (row, share) items in a fixed order, the query heads
// of all of them and then the key heads, and keep the weight gradients of their lanes' elements in
// registers; a CTA sums its warps in order and writes one partial per weight.  The next batch is not
// loaded ahead: that needs 168 registers, so 12 warps per SM instead of 16 (80 us against 62).
//   z = Rot^T(dy), u = z w, n = x r:  dx = r u - (r^2 mean(u n)) x,  dw += z n
template <typename T, int V, int J, bool INTER>
__global__ void __launch_bounds__(256, kGradCtas) norm_grad_kernel(const __grid_constant__ RotP p) {
  constexpr int U = J == 1 ? kGradBatch : 1;
  constexpr bool PAIRED = INTER || V == 1;
  using X = Vec<T, V>;
  extern __shared__ float red[];  // [warps][D]
  __shared__ uint64_t turns[kMaxPairs];
  __shared__ float2 angles[8][kMaxPairs];
  for (int i = threadIdx.x; i < p.half; i += blockDim.x) turns[i] = p.turns[i];
  __syncthreads();
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
  const int sub = lane & (p.L - 1), grp = lane >> p.logL, gpw = 32 >> p.logL;
  Unit un[J];
#pragma unroll
  for (int j = 0; j < J; ++j) un[j] = unit_of<V>(p, sub + j * p.L);
  const int64_t n_items = p.rows * p.parts, stride = (int64_t)gridDim.x * n_warps;
#pragma unroll 1
  for (int k = 0; k < p.classes; ++k) {
    const HeadsP& h = p.h[k];
    uint64_t dw[J][V], w[J][V];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const T* wp = static_cast<const T*>(h.w);
      widen<T, V>(wp && un[j].va ? X::load(wp + un[j].a) : X::zero(), wp && un[j].vb ? X::load(wp + un[j].b) : X::zero(),
                  w[j]);
      const float add = wp ? p.w_off : 1.f;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        w[j][e] = add_f32x2(w[j][e], pack_f32x2(add, add));
        dw[j][e] = 0;
      }
    }
    for (int64_t item = (int64_t)blockIdx.x * n_warps + warp; item < n_items; item += stride) {
      const int64_t row = p.parts == 1 ? item : item / p.parts;
      const int part = (int)(item - row * p.parts);
      const int lo = p.parts == 1 ? 0 : (int)((int64_t)part * h.its / p.parts);
      const int hi = p.parts == 1 ? h.its : (int)((int64_t)(part + 1) * h.its / p.parts);
      if (lo >= hi) continue;
      row_angles(p, turns, p.pos[row], angles[warp], lane);
      uint64_t fp[J][V], fq[J][V];
#pragma unroll
      for (int j = 0; j < J; ++j) unit_factors<V, PAIRED>(angles[warp], (sub + j * p.L) * V, p.half, fp[j], fq[j]);
      const int first = lo * gpw + grp;
      const T* xp = static_cast<const T*>(h.in) + row * h.in_row + first * h.in_head;
      const T* gp = static_cast<const T*>(h.g) + row * h.g_row + first * h.g_head;
      T* op = static_cast<T*>(h.out) + row * h.out_row + first * h.out_head;
      const int64_t x_step = gpw * h.in_head, g_step = gpw * h.g_head, out_step = gpw * h.out_head;
#pragma unroll 1
      for (int base = lo; base < hi; base += U) {
        typename X::R xa[U][J], xb[U][J], ga[U][J], gb[U][J];
        bool on[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          on[u] = base + u < hi && (base + u) * gpw + grp < h.heads;
#pragma unroll
          for (int j = 0; j < J; ++j) {
            xa[u][j] = on[u] && un[j].va ? X::load(xp + un[j].a) : X::zero();
            xb[u][j] = on[u] && un[j].vb ? X::load(xp + un[j].b) : X::zero();
            ga[u][j] = on[u] && un[j].va ? X::load(gp + un[j].a) : X::zero();
            gb[u][j] = on[u] && un[j].vb ? X::load(gp + un[j].b) : X::zero();
          }
          xp += x_step;
          gp += g_step;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (base + u >= hi) break;  // warp-uniform
          uint64_t x[J][V], z[J][V], ss2 = 0, dot2 = 0;
#pragma unroll
          for (int j = 0; j < J; ++j) {
            uint64_t g[V];
            widen<T, V>(xa[u][j], xb[u][j], x[j]);
            widen<T, V>(ga[u][j], gb[u][j], g);
            if (p.full) {
#pragma unroll
              for (int e = 0; e < V; ++e)
                z[j][e] = fma_f32x2(partner<V, PAIRED>(g, e), fq[j][e], mul_f32x2(g[e], fp[j][e]));
            } else {
#pragma unroll
              for (int e = 0; e < V; ++e)
                z[j][e] = turned<V, PAIRED, INTER>(un[j], e)
                              ? fma_f32x2(partner<V, PAIRED>(g, e), fq[j][e], mul_f32x2(g[e], fp[j][e]))
                              : g[e];
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
              ss2 = fma_f32x2(x[j][e], x[j][e], ss2);
              dot2 = fma_f32x2(mul_f32x2(z[j][e], w[j][e]), x[j][e], dot2);
            }
          }
          const float2 s2 = unpack_f32x2(ss2), d2 = unpack_f32x2(dot2);
          float ss = s2.x + s2.y, dot = d2.x + d2.y;
          for (int o = p.L >> 1; o > 0; o >>= 1) {
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
            dot += __shfl_xor_sync(0xffffffffu, dot, o);
          }
          // lanes without a head add nothing to the weight sums (eps may be 0)
          const float inv = on[u] ? rsqrtf(fmaf(ss, p.inv_d, p.eps)) : 0.f;
          const float pull = -inv * inv * (dot * inv * p.inv_d);  // -r^2 mean(u n)
          const uint64_t inv2 = pack_f32x2(inv, inv), pull2 = pack_f32x2(pull, pull);
#pragma unroll
          for (int j = 0; j < J; ++j) {
            uint64_t dx[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const uint64_t zr = mul_f32x2(z[j][e], inv2);
              dw[j][e] = fma_f32x2(zr, x[j][e], dw[j][e]);
              dx[e] = fma_f32x2(zr, w[j][e], mul_f32x2(x[j][e], pull2));
            }
            typename X::R oa, ob;
            narrow<T, V>(dx, oa, ob);
            if (on[u] && un[j].va) X::store(op + un[j].a, oa);
            if (on[u] && un[j].vb) X::store(op + un[j].b, ob);
          }
          op += out_step;
        }
      }
    }
    if (!p.dw_part) continue;
    if (k) __syncthreads();  // the sums of the query heads are read
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float2 v = unpack_f32x2(dw[j][e]);
        for (int o = 16; o >= p.L; o >>= 1) {  // the warp's heads
          v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
          v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
        }
        // pair e holds elements 2e, 2e + 1 of the unit's 2V (first vector, second vector)
        if (grp == 0 && (2 * e < V ? un[j].va : un[j].vb))
          red[warp * p.D + (2 * e < V ? un[j].a + 2 * e : un[j].b + 2 * e - V)] = v.x;
        if (grp == 0 && (2 * e + 1 < V ? un[j].va : un[j].vb))
          red[warp * p.D + (2 * e + 1 < V ? un[j].a + 2 * e + 1 : un[j].b + 2 * e + 1 - V)] = v.y;
      }
    __syncthreads();
    for (int i = threadIdx.x; i < p.D; i += blockDim.x) {
      float v = 0.f;
      for (int q = 0; q < n_warps; ++q) v += red[q * p.D + i];
      p.dw_part[((int64_t)blockIdx.x * 2 + k) * p.D + i] = v;
    }
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
  return (int)std::max<int64_t>(1, std::min<int64_t>((warps + 7) / 8, kGradCtas * sm_count()));
}

template <typename T, int V, int J>
cudaError_t launch_forward(const RotP& p, bool norm, cudaStream_t s) {
  const int64_t warps = p.rows * p.parts;
  // few warps: a small CTA on each of many SMs (40 bf16 heads of 128, 1 to 16 rows: 3.0-3.2 us, in CTAs of 8 warps
  // 3.4-3.5); many: 8 warps per CTA, persistent, kRotCtas CTAs per SM
  const int wpc = warps >= 8LL * sm_count() ? 8 : (int)std::max<int64_t>(1, warps / sm_count());
  const dim3 grid((unsigned)std::min<int64_t>((warps + wpc - 1) / wpc, kRotCtas * sm_count()));
  auto kern = norm ? (p.interleaved ? rotate_kernel<T, V, J, true, true> : rotate_kernel<T, V, J, true, false>)
                   : (p.interleaved ? rotate_kernel<T, V, J, false, true> : rotate_kernel<T, V, J, false, false>);
  return launch_pdl(kern, grid, dim3(32 * wpc), 0, s, p);
}

template <typename T, int V, int J>
cudaError_t launch_backward(const RotP& p, int ctas, cudaStream_t s) {
  const size_t sm = 8 * (size_t)p.D * sizeof(float);
  auto kern = p.interleaved ? norm_grad_kernel<T, V, J, true> : norm_grad_kernel<T, V, J, false>;
  return launch_pdl(kern, dim3(ctas), dim3(256), sm, s, p);
}

template <typename T>
cudaError_t launch_typed(const RotP& p, int v, int mode, int ctas, cudaStream_t s) {
  constexpr int W = 16 / (int)sizeof(T);
  if (v == W) return mode == 2 ? launch_backward<T, W, 1>(p, ctas, s) : launch_forward<T, W, 1>(p, mode == 1, s);
  if constexpr (sizeof(T) == 2)
    if (v == 4) return mode == 2 ? launch_backward<T, 4, 1>(p, ctas, s) : launch_forward<T, 4, 1>(p, mode == 1, s);
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
  p.full = r.rot_dim == r.head_dim;
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
    p.classes = i + 1;
  }
  // Shares of a row.  Fewer rows than persistent warps (2368 here): as many as give every warp work.  Beyond, whole
  // rows, since each share makes the row's angles and factors again: more of them, up to 14208 warps,
  // cost 40 bf16 heads of 128 (10 iterations) 39.7 against 30.6 us at 6000 rows normalised and rotated and 33.9
  // against 26.5 rotated alone.  But long rows (20 iterations were measured) go in two shares where that saves
  // half of the last of up to four rounds: 3000, 5001 and 8193 rows of 40 fp32 heads of 128 rotated in 26.4, 41.7
  // and 61.3 us against 29.5, 43.7 and 63.8, normalised too 29.7, 46.5 and 66.5 against 34.1, 48.8 and 68.6,
  // of 80 bf16 heads rotated 27.8, 43.2 and 63.2 against 31.4, 44.4 and 65.5; where it saves none they lose (4000 and
  // 6000 rows in fp32 34.2 and 48.7 against 32.6 and 48.0), and the gradients lose throughout.
  const int64_t warps = 16LL * sm_count(), rounds = (p.rows + warps - 1) / warps;
  const bool halves = c.mode != 2 && p.its >= 20 && rounds >= 2 && rounds <= 4 && (2 * p.rows + warps - 1) / warps < 2 * rounds;
  const int64_t want = halves ? 2 * p.rows : warps;
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
