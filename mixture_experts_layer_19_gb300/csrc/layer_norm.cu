// layer_norm.cu -- layer norm forward and backward over row-major [rows, d].
//
// Bound by HBM: the forward reads x and writes y, the backward reads x and dy
// and writes dx, each once.  A row stays in registers from its only read to
// its result, so the two passes of the variance -- mean first, then squares
// about it, which does not cancel as a difference of sums would -- cost no
// second read.
//   many rows, forward   one to four warps per row, the row packed in up to 16
//                        vectors of 16 bytes per lane, weights in shared
//                        memory; with one warp there is no barrier at all
//   narrow rows, forward  several rows per warp, four sets of them in flight
//   few rows             one block per row
//   odd widths           one element per access; the backward copies the aligned
//                        16-byte chunks that cover a row
//   backward             one block per row; each thread keeps its columns'
//                        sums of dw and db in registers over all its rows and
//                        prefetches later rows into its own shared memory
//   rows past 8192 elements are read again instead of kept
//   fp32 rows whose mean is far from zero beside their spread: rare, read again
// The backward's per-block column sums go to workspace once per block and are
// added in a fixed order by a second kernel: no atomics, bitwise repeatable.
// Measured, bf16 with fp32 weights: forward 16384 x 7168 80 us (5.9 TB/s),
// backward 113 us (6.3 TB/s); backward 4096 x 7168 38.4 us, 131072 x 256 forward
// 30 us (4.5 TB/s).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "kernels.h"
#include "moe.h"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxElems = 16;          // elements of a row per thread

template <class T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// VW elements of T moved as one access (16 bytes, or one element).
template <class T, int VW>
struct alignas(sizeof(T) * VW) Vec {
  T v[VW];
};

// VW weights as fp32, in accesses of up to 16 bytes.
template <class WT, int VW>
__device__ __forceinline__ void load_weights(const WT* p, float (&o)[VW]) {
  constexpr int N = VW * (int)sizeof(WT) > 16 ? 16 / (int)sizeof(WT) : VW;
#pragma unroll
  for (int k = 0; k < VW; k += N) {
    const Vec<WT, N> q = *reinterpret_cast<const Vec<WT, N>*>(p + k);
#pragma unroll
    for (int i = 0; i < N; ++i) o[k + i] = to_f(q.v[i]);
  }
}

// Sum of NV values over the block, the same on every thread.  `buf` alternates
// between calls so that one barrier per call is enough.
template <int NV>
__device__ __forceinline__ void block_sum(float (&s)[NV], float (*red)[NV], int nw) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
  if (nw == 1) return;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < NV; ++i) red[warp][i] = s[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) s[i] = 0.0f;
  for (int w = 0; w < nw; ++w)
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] += red[w][i];
}

// The mean of a row is off by a few units of its last place, which is far from nothing beside a small spread:
// rows of a constant 12345 came out as 0.3.  bf16 rows far from zero hold multiples of one unit, and their
// sum is exact up to 2^16 elements: mean_of, s times 1 / d corrected once by what it leaves of s, gives
// their mean to the last place.  An fp32 row whose mean is more than 16 spreads from zero is done over: the
// mean of the deviations corrects the mean, and the variance about it.  (Adding the deviations up beside
// the squares of every row cost 91 us instead of 82 at 16384 x 7168, bf16, and 36 instead of 29 at 131072 x 256;
// a division in place of the correction, 33.)
__device__ __forceinline__ float mean_of(float s, float d, float inv_d) {
  const float m = s * inv_d, c = fmaf(fmaf(-m, d, s), inv_d, m);
  return c == c ? c : m;                 // an infinite sum leaves no remainder
}
__device__ __forceinline__ bool mean_far(float m, float rs) { return fabsf(m * rs) > 16.0f; }
__device__ __forceinline__ void correct_mean(float dev, float& m, float& var) {
  m += dev;
  var = fmaf(-dev, dev, var);
  if (var < 0.0f) var = 0.0f;            // a NaN stays
}

template <class XT, class WT, int VW, int VPT>
__global__ void __launch_bounds__(kMaxThreads) ln_fwd_kernel(const XT* __restrict__ x, const WT* __restrict__ w,
                                                             const WT* __restrict__ b, int64_t rows, int d, float eps,
                                                             XT* __restrict__ y, float* __restrict__ mean,
                                                             float* __restrict__ rstd) {
  pdl_wait();
  pdl_release();
  using V = Vec<XT, VW>;
  __shared__ float red[3][16][1];
  const int vecs = d / VW, nw = blockDim.x >> 5, tid = threadIdx.x;
  const float inv_d = 1.0f / (float)d;
  float wr[VPT][VW], br[VPT][VW];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = tid + j * blockDim.x;
#pragma unroll
    for (int i = 0; i < VW; ++i) wr[j][i] = br[j][i] = 0.0f;
    if (c < vecs) {
      load_weights<WT, VW>(w + c * VW, wr[j]);
      if (b) load_weights<WT, VW>(b + c * VW, br[j]);
    }
  }
  V nx[VPT];
  int64_t r = blockIdx.x;
  auto fetch = [&](int64_t row) {
    const V* src = reinterpret_cast<const V*>(x + row * d);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = tid + j * blockDim.x;
      if (c < vecs) nx[j] = src[c];
    }
  };
  if (r < rows) fetch(r);
  for (; r < rows; r += gridDim.x) {
    float v[VPT][VW];
    float s[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const bool in = tid + j * blockDim.x < vecs;
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        v[j][i] = in ? to_f(nx[j].v[i]) : 0.0f;
        s[0] += v[j][i];
      }
    }
    if (r + gridDim.x < rows) fetch(r + gridDim.x);
    block_sum<1>(s, red[0], nw);
    float m = mean_of(s[0], (float)d, inv_d);
    float q[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const bool in = tid + j * blockDim.x < vecs;
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        v[j][i] -= m;
        if (in) q[0] = fmaf(v[j][i], v[j][i], q[0]);
      }
    }
    block_sum<1>(q, red[1], nw);
    float var = q[0] * inv_d, off = 0.0f;
    float rs = 1.0f / sqrtf(var + eps);
    if (mean_far(m, rs)) {
      q[0] = 0.0f;
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (tid + j * blockDim.x < vecs)
#pragma unroll
          for (int i = 0; i < VW; ++i) q[0] += v[j][i];
      block_sum<1>(q, red[2], nw);
      off = m;
      correct_mean(q[0] * inv_d, m, var);
      off = m - off;
      rs = 1.0f / sqrtf(var + eps);
    }
    V* dst = reinterpret_cast<V*>(y + r * d);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = tid + j * blockDim.x;
      if (c < vecs) {
        V o;
#pragma unroll
        for (int i = 0; i < VW; ++i) o.v[i] = from_f<XT>(fmaf((v[j][i] - off) * rs, wr[j][i], br[j][i]));
        dst[c] = o;
      }
    }
    if (tid == 0) {
      mean[r] = m;
      rstd[r] = rs;
    }
  }
}

// ---------------------------------------------------------------- packed fp32 pairs
using f2 = unsigned long long;
__device__ __forceinline__ f2 f2_make(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 f2_get(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// Pair p of a 16-byte vector of XT: 4 pairs of bf16 or 2 of fp32.
template <class XT>
struct Pairs;
template <>
struct Pairs<__nv_bfloat16> {
  static constexpr int n = 4;
  static __device__ __forceinline__ f2 get(const uint4& v, int p) {
    const uint32_t u = p == 0 ? v.x : p == 1 ? v.y : p == 2 ? v.z : v.w;
    return f2_make(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  static __device__ __forceinline__ void set(uint4& v, int p, f2 x) {
    const float2 f = f2_get(x);
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
    const uint32_t u = *reinterpret_cast<const uint32_t*>(&h);
    if (p == 0) v.x = u;
    else if (p == 1) v.y = u;
    else if (p == 2) v.z = u;
    else v.w = u;
  }
};
template <>
struct Pairs<float> {
  static constexpr int n = 2;
  static __device__ __forceinline__ f2 get(const uint4& v, int p) {
    return p == 0 ? f2_make(__uint_as_float(v.x), __uint_as_float(v.y))
                  : f2_make(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  static __device__ __forceinline__ void set(uint4& v, int p, f2 x) {
    const float2 f = f2_get(x);
    if (p == 0) {
      v.x = __float_as_uint(f.x);
      v.y = __float_as_uint(f.y);
    } else {
      v.z = __float_as_uint(f.x);
      v.w = __float_as_uint(f.y);
    }
  }
};
// Makes the packed row opaque between passes: the compiler would otherwise
// keep every element's fp32 form from pass to pass, twice the registers.
template <int NV>
__device__ __forceinline__ void keep_packed(uint4 (&v)[NV]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) asm volatile("" : "+r"(v[j].x), "+r"(v[j].y), "+r"(v[j].z), "+r"(v[j].w));
}
__device__ __forceinline__ float weight_at(const void* w, bool f32, int i) {
  return f32 ? reinterpret_cast<const float*>(w)[i] : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(w)[i]);
}

// ---------------------------------------------------------------- forward, many rows
// wpr (1, 2, 4) warps per row.  Shared memory holds
// (w, w, b, b) of each pair of columns, plane by plane so that neighbouring
// lanes read neighbouring 16 bytes.
// Warps per block (one block per SM): what the registers of NV packed vectors
// leave room for.
constexpr int row_warps(int nv) { return nv > 8 ? 16 : nv > 4 ? 24 : 32; }
template <class XT, int NV>
__global__ void __launch_bounds__(row_warps(NV) * 32, 1) ln_fwd_rows_kernel(const uint4* __restrict__ x, const void* w,
                                                                       const void* b, bool w_f32, int64_t rows, int d,
                                                                       int wpr, float eps, uint4* __restrict__ y,
                                                                       float* __restrict__ mean,
                                                                       float* __restrict__ rstd) {
  pdl_wait();
  pdl_release();
  using P = Pairs<XT>;
  constexpr int kRowWarps = row_warps(NV);
  extern __shared__ float4 wb[];                         // [P::n][vecs]
  __shared__ float red[4][kRowWarps];
  const int vecs = d / (2 * P::n);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < vecs * P::n; i += kRowWarps * 32) {
    const int c = i / P::n, p = i - c * P::n, e = 2 * i;
    wb[p * vecs + c] = make_float4(weight_at(w, w_f32, e), weight_at(w, w_f32, e + 1),
                                   b ? weight_at(b, w_f32, e) : 0.0f, b ? weight_at(b, w_f32, e + 1) : 0.0f);
  }
  __syncthreads();
  const int group = warp / wpr, gw = warp - group * wpr, groups = kRowWarps / wpr;
  const int tid = gw * 32 + lane, nt = wpr * 32;
  const float inv_d = 1.0f / (float)d;
  // sum over the row's warps, in warp order, the same on every lane
  auto row_sum = [&](float s, float* buf) {
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (wpr > 1) {
      if (lane == 0) buf[warp] = s;
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(nt) : "memory");
      s = 0.0f;
      for (int i = 0; i < wpr; ++i) s += buf[group * wpr + i];
    }
    return s;
  };
  // An fp32 row far from zero, from its first mean on.  Rare, so it is read again: keeping it in registers
  // for this would cost every row.
  [[maybe_unused]] auto redo = [&](int64_t r, float m) {
    const uint4* src = x + r * vecs;
    f2 s2 = f2_make(0, 0), c2 = s2;
    const f2 mm = f2_make(-m, -m);
#pragma unroll 1
    for (int c = tid; c < vecs; c += nt) {
      const uint4 u = src[c];
#pragma unroll
      for (int p = 0; p < P::n; ++p) {
        const f2 a = f2_add(P::get(u, p), mm);
        s2 = f2_fma(a, a, s2);
        c2 = f2_add(c2, a);
      }
    }
    const float2 s = f2_get(s2), t = f2_get(c2);
    float var = row_sum(s.x + s.y, red[2]) * inv_d;
    correct_mean(row_sum(t.x + t.y, red[3]) * inv_d, m, var);
    const float rs = 1.0f / sqrtf(var + eps);
#pragma unroll 1
    for (int c = tid; c < vecs; c += nt) {
      const uint4 u = src[c];
      uint4 o;
#pragma unroll
      for (int p = 0; p < P::n; ++p) {
        const float4 q = wb[p * vecs + c];
        P::set(o, p, f2_fma(f2_mul(f2_add(P::get(u, p), f2_make(-m, -m)), f2_make(rs, rs)), f2_make(q.x, q.y),
                            f2_make(q.z, q.w)));
      }
      __stcs(y + r * vecs + c, o);
    }
    if (tid == 0) {
      mean[r] = m;
      rstd[r] = rs;
    }
  };
  for (int64_t r = (int64_t)blockIdx.x * groups + group; r < rows; r += (int64_t)gridDim.x * groups) {
    const uint4* src = x + r * vecs;
    uint4 v[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = tid + j * nt;
      v[j] = c < vecs ? __ldcs(src + c) : make_uint4(0, 0, 0, 0);
    }
    f2 s2 = f2_make(0, 0), t2 = s2;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int p = 0; p < P::n; p += 2) {
        s2 = f2_add(s2, P::get(v[j], p));
        t2 = f2_add(t2, P::get(v[j], p + 1));
      }
    keep_packed<NV>(v);
    float2 s = f2_get(f2_add(s2, t2));
    const float m = mean_of(row_sum(s.x + s.y, red[0]), (float)d, inv_d);
    const f2 mm = f2_make(-m, -m);
    s2 = t2 = f2_make(0, 0);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (tid + j * nt < vecs) {
#pragma unroll
        for (int p = 0; p < P::n; p += 2) {
          const f2 a = f2_add(P::get(v[j], p), mm), c = f2_add(P::get(v[j], p + 1), mm);
          s2 = f2_fma(a, a, s2);
          t2 = f2_fma(c, c, t2);
        }
      }
    keep_packed<NV>(v);
    s = f2_get(f2_add(s2, t2));
    const float rs = 1.0f / sqrtf(row_sum(s.x + s.y, red[1]) * inv_d + eps);
    const f2 rr = f2_make(rs, rs);
    if (sizeof(XT) == 4 && mean_far(m, rs)) {
      redo(r, m);
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = tid + j * nt;
        if (c < vecs) {
          uint4 o;
#pragma unroll
          for (int p = 0; p < P::n; ++p) {
            const float4 q = wb[p * vecs + c];
            P::set(o, p, f2_fma(f2_mul(f2_add(P::get(v[j], p), mm), rr), f2_make(q.x, q.y), f2_make(q.z, q.w)));
          }
          __stcs(y + r * vecs + c, o);
        }
      }
      if (tid == 0) {
        mean[r] = m;
        rstd[r] = rs;
      }
    }
  }
}

// Narrow rows (at most 32 vectors): G lanes per row, 32 / G rows side by side
// in a warp and four such sets in flight; the weights stay in registers.  One
// row at a time leaves too few bytes in flight: 46.7 us at 131072 x 256
// against 31.9.
constexpr int kNarrowSets = 4;
template <class XT>
__global__ void __launch_bounds__(512, 2) ln_fwd_narrow_kernel(const uint4* __restrict__ x, const void* w,
                                                               const void* b, bool w_f32, int64_t rows, int d, int G,
                                                               float eps, uint4* __restrict__ y,
                                                               float* __restrict__ mean, float* __restrict__ rstd) {
  pdl_wait();
  pdl_release();
  using P = Pairs<XT>;
  const int vecs = d / (2 * P::n), lane = threadIdx.x & 31;
  const int c = lane & (G - 1), per = 32 / G;
  const bool in = c < vecs;
  const float inv_d = 1.0f / (float)d;
  f2 wr[P::n], br[P::n];
#pragma unroll
  for (int p = 0; p < P::n; ++p) {
    const int e = c * 2 * P::n + 2 * p;
    wr[p] = in ? f2_make(weight_at(w, w_f32, e), weight_at(w, w_f32, e + 1)) : f2_make(0, 0);
    br[p] = in && b ? f2_make(weight_at(b, w_f32, e), weight_at(b, w_f32, e + 1)) : f2_make(0, 0);
  }
  const int64_t warp = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 5) * per * kNarrowSets;
  for (int64_t r0 = warp * per * kNarrowSets + lane / G; r0 - lane / G < rows; r0 += step) {
    uint4 v[kNarrowSets];
    float s[kNarrowSets], m[kNarrowSets];
#pragma unroll
    for (int u = 0; u < kNarrowSets; ++u) {
      const int64_t r = r0 + u * per;
      v[u] = in && r < rows ? __ldcs(x + r * vecs + c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kNarrowSets; ++u) {
      f2 t = P::get(v[u], 0);
#pragma unroll
      for (int p = 1; p < P::n; ++p) t = f2_add(t, P::get(v[u], p));
      const float2 q = f2_get(t);
      s[u] = q.x + q.y;
    }
    for (int o = G >> 1; o; o >>= 1)
#pragma unroll
      for (int u = 0; u < kNarrowSets; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], o);
#pragma unroll
    for (int u = 0; u < kNarrowSets; ++u) {
      m[u] = mean_of(s[u], (float)d, inv_d);
      const f2 mm = f2_make(-m[u], -m[u]);
      f2 t = f2_make(0, 0);
#pragma unroll
      for (int p = 0; p < P::n; ++p) {
        const f2 a = f2_add(P::get(v[u], p), mm);
        t = f2_fma(a, a, t);
      }
      const float2 q = f2_get(t);
      s[u] = in ? q.x + q.y : 0.0f;
    }
    for (int o = G >> 1; o; o >>= 1)
#pragma unroll
      for (int u = 0; u < kNarrowSets; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], o);
    bool any = false;
#pragma unroll
    for (int u = 0; u < kNarrowSets; ++u) {
      const int64_t r = r0 + u * per;
      const float rs = 1.0f / sqrtf(s[u] * inv_d + eps);
      const bool far = sizeof(XT) == 4 && mean_far(m[u], rs);
      any |= far;
      const f2 rr = f2_make(rs, rs), mm = f2_make(-m[u], -m[u]);
      if (in && r < rows && !far) {
        uint4 o;
#pragma unroll
        for (int p = 0; p < P::n; ++p) P::set(o, p, f2_fma(f2_mul(f2_add(P::get(v[u], p), mm), rr), wr[p], br[p]));
        __stcs(y + r * vecs + c, o);
      }
      if (c == 0 && r < rows && !far) {
        mean[r] = m[u];
        rstd[r] = rs;
      }
    }
    if (!__any_sync(0xffffffffu, any)) continue;
    // rare, so the rows are read again, one set at a time; the sums of the same values come out the same
#pragma unroll 1
    for (int u = 0; u < kNarrowSets; ++u) {
      const int64_t r = r0 + u * per;
      const uint4 q = in && r < rows ? __ldcs(x + r * vecs + c) : make_uint4(0, 0, 0, 0);
      auto sum = [&](f2 t) {
        const float2 f = f2_get(t);
        float a = in ? f.x + f.y : 0.0f;
        for (int o = G >> 1; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
        return a;
      };
      f2 t = P::get(q, 0);
#pragma unroll
      for (int p = 1; p < P::n; ++p) t = f2_add(t, P::get(q, p));
      float mu = mean_of(sum(t), (float)d, inv_d);
      f2 sq = f2_make(0, 0), dev = sq;
#pragma unroll
      for (int p = 0; p < P::n; ++p) {
        const f2 a = f2_add(P::get(q, p), f2_make(-mu, -mu));
        sq = f2_fma(a, a, sq);
        dev = f2_add(dev, a);
      }
      float var = sum(sq) * inv_d;
      const bool far = mean_far(mu, 1.0f / sqrtf(var + eps));
      correct_mean(sum(dev) * inv_d, mu, var);
      if (!far || r >= rows) continue;
      const float rs = 1.0f / sqrtf(var + eps);
      if (in) {
        uint4 o;
#pragma unroll
        for (int p = 0; p < P::n; ++p)
          P::set(o, p, f2_fma(f2_mul(f2_add(P::get(q, p), f2_make(-mu, -mu)), f2_make(rs, rs)), wr[p], br[p]));
        __stcs(y + r * vecs + c, o);
      }
      if (c == 0) {
        mean[r] = mu;
        rstd[r] = rs;
      }
    }
  }
}

// ---------------------------------------------------------------- backward
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}

// DEPTH rows are prefetched with cp.async.  A thread reads from shared memory
// only what it copied there itself, so the copies need no barrier.  The two
// halves of a row's work -- its sums, then its dx -- are a step apart: a step
// adds up row k, then finishes row k - 1 from registers while the other warps'
// sums of row k arrive, and ends with the one barrier that row needs.  What
// bounds it is issuing: about 11 fp32 operations and the conversions per
// element, so everything per row that is not per element is kept out of the loop.
template <class XT, int VPT, int DEPTH>
__global__ void __launch_bounds__(kMaxThreads, 1) ln_bwd_rows_kernel(
    const uint4* __restrict__ dy, const uint4* __restrict__ x, const void* w, bool w_f32,
    const float* __restrict__ mean, const float* __restrict__ rstd, int64_t rows, int d,
    uint4* __restrict__ dx, float* __restrict__ part_w, float* __restrict__ part_b) {
  pdl_wait();
  pdl_release();
  using P = Pairs<XT>;
  extern __shared__ uint4 ring[];                        // [DEPTH][2][VPT * threads]
  __shared__ float2 red[2][32];                          // warps the block does not have stay 0
  __shared__ float2 stats[DEPTH][32];                    // (mean, rstd) of a row, copied by each warp for itself
  const int vecs = d / (2 * P::n), tid = threadIdx.x, nt = blockDim.x;
  if (tid < 32) red[0][tid] = red[1][tid] = make_float2(0.0f, 0.0f);
  __syncthreads();
  const int warp = tid >> 5, lane = tid & 31;
  const float inv_d = 1.0f / (float)d;
  f2 wr[VPT][P::n], aw[VPT][P::n], ab[VPT][P::n];
  bool in[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = tid + j * nt;
    in[j] = c < vecs;
    float wv[2 * P::n] = {};
    if (in[j]) {
      if (w_f32) load_weights<float, 2 * P::n>(reinterpret_cast<const float*>(w) + c * 2 * P::n, wv);
      else load_weights<__nv_bfloat16, 2 * P::n>(reinterpret_cast<const __nv_bfloat16*>(w) + c * 2 * P::n, wv);
    }
#pragma unroll
    for (int p = 0; p < P::n; ++p) {
      wr[j][p] = f2_make(wv[2 * p], wv[2 * p + 1]);
      aw[j][p] = ab[j][p] = f2_make(0, 0);
    }
    // slots of columns past the row stay zero: they add nothing
    if (!in[j])
      for (int k = 0; k < DEPTH; ++k)
        ring[((2 * k) * VPT + j) * nt + tid] = ring[((2 * k + 1) * VPT + j) * nt + tid] = make_uint4(0, 0, 0, 0);
  }
  const int mine = (int)((rows - blockIdx.x + gridDim.x - 1) / gridDim.x);    // rows blockIdx.x + k * gridDim.x
  const int64_t stride = (int64_t)gridDim.x * vecs;
  const uint4* fx = x + (int64_t)blockIdx.x * vecs + tid;
  const uint4* fg = dy + (int64_t)blockIdx.x * vecs + tid;
  uint4* out = dx + (int64_t)blockIdx.x * vecs + tid;
  const float* fs = (lane == 0 ? mean : rstd) + blockIdx.x;
  int to_fetch = mine;
  auto fetch = [&](uint4* slot, float2* st) {
    if (to_fetch > 0) {
      if (lane < 2) cp_async4(reinterpret_cast<float*>(st) + lane, fs);
      fs += gridDim.x;
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (in[j]) {
          cp_async16(slot + j * nt, fx + j * nt);
          cp_async16(slot + (VPT + j) * nt, fg + j * nt);
        }
      fx += stride;
      fg += stride;
      --to_fetch;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  uint4* const first = ring + tid;
  uint4* const past = first + DEPTH * 2 * VPT * nt;
  for (int k = 0; k < DEPTH; ++k) fetch(first + k * 2 * VPT * nt, &stats[k][warp]);
  uint4* slot = first;
  float2* st = &stats[0][warp];
  f2 px[VPT][P::n], pg[VPT][P::n];                       // row k - 1: x - mean, rstd g w
  float rs0 = 0.0f;                                      // rstd of row k - 1
#pragma unroll 2
  for (int k = 0; k <= mine; ++k) {
    const float* row_red = reinterpret_cast<const float*>(red[(k + 1) & 1]);
    // totals of row k - 1: lane l adds value (l & 1) of the warps l / 2 and l / 2 + 16
    float tot = 0.0f;
    if (dx && k > 0) {
      tot = row_red[lane] + row_red[lane + 32];
#pragma unroll
      for (int o = 2; o < 32; o <<= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
      // with s0 = rstd sum(g w), s1 = rstd sum(g w (x - mean)):
      // dx = rstd g w - s0 / d - (x - mean) rstd^2 s1 / d
      const float c1 = -__shfl_sync(0xffffffffu, tot, 0) * inv_d;
      const float c2 = -__shfl_sync(0xffffffffu, tot, 1) * inv_d * rs0 * rs0;
      const f2 k1 = f2_make(c1, c1), k2 = f2_make(c2, c2);
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        uint4 o;
#pragma unroll
        for (int p = 0; p < P::n; ++p) P::set(o, p, f2_fma(px[j][p], k2, f2_add(pg[j][p], k1)));
        if (in[j]) __stcs(out + j * nt, o);
      }
      out += stride;
    }
    if (k < mine) {
      asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
      __syncwarp();
      const float m = st->x, rs = st->y;
      __syncwarp();                                      // before lanes 0 and 1 copy over it
      const f2 rr = f2_make(rs, rs), mm = f2_make(-m, -m);
      f2 s0 = f2_make(0, 0), s1 = s0;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const uint4 vx = slot[j * nt], vg = slot[(VPT + j) * nt];
#pragma unroll
        for (int p = 0; p < P::n; ++p) {
          const f2 xm = f2_add(P::get(vx, p), mm), g = P::get(vg, p);
          const f2 gr = f2_mul(g, rr), gw = f2_mul(gr, wr[j][p]);
          s0 = f2_add(s0, gw);
          s1 = f2_fma(gw, xm, s1);
          aw[j][p] = f2_fma(gr, xm, aw[j][p]);
          ab[j][p] = f2_add(ab[j][p], g);
          px[j][p] = xm;
          pg[j][p] = gw;
        }
      }
      fetch(slot, st);
      slot += 2 * VPT * nt;
      st += 32;
      if (slot == past) {
        slot = first;
        st = &stats[0][warp];
      }
      rs0 = rs;
      const float2 a = f2_get(s0), c = f2_get(s1);
      const float t0 = a.x + a.y, t1 = c.x + c.y;
      // even lanes end with the sum of t0, odd lanes with that of t1
      float e = (lane & 1) ? t1 : t0;
      e += __shfl_xor_sync(0xffffffffu, (lane & 1) ? t0 : t1, 1);
#pragma unroll
      for (int o = 2; o < 32; o <<= 1) e += __shfl_xor_sync(0xffffffffu, e, o);
      if (lane < 2) reinterpret_cast<float*>(&red[k & 1][warp])[lane] = e;
    }
    __syncthreads();
  }
  if (!part_w) return;
  const int64_t base = (int64_t)blockIdx.x * d;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = tid + j * blockDim.x;
    if (c < vecs)
#pragma unroll
      for (int p = 0; p < P::n; ++p) {
        *reinterpret_cast<float2*>(part_w + base + c * 2 * P::n + 2 * p) = f2_get(aw[j][p]);
        *reinterpret_cast<float2*>(part_b + base + c * 2 * P::n + 2 * p) = f2_get(ab[j][p]);
      }
  }
}

// dw / db[c] = sum of the G per-block sums, in an order fixed by G: 32 slices
// of blocks, each in order, then the slices in order.  Block = 32 columns.
template <class WT>
__global__ void __launch_bounds__(1024) ln_cols_kernel(const float* __restrict__ part_w,
                                                       const float* __restrict__ part_b, int G, int d,
                                                       WT* __restrict__ dw, WT* __restrict__ db) {
  pdl_wait();
  pdl_release();
  __shared__ float sw[32][33], sb[32][33];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float a = 0.0f, b = 0.0f;
  if (c < d)
#pragma unroll 8
    for (int g = slice; g < G; g += 32) {
      a += part_w[(int64_t)g * d + c];
      b += part_b[(int64_t)g * d + c];
    }
  sw[slice][lane] = a;
  sb[slice][lane] = b;
  __syncthreads();
  if (slice < 2 && c < d) {
    float s = 0.0f;
    for (int i = 0; i < 32; ++i) s += slice ? sb[i][lane] : sw[i][lane];
    WT* out = slice ? db : dw;
    if (out) out[c] = from_f<WT>(s);
  }
}

// ---------------------------------------------------------------- odd widths
// Rows that do not start on 16-byte boundaries, many of them, forward: as
// ln_fwd_rows_kernel, one element per access.
constexpr int kOddElems = 32;                            // elements per lane
constexpr int kOddWarps = 20;
template <class XT>
__global__ void __launch_bounds__(kOddWarps * 32, 1) ln_fwd_odd_kernel(const XT* __restrict__ x, const void* w,
                                                                      const void* b, bool w_f32, int64_t rows, int d,
                                                                      int wpr, float eps, XT* __restrict__ y,
                                                                      float* __restrict__ mean,
                                                                      float* __restrict__ rstd) {
  pdl_wait();
  pdl_release();
  extern __shared__ float2 wb2[];                        // [d]
  __shared__ float red[3][kOddWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < d; i += kOddWarps * 32)
    wb2[i] = make_float2(weight_at(w, w_f32, i), b ? weight_at(b, w_f32, i) : 0.0f);
  __syncthreads();
  const int group = warp / wpr, gw = warp - group * wpr, groups = kOddWarps / wpr;
  const int tid = gw * 32 + lane, nt = wpr * 32;
  const float inv_d = 1.0f / (float)d;
  auto row_sum = [&](float s, float* buf) {
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (wpr > 1) {
      if (lane == 0) buf[warp] = s;
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(nt) : "memory");
      s = 0.0f;
      for (int i = 0; i < wpr; ++i) s += buf[group * wpr + i];
    }
    return s;
  };
  for (int64_t r = (int64_t)blockIdx.x * groups + group; r < rows; r += (int64_t)gridDim.x * groups) {
    const XT* src = x + r * d;
    float v[kOddElems], s = 0.0f;
#pragma unroll
    for (int j = 0; j < kOddElems; ++j) v[j] = tid + j * nt < d ? to_f(src[tid + j * nt]) : 0.0f;
#pragma unroll
    for (int j = 0; j < kOddElems; ++j) s += v[j];
    float m = mean_of(row_sum(s, red[0]), (float)d, inv_d);
    s = 0.0f;
#pragma unroll
    for (int j = 0; j < kOddElems; ++j) {
      v[j] -= m;
      if (tid + j * nt < d) s = fmaf(v[j], v[j], s);
    }
    float var = row_sum(s, red[1]) * inv_d;
    float rs = 1.0f / sqrtf(var + eps);
    if (sizeof(XT) == 2 || !mean_far(m, rs)) {
#pragma unroll
      for (int j = 0; j < kOddElems; ++j) {
        const int c = tid + j * nt;
        if (c < d) {
          const float2 q = wb2[c];
          y[r * d + c] = from_f<XT>(fmaf(v[j] * rs, q.x, q.y));
        }
      }
      if (tid == 0) {
        mean[r] = m;
        rstd[r] = rs;
      }
      continue;
    }
    // rare, so the row is read again
    s = 0.0f;
#pragma unroll 1
    for (int c = tid; c < d; c += nt) s += to_f(src[c]) - m;
    correct_mean(row_sum(s, red[2]) * inv_d, m, var);
    rs = 1.0f / sqrtf(var + eps);
#pragma unroll 1
    for (int c = tid; c < d; c += nt) {
      const float2 q = wb2[c];
      y[r * d + c] = from_f<XT>(fmaf((to_f(src[c]) - m) * rs, q.x, q.y));
    }
    if (tid == 0) {
      mean[r] = m;
      rstd[r] = rs;
    }
  }
}

// Backward: as ln_bwd_rows_kernel, but rows are copied as the aligned 16-byte
// chunks that cover them and read element by element, so threads read what
// others copied: the step's barrier also publishes the next row.
template <class XT, int EPT, int DEPTH>
__global__ void __launch_bounds__(kMaxThreads, 1) ln_bwd_odd_kernel(
    const XT* __restrict__ dy, const XT* __restrict__ x, const void* w, bool w_f32, const float* __restrict__ mean,
    const float* __restrict__ rstd, int64_t rows, int d, XT* __restrict__ dx, float* __restrict__ part_w,
    float* __restrict__ part_b) {
  pdl_wait();
  pdl_release();
  extern __shared__ uint4 ring[];                        // [DEPTH][2][chunks]
  __shared__ float2 red[2][32];                          // warps the block does not have stay 0
  __shared__ float2 stats[DEPTH];
  const int tid = threadIdx.x, nt = blockDim.x, warp = tid >> 5, lane = tid & 31;
  const int64_t row_bytes = (int64_t)d * sizeof(XT), all_bytes = rows * row_bytes;
  const int chunks = (int)(row_bytes / 16) + 2;
  const float inv_d = 1.0f / (float)d;
  float wr[EPT], aw[EPT], ab[EPT], px[EPT], pg[EPT];
#pragma unroll
  for (int j = 0; j < EPT; ++j) {
    const int c = tid + j * nt;
    wr[j] = c < d ? weight_at(w, w_f32, c) : 0.0f;
    aw[j] = ab[j] = 0.0f;
  }
  if (tid < 32) red[0][tid] = red[1][tid] = make_float2(0.0f, 0.0f);
  const int mine = (int)((rows - blockIdx.x + gridDim.x - 1) / gridDim.x);    // rows blockIdx.x + k * gridDim.x
  auto fetch = [&](int k) {
    if (k < mine) {
      const int64_t row = blockIdx.x + (int64_t)k * gridDim.x;
      const int64_t at = row * row_bytes, start = at & ~int64_t(15);
      const int n = (int)((at + row_bytes - start + 15) / 16);
      uint4* slot = ring + (k % DEPTH) * 2 * chunks;
      for (int c = tid; c < n; c += nt) {
        const int64_t from = start + 16 * c;
        const int bytes = (int)min((int64_t)16, all_bytes - from);           // the tensor ends inside its last chunk
        const uint32_t dst = (uint32_t)__cvta_generic_to_shared(slot + c);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
                     "l"(reinterpret_cast<const char*>(x) + from), "r"(bytes)
                     : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 16 * chunks),
                     "l"(reinterpret_cast<const char*>(dy) + from), "r"(bytes)
                     : "memory");
      }
      if (tid < 2) cp_async4(reinterpret_cast<float*>(&stats[k % DEPTH]) + tid, (tid ? rstd : mean) + row);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int k = 0; k < DEPTH - 1; ++k) fetch(k);
  asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 2) : "memory");
  __syncthreads();
  float rs0 = 0.0f;                                      // rstd of row k - 1
  for (int k = 0; k <= mine; ++k) {
    fetch(k + DEPTH - 1);                                // into row k - 1's slot
    const int64_t row = blockIdx.x + (int64_t)k * gridDim.x;
    if (dx && k > 0) {
      const float* row_red = reinterpret_cast<const float*>(red[(k + 1) & 1]);
      float tot = row_red[lane] + row_red[lane + 32];
#pragma unroll
      for (int o = 2; o < 32; o <<= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
      const float c1 = __shfl_sync(0xffffffffu, tot, 0) * inv_d;
      const float c2 = __shfl_sync(0xffffffffu, tot, 1) * inv_d * rs0 * rs0;
      XT* out = dx + (row - gridDim.x) * d;
#pragma unroll
      for (int j = 0; j < EPT; ++j)
        if (tid + j * nt < d) out[tid + j * nt] = from_f<XT>(fmaf(-px[j], c2, pg[j] - c1));
    }
    if (k < mine) {
      const float2 q = stats[k % DEPTH];
      const float m = q.x, rs = q.y;
      const uint4* slot = ring + (k % DEPTH) * 2 * chunks;
      const int shift = (int)((row * row_bytes) & 15) / (int)sizeof(XT);
      const XT* sx = reinterpret_cast<const XT*>(slot) + shift;
      const XT* sg = reinterpret_cast<const XT*>(slot + chunks) + shift;
      float t0 = 0.0f, t1 = 0.0f;
#pragma unroll
      for (int j = 0; j < EPT; ++j) {
        const int c = tid + j * nt;
        if (c < d) {
          const float xm = to_f(sx[c]) - m, g = to_f(sg[c]);
          const float gr = g * rs, gw = gr * wr[j];
          t0 += gw;
          t1 = fmaf(gw, xm, t1);
          aw[j] = fmaf(gr, xm, aw[j]);
          ab[j] += g;
          px[j] = xm;
          pg[j] = gw;
        }
      }
      rs0 = rs;
      float e = (lane & 1) ? t1 : t0;
      e += __shfl_xor_sync(0xffffffffu, (lane & 1) ? t0 : t1, 1);
#pragma unroll
      for (int o = 2; o < 32; o <<= 1) e += __shfl_xor_sync(0xffffffffu, e, o);
      if (lane < 2) reinterpret_cast<float*>(&red[k & 1][warp])[lane] = e;
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 2) : "memory");
    __syncthreads();
  }
  if (!part_w) return;
  const int64_t base = (int64_t)blockIdx.x * d;
#pragma unroll
  for (int j = 0; j < EPT; ++j) {
    const int c = tid + j * nt;
    if (c < d) {
      part_w[base + c] = aw[j];
      part_b[base + c] = ab[j];
    }
  }
}

// ---- rows that do not fit the registers: the row is read once per pass
template <class XT, class WT>
__global__ void __launch_bounds__(512) ln_fwd_long_kernel(const XT* __restrict__ x, const WT* __restrict__ w,
                                                          const WT* __restrict__ b, int64_t rows, int64_t d, float eps,
                                                          XT* __restrict__ y, float* __restrict__ mean,
                                                          float* __restrict__ rstd) {
  pdl_wait();
  pdl_release();
  __shared__ float red[3][16][1];
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const XT* src = x + r * d;
    float s[1] = {0.0f}, q[1] = {0.0f};
    for (int64_t c = threadIdx.x; c < d; c += 512) s[0] += to_f(src[c]);
    block_sum<1>(s, red[0], 16);
    float m = s[0] / (float)d;
    for (int64_t c = threadIdx.x; c < d; c += 512) {
      const float v = to_f(src[c]) - m;
      q[0] = fmaf(v, v, q[0]);
    }
    block_sum<1>(q, red[1], 16);
    float var = q[0] / (float)d;
    float rs = 1.0f / sqrtf(var + eps);
    if (mean_far(m, rs)) {
      s[0] = 0.0f;
      for (int64_t c = threadIdx.x; c < d; c += 512) s[0] += to_f(src[c]) - m;
      block_sum<1>(s, red[2], 16);
      correct_mean(s[0] / (float)d, m, var);
      rs = 1.0f / sqrtf(var + eps);
    }
    for (int64_t c = threadIdx.x; c < d; c += 512)
      y[r * d + c] = from_f<XT>(fmaf((to_f(src[c]) - m) * rs, to_f(w[c]), b ? to_f(b[c]) : 0.0f));
    if (threadIdx.x == 0) {
      mean[r] = m;
      rstd[r] = rs;
    }
  }
}

template <class XT, class WT>
__global__ void __launch_bounds__(512) ln_bwd_long_kernel(const XT* __restrict__ dy, const XT* __restrict__ x,
                                                          const WT* __restrict__ w, const float* __restrict__ mean,
                                                          const float* __restrict__ rstd, int64_t rows, int64_t d,
                                                          XT* __restrict__ dx) {
  pdl_wait();
  pdl_release();
  __shared__ float red[2][16][2];
  int flip = 0;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const XT *sx = x + r * d, *sg = dy + r * d;
    const float m = mean[r], rs = rstd[r];
    float s[2] = {0.0f, 0.0f};
    for (int64_t c = threadIdx.x; c < d; c += 512) {
      const float gw = to_f(sg[c]) * to_f(w[c]);
      s[0] += gw;
      s[1] = fmaf(gw, (to_f(sx[c]) - m) * rs, s[1]);
    }
    block_sum<2>(s, red[flip], 16);
    flip ^= 1;
    const float c1 = s[0] / (float)d, c2 = s[1] / (float)d;
    for (int64_t c = threadIdx.x; c < d; c += 512)
      dx[r * d + c] = from_f<XT>(rs * (to_f(sg[c]) * to_f(w[c]) - c1 - (to_f(sx[c]) - m) * rs * c2));
  }
}

// Column sums of one slice of rows: thread = column, blockIdx.y = slice.
template <class XT>
__global__ void __launch_bounds__(256) ln_bwd_long_cols_kernel(const XT* __restrict__ dy, const XT* __restrict__ x,
                                                               const float* __restrict__ mean,
                                                               const float* __restrict__ rstd, int64_t rows, int64_t d,
                                                               float* __restrict__ part_w, float* __restrict__ part_b) {
  pdl_wait();
  pdl_release();
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= d) return;
  const int64_t lo = rows * blockIdx.y / gridDim.y, hi = rows * (blockIdx.y + 1) / gridDim.y;
  float a = 0.0f, b = 0.0f;
  for (int64_t r = lo; r < hi; ++r) {
    const float g = to_f(dy[r * d + c]);
    a = fmaf(g, (to_f(x[r * d + c]) - mean[r]) * rstd[r], a);
    b += g;
  }
  part_w[blockIdx.y * d + c] = a;
  part_b[blockIdx.y * d + c] = b;
}

// ---------------------------------------------------------------- host side
struct Shape {
  bool reg;        // the row fits the registers
  int vw, vpt, threads;
};

// Elements per access: 16 bytes when every row starts on a 16-byte boundary,
// else one.  Accesses per thread: the fewest (a power of two) that cover the row
// with 512 threads.
Shape shape_of(int64_t d, int esize) {
  Shape s{};
  s.vw = (d * esize) % 16 == 0 ? 16 / esize : 1;
  const int64_t vecs = d / s.vw;
  for (s.vpt = 1; s.vpt * s.vw <= kMaxElems; s.vpt *= 2)
    if ((vecs + s.vpt - 1) / s.vpt <= kMaxThreads) {
      s.reg = true;
      s.threads = (int)(((vecs + s.vpt - 1) / s.vpt + 31) / 32 * 32);
      return s;
    }
  return s;
}

int current_sms() {
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return std::max(1, sms);
}

// The backward: 16 elements per thread, or fewer where that would leave a
// block with less than two warps.
Shape bwd_shape(int64_t d, int esize) {
  Shape s = shape_of(d, esize);
  if (!s.reg) return s;
  const int64_t vecs = d / s.vw;
  if (s.vw == 1) s.vpt = d <= 128 ? 4 : kMaxElems;
  else s.vpt = vecs < 128 ? 1 : kMaxElems / s.vw;
  s.threads = (int)(((vecs + s.vpt - 1) / s.vpt + 31) / 32 * 32);
  return s;
}

// Blocks of the persistent kernels; the backward's number of column partials.
int64_t fwd_blocks(int64_t rows, const Shape& s, int sms) {
  return std::min<int64_t>(rows, (int64_t)sms * std::max(1, std::min(16, 2048 / s.threads)));
}
int64_t bwd_blocks(int64_t rows, int threads, int sms) {
  return std::min<int64_t>(rows, (int64_t)sms * std::max(1, std::min(8, 512 / threads)));
}
int64_t long_slices(int64_t rows) { return std::min<int64_t>(rows, 32); }

// Leave for a launch's dynamic shared memory.  What needs none is 48 KB with the
// kernel's static part, up to 2.3 KB here.  Always the same maximum (with the static
// part below the 227 KB of a block): one call never lowers what another, on some
// other thread, is about to launch with.
constexpr int kMaxSmem = 224 << 10;
template <class K>
cudaError_t allow_smem(K kernel, int bytes) {
  if (bytes <= 44 << 10) return cudaSuccess;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
}

template <class XT, class WT, int VW, int VPT>
cudaError_t fwd_go(const void* x, const void* w, const void* b, int64_t rows, int d, float eps, void* y, float* mean,
                   float* rstd, const Shape& s, int sms, cudaStream_t st) {
  return launch_pdl(ln_fwd_kernel<XT, WT, VW, VPT>, dim3((unsigned)fwd_blocks(rows, s, sms)), dim3(s.threads), 0, st, 1,
                    (const XT*)x, (const WT*)w, (const WT*)b, rows, d, eps, (XT*)y, mean, rstd);
}
// Forward over many rows: the fewest warps per row (1, 2, 4) whose lanes hold
// it in 16 vectors, and how many vectors that takes (28 vectors and half the warps:
// 92 us against 84 at 16384 x 7168).  0 warps: not possible.
struct RowPlan {
  int wpr, nv;
};
RowPlan row_plan(int64_t d, int esize) {
  if ((d * esize) % 16 != 0) return {0, 0};
  const int64_t vecs = d * esize / 16;
  for (int wpr = 1; wpr <= 4; wpr *= 2) {
    const int64_t nv = (vecs + 32 * wpr - 1) / (32 * wpr);
    if (nv <= 16) return {wpr, (int)nv};
  }
  return {0, 0};
}

template <class XT, int NV>
cudaError_t fwd_rows_go(const void* x, const void* w, const void* b, bool w_f32, int64_t rows, int d, int wpr,
                        float eps, void* y, float* mean, float* rstd, int sms, cudaStream_t st) {
  const int smem = d * 8;
  auto kernel = ln_fwd_rows_kernel<XT, NV>;
  cudaError_t e = allow_smem(kernel, smem);
  if (e != cudaSuccess) return e;
  constexpr int kRowWarps = row_warps(NV);
  const int64_t groups = kRowWarps / wpr;
  return launch_pdl(kernel, dim3((unsigned)std::min<int64_t>((rows + groups - 1) / groups, sms)), dim3(kRowWarps * 32),
                    smem, st, 1, (const uint4*)x, w, b, w_f32, rows, d, wpr, eps, (uint4*)y, mean, rstd);
}

template <class XT, int VPT, int DEPTH>
cudaError_t bwd_depth_go(const void* dy, const void* x, const void* w, bool w_f32, const float* mean, const float* rstd,
                         int64_t rows, int d, void* dx, float* pw, float* pb, const Shape& s, int64_t blocks,
                         cudaStream_t st) {
  const int smem = DEPTH * 2 * VPT * s.threads * 16;
  auto kernel = ln_bwd_rows_kernel<XT, VPT, DEPTH>;
  cudaError_t e = allow_smem(kernel, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3((unsigned)blocks), dim3(s.threads), smem, st, 1, (const uint4*)dy, (const uint4*)x, w,
                    w_f32, mean, rstd, rows, d, (uint4*)dx, pw, pb);
}
// As many rows in flight as shared memory has room for, up to 7.
template <class XT, int VPT>
cudaError_t bwd_rows_go(const void* dy, const void* x, const void* w, bool w_f32, const float* mean, const float* rstd,
                        int64_t rows, int d, void* dx, float* pw, float* pb, const Shape& s, int64_t blocks,
                        cudaStream_t st) {
  const int per_sm = std::max(1, std::min(8, 512 / s.threads));
  const int fit = (220 << 10) / (2 * VPT * s.threads * 16) / per_sm;
  if (fit >= 7) return bwd_depth_go<XT, VPT, 7>(dy, x, w, w_f32, mean, rstd, rows, d, dx, pw, pb, s, blocks, st);
  if (fit >= 5) return bwd_depth_go<XT, VPT, 5>(dy, x, w, w_f32, mean, rstd, rows, d, dx, pw, pb, s, blocks, st);
  return bwd_depth_go<XT, VPT, 3>(dy, x, w, w_f32, mean, rstd, rows, d, dx, pw, pb, s, blocks, st);
}

template <class XT, int EPT, int DEPTH>
cudaError_t bwd_odd_depth_go(const void* dy, const void* x, const void* w, bool w_f32, const float* mean,
                             const float* rstd, int64_t rows, int d, void* dx, float* pw, float* pb, const Shape& s,
                             int64_t blocks, cudaStream_t st) {
  const int smem = DEPTH * 2 * (d * (int)sizeof(XT) / 16 + 2) * 16;
  auto kernel = ln_bwd_odd_kernel<XT, EPT, DEPTH>;
  cudaError_t e = allow_smem(kernel, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3((unsigned)blocks), dim3(s.threads), smem, st, 1, (const XT*)dy, (const XT*)x, w, w_f32,
                    mean, rstd, rows, d, (XT*)dx, pw, pb);
}
template <class XT, int EPT>
cudaError_t bwd_odd_go(const void* dy, const void* x, const void* w, bool w_f32, const float* mean, const float* rstd,
                       int64_t rows, int d, void* dx, float* pw, float* pb, const Shape& s, int64_t blocks,
                       cudaStream_t st) {
  // all of an SM's blocks at once: each has 1 KB taken by the system and its static part beside the rows, and
  // a block that has to wait starts when another has done all its rows (100000 x 691 fp32: 158 us against 239)
  const int per_sm = std::max(1, std::min(8, 512 / s.threads));
  const int room = std::min((220 << 10) / per_sm, (228 << 10) / per_sm - 2048);
  const int fit = room / (2 * (d * (int)sizeof(XT) / 16 + 2) * 16);
  return fit >= 5 ? bwd_odd_depth_go<XT, EPT, 5>(dy, x, w, w_f32, mean, rstd, rows, d, dx, pw, pb, s, blocks, st)
                  : bwd_odd_depth_go<XT, EPT, 3>(dy, x, w, w_f32, mean, rstd, rows, d, dx, pw, pb, s, blocks, st);
}

template <class XT>
cudaError_t fwd_narrow_go(const void* x, const void* w, const void* b, bool w_f32, int64_t rows, int d, float eps,
                          void* y, float* mean, float* rstd, int sms, cudaStream_t st) {
  const int vecs = d * (int)sizeof(XT) / 16;
  int G = 1;
  while (G < vecs) G <<= 1;
  const int64_t per_block = 16 * (32 / G) * kNarrowSets;
  return launch_pdl(ln_fwd_narrow_kernel<XT>,
                    dim3((unsigned)std::min<int64_t>((rows + per_block - 1) / per_block, 2 * sms)), dim3(512), 0, st, 1,
                    (const uint4*)x, w, b, w_f32, rows, d, G, eps, (uint4*)y, mean, rstd);
}

template <class XT>
cudaError_t fwd_odd_go(const void* x, const void* w, const void* b, bool w_f32, int64_t rows, int d, int wpr, float eps,
                       void* y, float* mean, float* rstd, int sms, cudaStream_t st) {
  auto kernel = ln_fwd_odd_kernel<XT>;
  const int64_t groups = kOddWarps / wpr;
  cudaError_t e = allow_smem(kernel, d * 8);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3((unsigned)std::min<int64_t>((rows + groups - 1) / groups, sms)), dim3(kOddWarps * 32),
                    d * 8, st, 1, (const XT*)x, w, b, w_f32, rows, d, wpr, eps, (XT*)y, mean, rstd);
}

// Calls GO<XT, WT, VW, VPT>(args...) for the shape's access width and count.
#define LN_SCALAR(GO, ...)                                                    \
  do {                                                                        \
    if (s.vpt <= 2) return GO<XT, WT, 1, 2>(__VA_ARGS__);                     \
    if (s.vpt <= 4) return GO<XT, WT, 1, 4>(__VA_ARGS__);                     \
    if (s.vpt <= 8) return GO<XT, WT, 1, 8>(__VA_ARGS__);                     \
    return GO<XT, WT, 1, 16>(__VA_ARGS__);                                    \
  } while (0)
#define LN_DISPATCH(GO, ...)                                                  \
  do {                                                                        \
    constexpr int kFull = 16 / (int)sizeof(XT);                               \
    if (s.vw == kFull) {                                                      \
      if (s.vpt == 1) return GO<XT, WT, kFull, 1>(__VA_ARGS__);               \
      if (s.vpt == 2) return GO<XT, WT, kFull, 2>(__VA_ARGS__);               \
      return GO<XT, WT, kFull, kMaxElems / kFull>(__VA_ARGS__);               \
    }                                                                         \
    LN_SCALAR(GO, __VA_ARGS__);                                               \
  } while (0)

template <class XT, class WT>
cudaError_t fwd_types(const void* x, const void* w, const void* b, int64_t rows, int64_t d, float eps, void* y,
                      float* mean, float* rstd, cudaStream_t st) {
  const Shape s = shape_of(d, sizeof(XT));
  const int sms = current_sms();
  const RowPlan p = row_plan(d, sizeof(XT));
  if (p.wpr && d * (int64_t)sizeof(XT) <= 512 && rows >= 512)
    return fwd_narrow_go<XT>(x, w, b, sizeof(WT) == 4, rows, (int)d, eps, y, mean, rstd, sms, st);
  // many rows: enough to give 12 warps of every SM work; few are split over a block each instead
  if (p.wpr && rows * p.wpr >= (int64_t)sms * 12) {
    const bool wf = sizeof(WT) == 4;
    if (p.nv <= 4) return fwd_rows_go<XT, 4>(x, w, b, wf, rows, (int)d, p.wpr, eps, y, mean, rstd, sms, st);
    if (p.nv <= 8) return fwd_rows_go<XT, 8>(x, w, b, wf, rows, (int)d, p.wpr, eps, y, mean, rstd, sms, st);
    return fwd_rows_go<XT, 16>(x, w, b, wf, rows, (int)d, p.wpr, eps, y, mean, rstd, sms, st);
  }
  if (!p.wpr && d <= 4 * 32 * kOddElems && rows >= (int64_t)sms * 12) {
    const int wpr = d <= 32 * kOddElems ? 1 : d <= 64 * kOddElems ? 2 : 4;
    return fwd_odd_go<XT>(x, w, b, sizeof(WT) == 4, rows, (int)d, wpr, eps, y, mean, rstd, sms, st);
  }
  if (s.reg) LN_DISPATCH(fwd_go, x, w, b, rows, (int)d, eps, y, mean, rstd, s, sms, st);
  return launch_pdl(ln_fwd_long_kernel<XT, WT>, dim3((unsigned)std::min<int64_t>(rows, 4 * sms)), dim3(512), 0, st, 1,
                    (const XT*)x, (const WT*)w, (const WT*)b, rows, d, eps, (XT*)y, mean, rstd);
}

template <class XT, class WT>
cudaError_t bwd_rows(const void* dy, const void* x, const void* w, const float* mean, const float* rstd, int64_t rows,
                     int64_t d, void* dx, float* pw, float* pb, const Shape& s, int64_t blocks, cudaStream_t st) {
  if (s.reg && s.vw > 1) {
    const bool wf = sizeof(WT) == 4;
    constexpr int kWide = kMaxElems * (int)sizeof(XT) / 16;
    return s.vpt == 1 ? bwd_rows_go<XT, 1>(dy, x, w, wf, mean, rstd, rows, (int)d, dx, pw, pb, s, blocks, st)
                      : bwd_rows_go<XT, kWide>(dy, x, w, wf, mean, rstd, rows, (int)d, dx, pw, pb, s, blocks, st);
  }
  if (s.reg)
    return s.vpt == 4
               ? bwd_odd_go<XT, 4>(dy, x, w, sizeof(WT) == 4, mean, rstd, rows, (int)d, dx, pw, pb, s, blocks, st)
               : bwd_odd_go<XT, 16>(dy, x, w, sizeof(WT) == 4, mean, rstd, rows, (int)d, dx, pw, pb, s, blocks, st);
  cudaError_t e = cudaSuccess;
  if (dx) {
    e = launch_pdl(ln_bwd_long_kernel<XT, WT>, dim3((unsigned)std::min<int64_t>(rows, 4 * current_sms())), dim3(512), 0,
                   st, 1, (const XT*)dy, (const XT*)x, (const WT*)w, mean, rstd, rows, d, (XT*)dx);
  }
  if (e == cudaSuccess && pw) {
    e = launch_pdl(ln_bwd_long_cols_kernel<XT>, dim3((unsigned)((d + 255) / 256), (unsigned)blocks), dim3(256), 0, st,
                   1, (const XT*)dy, (const XT*)x, mean, rstd, rows, d, pw, pb);
  }
  return e;
}

int64_t partials_of(int64_t rows, int64_t d, int esize, int sms) {
  const Shape s = bwd_shape(d, esize);
  return s.reg ? bwd_blocks(rows, s.threads, sms) : long_slices(rows);
}

template <class XT, class WT>
cudaError_t bwd_types(const void* dy, const void* x, const void* w, const float* mean, const float* rstd, int64_t rows,
                      int64_t d, void* dx, void* dw, void* db, float* ws, cudaStream_t st) {
  const Shape s = bwd_shape(d, sizeof(XT));
  const int64_t G = partials_of(rows, d, sizeof(XT), current_sms());
  const bool sums = dw || db;
  float* pw = sums ? ws : nullptr;
  float* pb = sums ? ws + G * d : nullptr;
  cudaError_t e = bwd_rows<XT, WT>(dy, x, w, mean, rstd, rows, d, dx, pw, pb, s, G, st);
  if (e != cudaSuccess || !sums) return e;
  return launch_pdl(ln_cols_kernel<WT>, dim3((unsigned)((d + 31) / 32)), dim3(1024), 0, st, 1, pw, pb, (int)G, (int)d,
                    (WT*)dw, (WT*)db);
}

moe_status_t bad(const char* where, const char* what) {
  set_error_detail((std::string(where) + ": " + what).c_str());
  return MOE_ERR_INVALID_ARG;
}
moe_status_t done(const char* where, cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  set_error_detail((std::string(where) + ": launch: " + cudaGetErrorString(e)).c_str());
  return MOE_ERR_CUDA;
}
bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool sizes_ok(int64_t rows, int64_t d) {
  return rows >= 0 && d >= 1 && d <= (1 << 20) && rows <= ((int64_t)1 << 40) / d;
}

size_t workspace_of(int64_t rows, int64_t d) {
  if (rows == 0) return 0;
  const int sms = current_sms();
  const int64_t G = std::max(partials_of(rows, d, 2, sms), partials_of(rows, d, 4, sms));
  return (size_t)G * 2 * d * 4;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_layer_norm_forward(const void* x, const void* w, const void* b, int64_t rows, int64_t d,
                                    int32_t x_f32, int32_t w_f32, float eps, void* y, float* mean, float* rstd,
                                    moe_stream_t stream) {
  const char* where = "moe_layer_norm_forward";
  try {
    if (!sizes_ok(rows, d)) return bad(where, "need rows >= 0, 1 <= d <= 2^20 and rows * d <= 2^40");
    if (!(eps >= 0.0f && std::isfinite(eps))) return bad(where, "eps must be finite and not negative");
    if (rows == 0) return MOE_OK;
    if (!x || !w || !y || !mean || !rstd) return bad(where, "null pointer");
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(b, 16) || !aligned(y, 16) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
      return bad(where, "misaligned pointer (tensors 16 bytes)");
    (void)cudaGetLastError();
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    using bf = __nv_bfloat16;
    if (x_f32)
      return done(where, w_f32 ? fwd_types<float, float>(x, w, b, rows, d, eps, y, mean, rstd, st)
                               : fwd_types<float, bf>(x, w, b, rows, d, eps, y, mean, rstd, st));
    return done(where, w_f32 ? fwd_types<bf, float>(x, w, b, rows, d, eps, y, mean, rstd, st)
                             : fwd_types<bf, bf>(x, w, b, rows, d, eps, y, mean, rstd, st));
  } catch (...) {
    return MOE_ERR_INTERNAL;
  }
}

moe_status_t moe_layer_norm_workspace_bytes(int64_t rows, int64_t d, size_t* bytes) {
  const char* where = "moe_layer_norm_workspace_bytes";
  try {
    if (!bytes) return bad(where, "null argument");
    if (!sizes_ok(rows, d)) return bad(where, "need rows >= 0, 1 <= d <= 2^20 and rows * d <= 2^40");
    *bytes = workspace_of(rows, d);
    return MOE_OK;
  } catch (...) {
    return MOE_ERR_INTERNAL;
  }
}

moe_status_t moe_layer_norm_backward(const void* dy, const void* x, const void* w, const float* mean,
                                     const float* rstd, int64_t rows, int64_t d, int32_t x_f32, int32_t w_f32,
                                     void* dx, void* dw, void* db, void* workspace, size_t workspace_bytes,
                                     moe_stream_t stream) {
  const char* where = "moe_layer_norm_backward";
  try {
    if (!sizes_ok(rows, d)) return bad(where, "need rows >= 0, 1 <= d <= 2^20 and rows * d <= 2^40");
    if (!aligned(dx, 16) || !aligned(dw, 16) || !aligned(db, 16)) return bad(where, "misaligned output (16 bytes)");
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    (void)cudaGetLastError();
    if (rows == 0) {
      cudaError_t e = cudaSuccess;
      const size_t n = (size_t)d * (w_f32 ? 4 : 2);
      if (dw) e = cudaMemsetAsync(dw, 0, n, st);
      if (e == cudaSuccess && db) e = cudaMemsetAsync(db, 0, n, st);
      return done(where, e);
    }
    if (!dy || !x || !w || !mean || !rstd) return bad(where, "null pointer");
    if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(w, 16) || !aligned(mean, 4) || !aligned(rstd, 4))
      return bad(where, "misaligned pointer (tensors 16 bytes)");
    if (!dx && !dw && !db) return MOE_OK;
    if (dw || db) {
      if (!workspace || !aligned(workspace, 256)) return bad(where, "null or misaligned workspace (256 bytes)");
      if (workspace_bytes < workspace_of(rows, d))
        return bad(where, "workspace smaller than moe_layer_norm_workspace_bytes");
    }
    float* ws = static_cast<float*>(workspace);
    using bf = __nv_bfloat16;
    if (x_f32)
      return done(where, w_f32 ? bwd_types<float, float>(dy, x, w, mean, rstd, rows, d, dx, dw, db, ws, st)
                               : bwd_types<float, bf>(dy, x, w, mean, rstd, rows, d, dx, dw, db, ws, st));
    return done(where, w_f32 ? bwd_types<bf, float>(dy, x, w, mean, rstd, rows, d, dx, dw, db, ws, st)
                             : bwd_types<bf, bf>(dy, x, w, mean, rstd, rows, d, dx, dw, db, ws, st));
  } catch (...) {
    return MOE_ERR_INTERNAL;
  }
}

}  // extern "C"
