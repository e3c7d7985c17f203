// head_rows.cu -- the loss head's row kernels: which rows have a loss, the
// teacher's entries sorted by vocabulary id, the join of the per-tile softmax
// statistics into losses, and the last rounding of dX.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "head.h"
#include "ptx.cuh"

namespace moe {

namespace {

__device__ __forceinline__ int64_t load_id(const void* p, bool is64, int64_t i) {
  return is64 ? reinterpret_cast<const int64_t*>(p)[i] : (int64_t)reinterpret_cast<const int32_t*>(p)[i];
}

// One block per token.  Entry k is in use when its id lies in [0, V) and its
// teacher logit is not -inf.  p = softmax of the logits in use over the
// temperature; entries in use are stored by ascending id (ties by k), so that
// a tile finds its own by binary search and equal ids keep one order.
__global__ void __launch_bounds__(256) head_entries_kernel(const void* teacher, int teacher_bf16, const void* ids,
                                                           int ids64, int K, int Kp2, int64_t V, float inv_temp,
                                                           HeadRows r) {
  extern __shared__ unsigned long long key[];          // [Kp2] id * 2^11 + k, then probabilities
  float* u = reinterpret_cast<float*>(key + Kp2);      // [K]
  __shared__ float red[8];
  __shared__ float s_max, s_sum;
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, nt = blockDim.x, warp = tid >> 5, lane = tid & 31, nw = nt >> 5;
  float m = -CUDART_INF_F;
  bool nan = false;
  for (int k = tid; k < Kp2; k += nt) {
    unsigned long long kk = ~0ull;
    if (k < K) {
      const int64_t id = load_id(ids, ids64, t * K + k);
      float v = teacher_bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(teacher)[t * K + k])
                             : reinterpret_cast<const float*>(teacher)[t * K + k];
      v *= inv_temp;
      const bool use = id >= 0 && id < V && v != -CUDART_INF_F;
      u[k] = use ? v : -CUDART_INF_F;
      if (use) {
        kk = ((unsigned long long)id << 11) | (unsigned)k;
        m = fmaxf(m, v);
        nan |= v != v;
      }
    }
    key[k] = kk;
  }
  if (nan) m = CUDART_NAN_F;
  // max with NaN kept
  auto nmax = [](float a, float b) { return (a != a || b != b) ? CUDART_NAN_F : fmaxf(a, b); };
  for (int o = 16; o; o >>= 1) m = nmax(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red[warp] = m;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < nw; ++i) m = nmax(m, red[i]);
    s_max = m;
  }
  // bitonic sort of the keys, ascending
  for (int size = 2; size <= Kp2; size <<= 1)
    for (int stride = size >> 1; stride; stride >>= 1) {
      __syncthreads();
      for (int i = tid; i < Kp2 / 2; i += nt) {
        const int lo = 2 * i - (i & (stride - 1)), hi = lo + stride;
        const bool up = (lo & size) == 0;
        const unsigned long long a = key[lo], b = key[hi];
        if ((a > b) == up) {
          key[lo] = b;
          key[hi] = a;
        }
      }
    }
  __syncthreads();
  m = s_max;
  // a row without entries: m = -inf, no key in use
  float s = 0.0f;
  int c = 0;
  for (int k = tid; k < K; k += nt)
    if (key[k] != ~0ull) {
      s += expf(u[(unsigned)key[k] & 2047u] - m);
      ++c;
    }
  for (int o = 16; o; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    c += __shfl_xor_sync(0xffffffffu, c, o);
  }
  __shared__ int redc[8];
  if (lane == 0) {
    red[warp] = s;
    redc[warp] = c;
  }
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < nw; ++i) {
      s += red[i];
      c += redc[i];
    }
    s_sum = s;
    r.cnt[t] = c;
  }
  __syncthreads();
  s = s_sum;
  const float logs = logf(s);
  float h = 0.0f;
  for (int k = tid; k < K; k += nt) {
    const unsigned long long kk = key[k];
    if (kk == ~0ull) continue;
    const float x = u[(unsigned)kk & 2047u] - m;
    const float p = expf(x) / s;
    r.ids[t * K + k] = (int32_t)(kk >> 11);
    r.probs[t * K + k] = p;
    if (p != 0.0f) h += p * (x - logs);      // p log p
  }
  for (int o = 16; o; o >>= 1) h += __shfl_xor_sync(0xffffffffu, h, o);
  if (lane == 0) red[warp] = h;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < nw; ++i) h += red[i];
    r.plogp[t] = h;
  }
}

// One block: lists the rows that count, in token order, and (backward) the
// factor common to their upstream gradients: with one value for all of them
// (a mean) it is taken out of D before D is rounded to bf16.
__global__ void __launch_bounds__(1024) head_scan_kernel(const void* labels, int ids64, const float* dloss, int T,
                                                         int64_t V, HeadRows r) {
  __shared__ int wsum[32];
  __shared__ int s_base;
  __shared__ float smin[32], smax[32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) s_base = 0;
  float lo = CUDART_INF_F, hi = -CUDART_INF_F;
  bool odd = false;                                   // an upstream gradient that is not finite
  __syncthreads();
  for (int64_t t0 = 0; t0 < T; t0 += 1024) {
    const int64_t t = t0 + tid;
    bool on = false;
    if (t < T) {
      if (labels) {
        const int64_t id = load_id(labels, ids64, t);
        on = id >= 0 && id < V;
        r.ids[t] = on ? (int32_t)id : -1;
      } else {
        on = r.cnt[t] > 0;
      }
      if (dloss && on) {
        const float gv = dloss[t];
        on = gv != 0.0f;                              // NaN counts
        if (on) {
          odd |= !(fabsf(gv) < CUDART_INF_F);
          lo = fminf(lo, gv);
          hi = fmaxf(hi, gv);
        }
      }
    }
    const unsigned b = __ballot_sync(0xffffffffu, on);
    if (lane == 0) wsum[warp] = __popc(b);
    __syncthreads();
    if (warp == 0) {
      int v = wsum[lane];
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      wsum[lane] = v;
    }
    __syncthreads();
    const int pos = s_base + (warp ? wsum[warp - 1] : 0) + __popc(b & ((1u << lane) - 1u));
    if (t < T) {
      r.inv[t] = on ? pos : -1;
      if (on) r.rowmap[pos] = (int32_t)t;
    }
    __syncthreads();
    if (tid == 0) s_base += wsum[31];
    __syncthreads();
  }
  if (tid == 0) r.n_active[0] = s_base;
  if (!dloss) return;
  if (odd) lo = -CUDART_INF_F;
  for (int o = 16; o; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  if (lane == 0) {
    smin[warp] = lo;
    smax[warp] = hi;
  }
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < 32; ++i) {
      lo = fminf(lo, smin[i]);
      hi = fmaxf(hi, smax[i]);
    }
    *r.scale = lo == hi ? lo : 1.0f;
  }
}

// Compact copy of the rows that count, zero rows up to the next multiple of
// 256.  Nothing to do when every row counts (X is then read in place).
__global__ void __launch_bounds__(256) head_gather_kernel(const uint4* __restrict__ X, int T, int vecs, HeadRows r) {
  const int na = *r.n_active;
  if (na == T) return;
  const int rows = (na + kHeadRowPad - 1) / kHeadRowPad * kHeadRowPad;
  uint4* out = reinterpret_cast<uint4*>(r.Xc);
  for (int i = blockIdx.x; i < rows; i += gridDim.x) {
    const int64_t src = i < na ? r.rowmap[i] : -1;
    for (int c = threadIdx.x; c < vecs; c += blockDim.x)
      out[(int64_t)i * vecs + c] = src >= 0 ? X[src * vecs + c] : make_uint4(0, 0, 0, 0);
  }
}

// Joins the (max, sum) pairs of a row's 128-column blocks in block order
// inside 32 slices, then the slices in order, and writes the row's loss.  One block
// per 32 tokens: lane = token for the join (pairs of neighbouring rows are
// neighbours in memory), warp = token for the sum over the target entries.
__global__ void __launch_bounds__(1024) head_loss_kernel(int T, int K, int np, int64_t Tp, float temperature,
                                                         int distill, HeadRows r, float* loss, float* lse) {
  __shared__ float sm[32][33], ss[32][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * 32;
  {
    const int t = t0 + lane;
    const int row = t < T ? r.inv[t] : -1;
    float m = -CUDART_INF_F, s = 0.0f;
    if (row >= 0) {
      const int lo = (int)((int64_t)np * warp / 32), hi = (int)((int64_t)np * (warp + 1) / 32);
      for (int i = lo; i < hi; ++i) {
        const float2 p = r.part[i * Tp + row];
        const float mn = fmaxf(m, p.x);
        const float a = mn == -CUDART_INF_F ? 0.0f : mn;
        s = s * expf(m - a) + p.y * expf(p.x - a);
        m = mn;
      }
    }
    sm[warp][lane] = m;
    ss[warp][lane] = s;
  }
  __syncthreads();
  const int t = t0 + warp;
  if (t >= T) return;
  const int row = r.inv[t];
  if (row < 0) {
    if (lane == 0) {
      loss[t] = 0.0f;
      lse[t] = 0.0f;
    }
    return;
  }
  // slice `lane` of token `warp`
  float m = sm[lane][warp];
  const float s0 = ss[lane][warp];
  float mx = m;
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  float s = s0 * expf(m - (mx == -CUDART_INF_F ? 0.0f : mx));
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const float l = mx + logf(s);
  const float it = 1.0f / temperature;
  float out;
  if (distill) {
    const int cnt = r.cnt[t];
    float a = 0.0f;                               // sum p (lse - z / temperature)
    for (int k = lane; k < cnt; k += 32) {
      const float p = r.probs[(int64_t)t * K + k];
      if (p != 0.0f) a += p * (l - r.zt[(int64_t)t * K + k] * it);
    }
    for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    out = temperature * temperature * (r.plogp[t] + a);
  } else {
    out = l - r.zt[t];
  }
  if (lane == 0) {
    loss[t] = out;
    lse[t] = l;
  }
}

// dX[t] = factor * (sum over the splits, in order) for the rows that count, 0 elsewhere.
__global__ void __launch_bounds__(256) head_dx_kernel(int T, int d, int nsplit, int64_t Tp, float out_scale, HeadRows r,
                                                      uint2* __restrict__ dX) {
  const int vecs = d / 4;
  const float sc = *r.scale * out_scale;
  const float4* acc = reinterpret_cast<const float4*>(r.acc);
  const int64_t n = (int64_t)T * vecs;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t t = i / vecs;
    const int c = (int)(i - t * vecs);
    const int row = r.inv[t];
    uint2 o = make_uint2(0, 0);
    if (row >= 0) {
      float4 a = acc[(int64_t)row * vecs + c];
      for (int s = 1; s < nsplit; ++s) {
        const float4 b = acc[(s * Tp + row) * vecs + c];
        a.x += b.x;
        a.y += b.y;
        a.z += b.z;
        a.w += b.w;
      }
      o = make_uint2(pack_bf16(a.x * sc, a.y * sc), pack_bf16(a.z * sc, a.w * sc));
    }
    dX[i] = o;
  }
}

}  // namespace

cudaError_t launch_head_entries(const void* teacher, bool teacher_bf16, const void* ids, bool ids64, int T, int K,
                                int64_t V, float inv_temp, const HeadRows& r, cudaStream_t st) {
  int kp = 2;
  while (kp < K) kp <<= 1;
  int threads = 32;
  while (threads < kp / 2 && threads < 256) threads <<= 1;
  head_entries_kernel<<<T, threads, kp * 8 + K * 4, st>>>(teacher, teacher_bf16, ids, ids64, K, kp, V, inv_temp, r);
  return cudaGetLastError();
}

cudaError_t launch_head_scan(const void* labels, bool ids64, const float* dloss, int T, int64_t V, const HeadRows& r,
                             cudaStream_t st) {
  head_scan_kernel<<<1, 1024, 0, st>>>(labels, ids64, dloss, T, V, r);
  return cudaGetLastError();
}

cudaError_t launch_head_gather(const void* X, int T, int d, const HeadRows& r, int num_sms, cudaStream_t st) {
  const int rows = (T + kHeadRowPad - 1) / kHeadRowPad * kHeadRowPad;
  head_gather_kernel<<<rows < 8 * num_sms ? rows : 8 * num_sms, 256, 0, st>>>(reinterpret_cast<const uint4*>(X), T,
                                                                             d / 8, r);
  return cudaGetLastError();
}

cudaError_t launch_head_loss(int T, int K, int np, int64_t Tp, float temperature, bool distill, const HeadRows& r,
                             float* loss, float* lse, cudaStream_t st) {
  head_loss_kernel<<<(T + 31) / 32, 1024, 0, st>>>(T, K, np, Tp, temperature, distill, r, loss, lse);
  return cudaGetLastError();
}

cudaError_t launch_head_dx(int T, int d, int nsplit, int64_t Tp, float out_scale, const HeadRows& r, void* dX,
                           int num_sms, cudaStream_t st) {
  const int64_t n = ((int64_t)T * (d / 4) + 255) / 256;
  head_dx_kernel<<<(int)(n < 8 * num_sms ? n : 8 * num_sms), 256, 0, st>>>(T, d, nsplit, Tp, out_scale, r,
                                                                          reinterpret_cast<uint2*>(dX));
  return cudaGetLastError();
}

}  // namespace moe
