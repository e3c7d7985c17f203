// head_rows.cu -- the loss head's row kernels: which rows have a loss, the
// teacher's entries sorted by vocabulary id, the join of the per-tile softmax
// statistics into losses, and the last rounding of dX.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "head.h"
#include "pdl.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

__device__ __forceinline__ int64_t load_id(const void* p, bool is64, int64_t i) {
  return is64 ? reinterpret_cast<const int64_t*>(p)[i] : (int64_t)reinterpret_cast<const int32_t*>(p)[i];
}

// One block per token.  Entry k is in use when its id lies in [0, V) and its
// teacher logit is not -inf.  p = softmax of the logits in use over the
// temperature; entries in use are stored by ascending id (ties by k), so that
// a tile finds its own by binary search and equal ids keep one order.  What is
// scaled is a logit's distance to the largest one, which no temperature turns
// into infinity minus infinity: a mask of fp32's lowest value stays a finite logit.
__global__ void __launch_bounds__(256) head_entries_kernel(const void* teacher, int teacher_bf16, const void* ids,
                                                           int ids64, int K, int Kp2, int64_t V, float inv_temp,
                                                           HeadRows r) {
  extern __shared__ unsigned long long key[];          // [Kp2] id * 2^11 + k, then probabilities
  float* u = reinterpret_cast<float*>(key + Kp2);      // [K]
  __shared__ float red[8];
  __shared__ float s_max, s_sum;
  pdl_wait();
  pdl_release();
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, nt = blockDim.x, warp = tid >> 5, lane = tid & 31, nw = nt >> 5;
  float m = -CUDART_INF_F;
  bool nan = false;
  for (int k = tid; k < Kp2; k += nt) {
    unsigned long long kk = ~0ull;
    if (k < K) {
      const int64_t id = load_id(ids, ids64, t * K + k);
      const float v = teacher_bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(teacher)[t * K + k])
                                   : reinterpret_cast<const float*>(teacher)[t * K + k];
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
      s += expf((u[(unsigned)key[k] & 2047u] - m) * inv_temp);
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
    const float x = (u[(unsigned)kk & 2047u] - m) * inv_temp;
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
  // where each block of 128 vocabulary columns starts in the sorted list
  for (int64_t b = tid; b < r.blocks; b += nt) {
    const unsigned long long least = (unsigned long long)(128 * b) << 11;
    int at = 0;
    for (int step = Kp2 >> 1; step; step >>= 1)
      if (key[at + step - 1] < least) at += step;
    at += at < Kp2 && key[at] < least;
    r.first[t * r.blocks + b] = (uint16_t)at;
  }
}

__device__ __forceinline__ bool row_counts(const void* labels, bool ids64, const float* dloss, int64_t V,
                                           const HeadRows& r, int64_t t) {
  bool on;
  if (labels) {
    const int64_t id = load_id(labels, ids64, t);
    on = id >= 0 && id < V;
  } else {
    on = r.cnt[t] > 0;
  }
  return on && !(dloss && dloss[t] == 0.0f);          // a NaN gradient counts
}

// Lists the rows that count, in token order, and copies their rows of X
// together when some are left out (X is read in place otherwise); zero rows
// follow up to the next multiple of 256.  Every block walks all T tokens to
// know how many count before its own and in all -- a few bytes per token from L2,
// less than a second launch would cost -- and then serves its own range.
// (Backward) a factor common to all upstream gradients, as in a mean, is
// taken out of D before D is rounded to bf16.
__global__ void __launch_bounds__(256) head_prep_kernel(const void* labels, int ids64, const float* dloss,
                                                        const float* lse, int T, int64_t V,
                                                        const uint4* __restrict__ X, int vecs, HeadRows r,
                                                        uint4* __restrict__ dX) {
  __shared__ int s_cnt[8][2];
  __shared__ float s_lo[8], s_hi[8];
  __shared__ int s_on[256], s_off[256];                // tokens of the range that count, and that do not
  pdl_wait();
  pdl_release();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (T + gridDim.x - 1) / gridDim.x;
  const int t0 = min(T, (int)blockIdx.x * per), t1 = min(T, t0 + per);
  int before = 0, total = 0;
  float lo = CUDART_INF_F, hi = -CUDART_INF_F;
#pragma unroll 4
  for (int t = tid; t < T; t += 256) {
    const bool on = row_counts(labels, ids64, dloss, V, r, t);
    total += on;
    before += on && t < t0;
    if (dloss && on) {
      const float gv = dloss[t];
      if (!(fabsf(gv) < CUDART_INF_F)) lo = -CUDART_INF_F;    // not finite: no common factor
      lo = fminf(lo, gv);
      hi = fmaxf(hi, gv);
    }
  }
  for (int o = 16; o; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    total += __shfl_xor_sync(0xffffffffu, total, o);
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  if (lane == 0) {
    s_cnt[warp][0] = before;
    s_cnt[warp][1] = total;
    s_lo[warp] = lo;
    s_hi[warp] = hi;
  }
  __syncthreads();
  before = total = 0;
  for (int i = 0; i < 8; ++i) {
    before += s_cnt[i][0];
    total += s_cnt[i][1];
  }
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, s_lo[i]);
    hi = fmaxf(hi, s_hi[i]);
  }
  const float scale = lo == hi && fabsf(lo) < CUDART_INF_F ? lo : 1.0f;
  if (blockIdx.x == 0 && tid == 0) {
    r.n_active[0] = total;
    *r.scale = scale;
  }
  const bool copy = total != T;
  uint4* out = reinterpret_cast<uint4*>(r.Xc);
  for (int base = t0; base < t1; base += 256) {
    const int t = base + tid;
    const bool on = t < t1 && row_counts(labels, ids64, dloss, V, r, t);
    const unsigned b = __ballot_sync(0xffffffffu, on);
    __syncthreads();                                   // the lists are free again
    if (lane == 0) s_cnt[warp][0] = __popc(b);
    __syncthreads();
    int at = __popc(b & ((1u << lane) - 1u)), n = 0;
    for (int i = 0; i < 8; ++i) {
      if (i < warp) at += s_cnt[i][0];
      n += s_cnt[i][0];
    }
    if (t < t1) r.inv[t] = on ? before + at : -1;
    const int rows = min(256, t1 - base);
    if (on) {
      r.rec[before + at] = make_int4(t, labels ? (int)load_id(labels, ids64, t) : r.cnt[t],
                                     __float_as_int(dloss ? lse[t] : 0.0f),
                                     __float_as_int(dloss ? dloss[t] / scale : 0.0f));
      s_on[at] = t;
    } else if (t < t1) {
      s_off[tid - at] = t;
    }
    __syncthreads();
    if (copy) {
      const int64_t all = (int64_t)n * vecs;
#pragma unroll 4
      for (int64_t i = tid; i < all; i += 256) {
        const int row = (int)(i / vecs), c = (int)(i - (int64_t)row * vecs);
        out[(int64_t)(before + row) * vecs + c] = X[(int64_t)s_on[row] * vecs + c];
      }
      if (dX)
        for (int64_t i = tid; i < (int64_t)(rows - n) * vecs; i += 256) {
          const int row = (int)(i / vecs), c = (int)(i - (int64_t)row * vecs);
          dX[(int64_t)s_off[row] * vecs + c] = make_uint4(0, 0, 0, 0);
        }
    }
    before += n;
  }
  if (copy) {
    const int pad = (total + kHeadRowPad - 1) / kHeadRowPad * kHeadRowPad;
    for (int i = total + (int)blockIdx.x; i < pad; i += gridDim.x)
      for (int c = tid; c < vecs; c += 256) out[(int64_t)i * vecs + c] = make_uint4(0, 0, 0, 0);
  }
}

// (max, sum of exp) of two disjoint sets of columns, joined; (-inf, 0) is the
// empty set.  A NaN sum stays.
__device__ __forceinline__ void join(float& m, float& s, float om, float os) {
  const float mn = fmaxf(m, om);
  const float a = mn == -CUDART_INF_F ? 0.0f : mn;
  s = s * expf(m - a) + os * expf(om - a);
  m = mn;
}

// Joins the (max, sum) pairs of a token's 128-column blocks and writes its
// loss.  Four tokens per block (their pairs share a 32-byte sector): each
// thread joins every 8 * warps-th pair, then threads and warps join in
// a fixed order; one warp per token then adds up the target entries.
__global__ void __launch_bounds__(1024) head_loss_kernel(const void* labels, int ids64, int T, int64_t V, int K, int np,
                                                         int64_t Tp, float temperature, int distill, HeadRows r,
                                                         float* loss, float* lse) {
  __shared__ float sm[4][32], ss[4][32];
  pdl_wait();
  pdl_release();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  const int t0 = blockIdx.x * 4;
  auto row_of = [&](int t) {             // the row of a token that counts, else -1
    if (r.inv) return r.inv[t];
    return row_counts(labels, ids64, nullptr, V, r, t) ? t : -1;
  };
  {
    const int t = t0 + (lane & 3);
    const int row = t < T ? row_of(t) : -1;
    float m = -CUDART_INF_F, s = 0.0f;
    if (row >= 0) {
      const float2* src = r.part + row;
      const int step = 8 * nw;
      int i = warp * 8 + (lane >> 2);
      for (; i + 3 * step < np; i += 4 * step) {
        float2 p[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) p[u] = src[(i + u * step) * Tp];
#pragma unroll
        for (int u = 0; u < 4; ++u) join(m, s, p[u].x, p[u].y);
      }
      for (; i < np; i += step) join(m, s, src[i * Tp].x, src[i * Tp].y);
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      const float om = __shfl_xor_sync(0xffffffffu, m, o), os = __shfl_xor_sync(0xffffffffu, s, o);
      join(m, s, om, os);
    }
    if (lane < 4) {
      sm[lane][warp] = m;
      ss[lane][warp] = s;
    }
  }
  __syncthreads();
  const int t = t0 + warp;
  if (warp >= 4 || t >= T) return;
  const int row = row_of(t);
  if (row < 0) {
    if (lane == 0) {
      loss[t] = 0.0f;
      lse[t] = 0.0f;
    }
    return;
  }
  float m = lane < nw ? sm[warp][lane] : -CUDART_INF_F, s = lane < nw ? ss[warp][lane] : 0.0f;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float om = __shfl_xor_sync(0xffffffffu, m, o), os = __shfl_xor_sync(0xffffffffu, s, o);
    join(m, s, om, os);
  }
  const float l = m + logf(s);
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

// dX of each token that counts = factor * (sum over the splits, in order).
__global__ void __launch_bounds__(256) head_dx_kernel(int d, int nsplit, int64_t Tp, float out_scale, HeadRows r,
                                                      uint2* __restrict__ dX) {
  pdl_wait();
  pdl_release();
  const int vecs = d / 4;
  const float sc = *r.scale * out_scale;
  const float4* acc = reinterpret_cast<const float4*>(r.acc);
  const int64_t n = (int64_t)*r.n_active * vecs;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = i / vecs;
    const int c = (int)(i - row * vecs);
    float4 a = acc[i];
#pragma unroll 8
    for (int s = 1; s < nsplit; ++s) {
      const float4 b = acc[(s * Tp + row) * vecs + c];
      a.x += b.x;
      a.y += b.y;
      a.z += b.z;
      a.w += b.w;
    }
    dX[(int64_t)r.rec[row].x * vecs + c] = make_uint2(pack_bf16(a.x * sc, a.y * sc), pack_bf16(a.z * sc, a.w * sc));
  }
}

}  // namespace

cudaError_t launch_head_entries(const void* teacher, bool teacher_bf16, const void* ids, bool ids64, int T, int K,
                                int64_t V, float inv_temp, const HeadRows& r, cudaStream_t st) {
  int kp = 2;
  while (kp < K) kp <<= 1;
  int threads = 32;
  while (threads < kp / 2 && threads < 256) threads <<= 1;
  return launch_pdl(head_entries_kernel, dim3(T), dim3(threads), kp * 8 + K * 4, st, 1, teacher, (int)teacher_bf16, ids,
                    (int)ids64, K, kp, V, inv_temp, r);
}

cudaError_t launch_head_prep(const void* labels, bool ids64, const float* dloss, const float* lse, const void* X,
                             int T, int d, int64_t V, const HeadRows& r, void* dX, int num_sms, cudaStream_t st) {
  // few tokens per block, so that a block's copy is short, up to one wave of
  // blocks; fewer when T is large, since every block reads all T tokens' labels
  const int most = (T <= 32768 ? 8 : 2) * num_sms;
  const int blocks = (T + 3) / 4 < most ? (T + 3) / 4 : most;
  return launch_pdl(head_prep_kernel, dim3(blocks), dim3(256), 0, st, 1, labels, (int)ids64, dloss, lse, T, V,
                    reinterpret_cast<const uint4*>(X), d / 8, r, reinterpret_cast<uint4*>(dX));
}

cudaError_t launch_head_loss(const void* labels, bool ids64, int T, int64_t V, int K, int np, int64_t Tp,
                             float temperature, bool distill, const HeadRows& r, float* loss, float* lse,
                             cudaStream_t st) {
  // few blocks: more threads each
  return launch_pdl(head_loss_kernel, dim3((T + 3) / 4), dim3(T <= 1024 ? 1024 : 256), 0, st, 1, labels, (int)ids64, T,
                    V, K, np, Tp, temperature, (int)distill, r, loss, lse);
}

cudaError_t launch_head_dx(int T, int d, int nsplit, int64_t Tp, float out_scale, const HeadRows& r, void* dX,
                           int num_sms, cudaStream_t st) {
  const int64_t n = ((int64_t)T * (d / 4) + 255) / 256;
  return launch_pdl(head_dx_kernel, dim3((unsigned)(n < 8 * num_sms ? n : 8 * num_sms)), dim3(256), 0, st, 1, d, nsplit,
                    Tp, out_scale, r, reinterpret_cast<uint2*>(dX));
}

}  // namespace moe
