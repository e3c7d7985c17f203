// logits.cu -- what happens to logits between the head and a sampler: penalties
// for tokens that a text already holds, biases of single tokens, masks of what a
// grammar allows.  One pass; per row t and column v
//   z = logits[t, v]
//   z = z > 0 ? z / repetition_t : z * repetition_t     if v occurs in the row's history
//   z = z - frequency_t * n - presence_t                if v was generated n > 0 times
//   z = z + each of the row's biases with id v, in their order
//   z = -inf                                            if the row's mask leaves v out
// in fp32, an operation at a time as they stand here, rounded once to the type of the logits.
//
// A block owns a range of columns of one row.  Its logits go into registers; while they are on their way the block
// counts the row's history into one word per column in shared memory (integer atomics: the result does not depend
// on their order) and marks the columns that have a bias.  Then vectors whose words are all zero are written as they
// are, masked, and the others worked out.  Where histories are long, up to eight of a row's blocks make a
// cluster and count an eighth of it each, into the block that owns the column.
//
// What bounds it (in a graph; HBM would take 5.3 us for 64 rows of 65536 in fp32): 6.6 us with histories of 512, 20.3
// with 8192, half of them in use, where each warp meets a marked column at nearly every step.  Of these 1.2 are the
// division (a product with the reciprocal, which rounds twice and overflows where z / repetition does not: 19.1).  Tried
// with the reciprocal, against 18.6: lists of the marked columns, each worked out by a thread of its own (20.7), blocks of
// 512 threads, half the columns to a block, and each block counting the whole history (27 with 16384 columns to a block).
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <string>

#include "kernels.h"
#include "moe.h"
#include "pdl.cuh"
#include "ptx.cuh"

namespace {

using namespace moe;

constexpr int kThreads = 256;
constexpr int kMaxBias = 1024;
// Histories up to this length are read by every block of a row on its own: a cluster's two
// barriers cost more (300 rows of 50001 in bf16, histories of 777: 32.2 us against 25.9; one row of 131072 with 8192: 5.8
// us in clusters, 8.0 alone).
constexpr int64_t kAlone = 2048;
constexpr int64_t kMaxHistory = (1 << 20) - 1;
// A column's word: how often it was generated, whether the history holds it, its first bias
// entry (plus one).
constexpr uint32_t kCountMask = (1u << 20) - 1, kSeen = 1u << 20;
constexpr int kBiasShift = 21;

struct LogitsArgs {
  moe_logits_t a;
  uint32_t chunks;    // blocks per row, a multiple of the cluster's
  uint32_t cluster;   // blocks that share a row's history
};

template <class T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int n = 4;
  // the elements whose bit is clear become -inf
  static __device__ __forceinline__ void mask(uint32_t& w, uint32_t bits) { w = (bits & 1) ? w : 0xff800000u; }
  static __device__ __forceinline__ float get(uint32_t w, int) { return __uint_as_float(w); }
  static __device__ __forceinline__ void put(uint32_t& w, int, float v) { w = __float_as_uint(v); }
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ void store(float* p, float v) { *p = v; }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int n = 8;
  static __device__ __forceinline__ void mask(uint32_t& w, uint32_t bits) {
    w = ((bits & 1) ? w & 0xffffu : 0xff80u) | ((bits & 2) ? w & 0xffff0000u : 0xff800000u);
  }
  static __device__ __forceinline__ float get(uint32_t w, int half) { return __uint_as_float(half ? w & 0xffff0000u : w << 16); }
  static __device__ __forceinline__ void put(uint32_t& w, int half, float v) {
    const uint32_t b = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    w = half ? (w & 0xffffu) | b << 16 : (w & 0xffff0000u) | b;
  }
  static __device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
};

__device__ __forceinline__ int64_t load_id(const void* p, int64_t i, bool wide) {
  return wide ? __ldg(static_cast<const long long*>(p) + i) : (long long)__ldg(static_cast<const int*>(p) + i);
}
__device__ __forceinline__ uint32_t shared_at(uint32_t saddr, uint32_t rank) {   // the same place in another block of the cluster
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ void shared_add(uint32_t at, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void shared_or(uint32_t at, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// X: type of the logits; NV: 16-byte vectors per thread; a block's columns: kThreads * NV vectors.
// (The most vectors, 8192 columns, took 76 registers with the division: three blocks to an SM, 28.4 us where four take 20.3.)
template <class X, int NV>
__global__ void __launch_bounds__(kThreads, NV * Vec<X>::n == 32 ? 4 : 1) logits_kernel(const __grid_constant__ LogitsArgs g) {
  constexpr int W = Vec<X>::n, kPer = W / 4;
  constexpr int kCols = kThreads * NV * W;
  extern __shared__ __align__(16) uint32_t word[];   // [kCols], then the biases' columns, values and successors, [K] each
  const moe_logits_t& a = g.a;
  int* bias_col = reinterpret_cast<int*>(word + kCols);
  float* bias_val = reinterpret_cast<float*>(bias_col + a.K);
  int* bias_next = reinterpret_cast<int*>(bias_val + a.K);       // the next entry with the same id, or -1
  const int tid = threadIdx.x;
  const uint32_t row_ = blockIdx.x / g.chunks, chunk = blockIdx.x - row_ * g.chunks;
  const uint32_t rank = chunk % g.cluster;            // of the block in its cluster
  const int64_t row = row_;
  const X* src = static_cast<const X*>(a.logits) + row * a.ld_logits;
  X* dst = static_cast<X*>(a.out) + row * a.ld_out;
  // Columns are counted from the 16-byte boundary at or before the row's first element, so that every
  // whole vector is aligned; vectors at the row's two ends are taken element by element.
  const int lead = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(X));
  const bool together = (int)((reinterpret_cast<uintptr_t>(dst) & 15) / sizeof(X)) == lead;
  const int64_t c0 = (int64_t)chunk * kCols - lead;   // the block's first column (may lie before the row)
  const bool inside = c0 >= 0 && c0 + kCols <= a.V;   // no vector at an end of the row

  pdl_wait();
  pdl_release();
  const bool counts = a.history != nullptr && (a.repetition || a.frequency || a.presence);
  const bool marks = counts || a.K > 0;
  // the row's numbers, all on their way at once
  const int64_t m = a.mask_rows ? (int64_t)__ldg(a.mask_rows + row) : row;
  const int64_t said = counts && a.lengths ? (int64_t)__ldg(a.lengths + row) : a.L;
  const int64_t given = counts && a.prompt_lengths ? (int64_t)__ldg(a.prompt_lengths + row) : 0;
  const float rep = a.repetition ? __ldg(a.repetition + row) : 1.0f;
  const float freq = a.frequency ? __ldg(a.frequency + row) : 0.0f;
  const float pres = a.presence ? __ldg(a.presence + row) : 0.0f;
  uint4 q[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t c = c0 + (i * kThreads + tid) * W;
    if (inside || (c >= 0 && c + W <= a.V)) q[i] = *reinterpret_cast<const uint4*>(src + c);
  }
  const int32_t* mask = a.mask && m >= 0 && m < a.G ? a.mask + m * a.ld_mask : nullptr;

  if (marks) {
    for (int i = tid; i < kCols / 4; i += kThreads) reinterpret_cast<uint4*>(word)[i] = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < a.K; i += kThreads) {
      const int64_t v = load_id(a.bias_ids, row * a.ld_bias_ids + i, a.bias_ids_int64);
      bias_col[i] = v >= 0 && v < a.V && v - c0 >= 0 && v - c0 < kCols ? (int)(v - c0) : -1;
      bias_val[i] = __ldg(a.bias + row * a.ld_bias + i);
    }
    if (counts) {
      const int len = (int)min(max(said, (int64_t)0), a.L);
      const int64_t f0 = c0 - (int64_t)rank * kCols;  // first column of the cluster
      const int64_t lo = max(f0, (int64_t)0);
      const uint64_t cols = (uint64_t)max(min(f0 + (int64_t)g.cluster * kCols, a.V) - lo, (int64_t)0);
      const uint32_t skip = (uint32_t)(lo - f0), here = smem_u32(word);
      auto count = [&](int i, int64_t v) {
        const uint64_t c = (uint64_t)(v - lo);
        if (c >= cols) return;
        const uint32_t at = (uint32_t)c + skip, block = at / kCols;
        const uint32_t to = shared_at(here + (at - block * kCols) * 4, block);
        if (i < given) shared_or(to, kSeen);
        else shared_add(to, 1u);                      // counts up to kMaxHistory do not reach kSeen
      };
      if (g.cluster > 1) cluster_barrier();           // every block's words are zero
      else __syncthreads();
      const int step = kThreads * g.cluster;
      for (int i0 = rank * kThreads + tid; i0 < len; i0 += 4 * step) {
        int64_t v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          v[k] = i0 + k * step < len ? load_id(a.history, row * a.ld_history + i0 + k * step, a.history_int64) : -1;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (v[k] >= 0) count(i0 + k * step, v[k]);
      }
      if (g.cluster > 1) cluster_barrier();           // and every count is there
      else __syncthreads();
    } else {
      __syncthreads();
    }
    // The first entry with an id stands in its column's word, the others follow it in their order.
    if (a.K > 0) {
      for (int i = tid; i < a.K; i += kThreads) {
        const int c = bias_col[i];
        if (c < 0) continue;
        bool first = true;
        for (int j = 0; j < i && first; ++j) first = bias_col[j] != c;
        int next = i + 1;
        while (next < a.K && bias_col[next] != c) ++next;
        bias_next[i] = next < a.K ? next : -1;
        if (first) word[c] |= (uint32_t)(i + 1) << kBiasShift;     // no other thread writes here
      }
      __syncthreads();
    }
  }

  auto finish = [&](float z, uint32_t w) {
    const uint32_t n = w & kCountMask;
    if (w & (kSeen | kCountMask)) z = z > 0.0f ? __fdiv_rn(z, rep) : z * rep;
    if (n) z = __fsub_rn(__fsub_rn(z, __fmul_rn(freq, (float)n)), pres);
    for (int i = (int)(w >> kBiasShift) - 1; i >= 0; i = bias_next[i]) z += bias_val[i];
    return z;
  };
  const bool copies = static_cast<const void*>(src) != static_cast<const void*>(dst);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (i * kThreads + tid) * W;
    const int64_t c = c0 + at;
    if (!inside && (c >= a.V || c + W <= 0)) continue;
    if (inside || (c >= 0 && c + W <= a.V)) {
      bool write = copies;
      uint32_t x[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
      if (marks) {
        uint4 u[kPer];
        const int flip = kPer == 2 ? (tid >> 2) & 1 : 0;   // eight lanes read 128 bytes from different banks
#pragma unroll
        for (int e = 0; e < kPer; ++e) u[e] = *reinterpret_cast<const uint4*>(word + at + 4 * (e ^ flip));
        if (kPer == 2 && flip) {
          const uint4 other = u[0];
          u[0] = u[kPer - 1];
          u[kPer - 1] = other;
        }
        // The marked elements one by one: a warp takes as many steps as its fullest lane has of them, not one per element.
        const uint32_t* w = reinterpret_cast<const uint32_t*>(u);
        uint32_t left = 0;
#pragma unroll
        for (int e = 0; e < W; ++e) left |= w[e] ? 1u << e : 0u;
        write |= left != 0;
#pragma unroll 1
        for (; left; left &= left - 1) {
          const int e = __ffs(left) - 1;
          uint32_t v = x[0];
#pragma unroll
          for (int o = 1; o < 4; ++o) v = e / kPer == o ? x[o] : v;
          Vec<X>::put(v, e % kPer, finish(Vec<X>::get(v, e % kPer), word[at + e]));
#pragma unroll
          for (int o = 0; o < 4; ++o) x[o] = e / kPer == o ? v : x[o];
        }
      }
      if (mask) {
        write = true;
        const uint32_t bit = (uint32_t)c & 31, w0 = __ldg(mask + (c >> 5));
        const uint32_t w1 = bit + W > 32 ? __ldg(mask + (c >> 5) + 1) : 0u;
        const uint32_t bits = __funnelshift_r(w0, w1, bit);
#pragma unroll
        for (int e = 0; e < 4; ++e) Vec<X>::mask(x[e], bits >> (e * kPer));
      }
      if (!write) continue;
      if (together) {
        *reinterpret_cast<uint4*>(dst + c) = make_uint4(x[0], x[1], x[2], x[3]);
      } else {
#pragma unroll
        for (int e = 0; e < W; ++e) Vec<X>::store(dst + c + e, Vec<X>::get(x[e / kPer], e % kPer));
      }
    } else {
      for (int e = 0; e < W; ++e) {
        const int64_t v = c + e;
        if (v < 0 || v >= a.V) continue;
        const float z = Vec<X>::load(src + v);
        const uint32_t w = marks ? word[at + e] : 0u;
        const bool shut = mask && !(__ldg(mask + (v >> 5)) >> (v & 31) & 1);
        Vec<X>::store(dst + v, shut ? -INFINITY : w ? finish(z, w) : z);
      }
    }
  }
}

moe_status_t bad(const std::string& what, moe_status_t s = MOE_ERR_INVALID_ARG) {
  set_error_detail(("moe_process_logits: " + what).c_str());
  return s;
}

template <class X, int NV>
cudaError_t launch(const LogitsArgs& g, cudaStream_t st) {
  constexpr int64_t cols = kThreads * NV * Vec<X>::n;
  const bool counts = g.a.history && (g.a.repetition || g.a.frequency || g.a.presence);
  const size_t smem = counts || g.a.K > 0 ? cols * 4 + g.a.K * 12 : 0;
  static_assert(cols * 4 + kMaxBias * 12 <= 48 * 1024, "shared memory");
  if (smem > 16 * 1024) {   // six blocks to an SM
    const cudaError_t e = cudaFuncSetAttribute(logits_kernel<X, NV>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                               cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(logits_kernel<X, NV>, dim3((unsigned)(g.a.T * g.chunks)), dim3(kThreads), smem, st, (int)g.cluster, g);
}

// Vectors per thread: as few as give the call a block per SM at least, so that few rows are spread over the GPU.
template <class X>
cudaError_t launch_rows(LogitsArgs& g, int sms, cudaStream_t st) {
  constexpr int W = Vec<X>::n;
  int nv = 32 / W;                                    // 8192 columns
  // rows that do not all start on 16 bytes may begin before their first column
  const bool aligned = (reinterpret_cast<uintptr_t>(g.a.logits) & 15) == 0 && g.a.ld_logits % W == 0;
  const int64_t most = g.a.V + (aligned ? 0 : W - 1);
  auto chunks = [&](int n) { return (most + (int64_t)kThreads * n * W - 1) / ((int64_t)kThreads * n * W); };
  while (nv > 1 && g.a.T * chunks(nv) < sms) nv /= 2;
  // clusters of up to eight blocks share a history; a row is a whole number of them
  const bool counts = g.a.history && g.a.L > kAlone && (g.a.repetition || g.a.frequency || g.a.presence);
  const int64_t clusters = counts ? (chunks(nv) + 7) / 8 : chunks(nv);
  g.cluster = (uint32_t)((chunks(nv) + clusters - 1) / clusters);
  g.chunks = (uint32_t)(clusters * g.cluster);
  if (g.a.T * g.chunks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  switch (nv) {
    case 8: if constexpr (W == 4) return launch<X, 8>(g, st);
    case 4: return launch<X, 4>(g, st);
    case 2: return launch<X, 2>(g, st);
    default: return launch<X, 1>(g, st);
  }
}

bool at(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

extern "C" moe_status_t moe_process_logits(const moe_logits_t* args, moe_stream_t stream) {
  if (!args) return bad("null argument");
  const moe_logits_t& a = *args;
  const size_t es = a.bf16 ? 2 : 4;
  if (a.T < 0 || a.T > (1 << 20)) return bad("T must be in [0, 2^20]");
  if (a.V < 1 || a.V > (1 << 24)) return bad("V must be in [1, 2^24]");
  if (a.T == 0) return MOE_OK;
  if (!a.logits || !a.out || !at(a.logits, es) || !at(a.out, es)) return bad("logits and out are required, aligned to their type");
  if (a.ld_logits < a.V || a.ld_out < a.V) return bad("a row stride is smaller than V");
  const uintptr_t x0 = reinterpret_cast<uintptr_t>(a.logits), x1 = x0 + ((a.T - 1) * a.ld_logits + a.V) * es;
  const uintptr_t y0 = reinterpret_cast<uintptr_t>(a.out), y1 = y0 + ((a.T - 1) * a.ld_out + a.V) * es;
  if (x0 < y1 && y0 < x1 && !(x0 == y0 && a.ld_logits == a.ld_out)) return bad("out overlaps the logits without being them");
  if (a.history) {
    if (a.L < 0 || a.L > kMaxHistory) return bad("L must be in [0, 2^20 - 1]");
    if (a.ld_history < a.L || !at(a.history, a.history_int64 ? 8 : 4)) return bad("history: row stride or alignment");
  }
  if (!at(a.lengths, 4) || !at(a.prompt_lengths, 4) || !at(a.repetition, 4) || !at(a.frequency, 4) || !at(a.presence, 4) ||
      !at(a.mask, 4) || !at(a.mask_rows, 4) || !at(a.bias, 4))
    return bad("misaligned pointer");
  if (a.K < 0 || a.K > kMaxBias) return bad("K must be in [0, 1024]");
  if (a.K > 0 && (!a.bias_ids || !a.bias || a.ld_bias_ids < a.K || a.ld_bias < a.K || !at(a.bias_ids, a.bias_ids_int64 ? 8 : 4)))
    return bad("bias_ids and bias: pointer, row stride or alignment");
  if (a.mask) {
    if (a.ld_mask < (a.V + 31) / 32) return bad("mask: a row holds ceil(V / 32) words");
    if (a.G < 0 || (!a.mask_rows && a.G < a.T)) return bad("mask: fewer rows than logits and no mask_rows");
  }
  int dev = 0, sms = 0, major = 0, minor = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (e == cudaSuccess && (major != 10 || minor != 3))
    return bad("this library is built for sm_103a (GB300) only", MOE_ERR_UNSUPPORTED);
  if (e == cudaSuccess) {
    LogitsArgs g{a, 0, 1};
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    e = a.bf16 ? launch_rows<__nv_bfloat16>(g, sms, st) : launch_rows<float>(g, sms, st);
  }
  if (e != cudaSuccess) return bad(std::string("launch: ") + cudaGetErrorString(e), MOE_ERR_CUDA);
  return MOE_OK;
}
