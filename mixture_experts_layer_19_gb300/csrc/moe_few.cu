// moe_few.cu -- the whole MoE layer for up to 64 tokens in one cooperative launch.
//
//   [logits = X Wr^T]  ->  top-k, softmax  ->  h = silu(x Wg^T) (x Wu^T)  ->  y = h Wd^T  ->  Y = sum_j w_j y_j
//
// The chosen experts' weights are read once and nothing else is large, so the
// kernel is built around their stream: every SM reads an equal share of the
// 128-byte-deep slices of the [Wg; Wu] tiles, then of the Wd tiles, in one run
// through a ring of stages that never drains -- slices of Wd are fetched while h
// is still being finished elsewhere.  Tiles that fall into several SMs' shares are
// summed, in the order of the SMs, by whichever of them finishes last (warp by warp).
//   warp 0  weights into the stages (TMA)
//   warp 1  activations into the same stages: all tokens (up), the expert's rows of h (down; waits for them)
//   warp 2  tcgen05.mma: M = 128 weight rows, N = activation rows, two tiles of 128 rows per slice
//   warps 4-11  epilogue: lane = weight row, register = token
// Every sum has one fixed order, so results repeat bitwise; they do not depend on
// which other tokens share the call, except through where the sums are cut.
// bf16: h is kept as a bf16 value and what its rounding left, two rows of B each, so the
// down product loses nothing to it (its columns are nearly free: one token needs 16 anyway).
// Block-scaled plans quantise X and h as the plan's forward does.
#include "few.cuh"
#include "kernels.h"
#include "moe_few.h"
#include "mx.cuh"
#include "nv.cuh"

namespace moe {

namespace {

enum { kFmtBf16 = 0, kFmtMx = 1, kFmtNv = 2 };

template <int FMT>
struct FewTraits {
  static constexpr int kelems = FMT == kFmtBf16 ? 64 : FMT == kFmtMx ? 128 : 256;   // K values of a slice
  static constexpr int atom_k = FMT == kFmtNv ? 64 : 128;            // K values of a scale atom
  static constexpr int sf = FMT == kFmtBf16 ? 0 : FMT == kFmtMx ? 512 : 2048;       // scale bytes of 128 rows
  [[maybe_unused]] static constexpr int sf_cols = FMT == kFmtNv ? 48 : 16;            // TMEM columns of a stage's scales
  static constexpr int acc_cols = FMT == kFmtBf16 ? 256 : 128;       // TMEM columns of one accumulator pair
  static constexpr int per = FMT == kFmtBf16 ? 2 : 1;                // B rows of one row of h
};

// Shared memory behind the stages: barriers, then the routing that every CTA works out for itself.
struct FewSmem {
  uint64_t *full, *empty, *tfull, *tempty, *drain;
  uint32_t* tmem_slot;
  int* abort_flag;
  int* flag;          // prologue; last CTA; [2] accumulator ready; all CTAs done
  float* sums;        // [12][8] router partial sums
  uint64_t* mask;     // [E] tokens of each expert
  float* w;           // [T k]
  int* off;           // [active + 1] first sorted row of each active expert
  uint16_t* idx;      // [T k]
  uint16_t* act;      // [active] experts that have tokens
  uint16_t* slot;     // [E] position among them
  uint16_t* row;      // [T k] sorted row of each pair
  int* n_act;
};

__host__ __device__ constexpr size_t few_tail_bytes(int T, int E, int k) {
  const int active = E < T * k ? E : T * k;
  return 256 + 32 + 12 * 8 * 4 + (size_t)E * 8 + (size_t)T * k * 4 + (size_t)(active + 1) * 4 + 4 +
         ((size_t)2 * T * k + active + E) * 2 + 64;
}

__device__ __forceinline__ FewSmem few_smem(uint8_t* p, int T, int E, int k) {
  FewSmem s;
  const int active = min(E, T * k);
  s.full = reinterpret_cast<uint64_t*>(p);
  s.empty = s.full + kFewMaxStages;
  s.tfull = s.empty + kFewMaxStages;
  s.tempty = s.tfull + 2;
  s.drain = s.tempty + 2;
  s.tmem_slot = reinterpret_cast<uint32_t*>(s.drain + 1);
  s.abort_flag = reinterpret_cast<int*>(s.tmem_slot + 1);
  p += 256;
  s.mask = reinterpret_cast<uint64_t*>(p);
  p += (size_t)E * 8;
  s.flag = reinterpret_cast<int*>(p);
  s.sums = reinterpret_cast<float*>(s.flag + 8);
  s.w = s.sums + 12 * 8;
  s.off = reinterpret_cast<int*>(s.w + T * k);
  s.n_act = s.off + active + 1;
  s.idx = reinterpret_cast<uint16_t*>(s.n_act + 1);
  s.act = s.idx + T * k;
  s.slot = s.act + active;
  s.row = s.slot + E;
  return s;
}

// Which halves of the epilogue's warps (groups of eight tokens, in turn) have tokens of an expert.
__device__ __forceinline__ int halves(uint64_t mask) {
  return ((mask & 0x00ff00ff00ff00ffull) != 0) + ((mask & 0xff00ff00ff00ff00ull) != 0);
}

// Top-k and softmax of one token by a warp, the rules and the arithmetic of route_token (routing.cuh): larger
// logit first, lower expert on ties, weights relative to the largest.  NPER logits per lane.  Logits are compared as
// integers of the same order, so that a round is two warp reductions (32 tokens x 64 experts, top 8: the prologue takes
// 8.4 us; 12.0 with shuffles).
template <int NPER>
__device__ __forceinline__ void few_route(const float* row, int t, int E, int k, int lane, const FewSmem& s) {
  uint32_t key[NPER];                                               // 0: none, or taken
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    const int e = lane + 32 * i;
    const uint32_t u = e < E ? __float_as_uint(__ldcg(row + e) + 0.0f) : 0xffffffffu;   // -0 counts as 0
    key[i] = (u & 0x80000000u) ? ~u : u | 0x80000000u;
    // NaN logits (outside the contract) come last, but above "none": a token's experts stay distinct
    if ((u & 0x7fffffffu) > 0x7f800000u) key[i] = 1;
    if (e >= E) key[i] = 0;
  }
  int my_id = 0;
  float my_val = 0.0f;
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < NPER; ++i) best = max(best, key[i]);
    best = __reduce_max_sync(0xffffffffu, best);
    uint32_t id = 0xffffffffu;
#pragma unroll
    for (int i = NPER - 1; i >= 0; --i)
      if (key[i] == best) id = lane + 32 * i;
    id = __reduce_min_sync(0xffffffffu, id);
    if ((id & 31u) == (uint32_t)lane) {
#pragma unroll
      for (int i = 0; i < NPER; ++i)
        if ((id >> 5) == (uint32_t)i) key[i] = 0;
    }
    if (lane == j) {
      my_id = (int)id;
      my_val = best == 1 ? NAN : __uint_as_float((best & 0x80000000u) ? best & 0x7fffffffu : ~best);
    }
  }
  const float top = __shfl_sync(0xffffffffu, my_val, 0);
  const float z = lane < k ? expf(my_val - top) : 0.0f;
  float sum = z;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane < k) {
    s.idx[t * k + lane] = (uint16_t)my_id;
    s.w[t * k + lane] = z / sum;
    atomicOr(reinterpret_cast<unsigned long long*>(s.mask + my_id), 1ull << t);
  }
}

// Router logits of one expert and up to 8 tokens by the whole CTA: each warp a strided share of the width,
// the warps' sums added in their order.
__device__ __forceinline__ void few_logits(const FewArgs& g, const FewSmem& s, int item, int groups) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e = item / groups, t0 = (item - e * groups) * 8;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
  for (int v = threadIdx.x; v < g.d / 8; v += kFewThreads) {
    const uint4 wq = __ldg(reinterpret_cast<const uint4*>(g.Wr + (size_t)e * g.d) + v);
    const uint32_t ww[4] = {wq.x, wq.y, wq.z, wq.w};
    uint4 xq[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      xq[i] = t0 + i < g.T ? __ldg(reinterpret_cast<const uint4*>(g.X + (size_t)(t0 + i) * g.d) + v) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t xx[4] = {xq[i].x, xq[i].y, xq[i].z, xq[i].w};
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&ww[p]));
        const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&xx[p]));
        acc[i] = fmaf(a.x, b.x, acc[i]);
        acc[i] = fmaf(a.y, b.y, acc[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    if (lane == i) s.sums[warp * 8 + i] = acc[i];
  }
  __syncthreads();
  if (threadIdx.x < 8 && t0 + (int)threadIdx.x < g.T) {
    float z = 0.0f;
    for (int w = 0; w < kFewThreads / 32; ++w) z += s.sums[w * 8 + threadIdx.x];
    g.logits_out[(size_t)(t0 + threadIdx.x) * g.E + e] = z;
  }
  __syncthreads();
}

template <int FMT>
__global__ void __launch_bounds__(kFewThreads, 1) moe_few_kernel(const __grid_constant__ FewArgs g) {
  using TR = FewTraits<FMT>;
  constexpr bool kQ = FMT != kFmtBf16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int St = g.stages;
  const int stage_bytes = kFewABytes + g.b_bytes;
  uint8_t* sf_base = smem + St * stage_bytes;                      // [stages][A tile 0, A tile 1, B]
  const FewSmem s = few_smem(sf_base + St * 3 * TR::sf, g.T, g.E, g.k);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = gridDim.x, cta = blockIdx.x;

  if (threadIdx.x == 0) {
    for (int i = 0; i < St; ++i) {
      mbar_init(&s.full[i], 2);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.tfull[i], 1);
      mbar_init(&s.tempty[i], kFewEpiWarps);
    }
    mbar_init(s.drain, 1);
    *s.abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&g.mapG);
    tma_prefetch_desc(&g.mapU);
    tma_prefetch_desc(&g.mapD);
    tma_prefetch_desc(&g.mapX);
    tma_prefetch_desc(&g.mapH);
  }
  if (warp == 2) {
    tmem_alloc(s.tmem_slot, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  for (int e = threadIdx.x; e < g.E; e += kFewThreads) s.mask[e] = 0;
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *s.tmem_slot;
  WaitCtl wc{g.status, s.abort_flag, g.timeout_ns};

  // ---------------------------------------------------------------- prologue
  bool ok = true;
  const bool gated = g.Wr != nullptr || kQ;
  if (gated) {
    if constexpr (kQ) {
      for (int i = cta * kFewThreads + threadIdx.x; i < g.T * (g.d / 32); i += G * kFewThreads) {
        const int t = i / (g.d / 32), b = i - t * (g.d / 32);
        float v[32];
        load_bf16x32_f(g.X + (size_t)t * g.d + 32 * b, v);
        if constexpr (FMT == kFmtMx) {
          quant_block_store(v, g.Xq + (size_t)t * g.d + 32 * b, g.Xs + sf_atom_offset(t, b, g.d / 32));
        } else {
          uint4 o;
          const uint32_t sc = nv_encode32(v, nv_rc(1.0f), 1.0f, o);
          *reinterpret_cast<uint4*>(g.Xq + (size_t)t * (g.d / 2) + 16 * b) = o;
          *reinterpret_cast<uint16_t*>(g.Xs + sf_atom_offset(t, 2 * b, g.d / 16)) = (uint16_t)sc;
        }
      }
      fence_proxy_async_global();
    }
    if (g.Wr) {
      const int groups = (g.T + 7) / 8;
      for (int i = cta; i < g.E * groups; i += G) few_logits(g, s, i, groups);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      __threadfence();
      atomicAdd(g.gate, 1ull);
      if (g.Wr) s.flag[0] = few_wait(g.gate, (unsigned long long)G, wc) ? 1 : 0;
    }
    __syncthreads();
    if (g.Wr) ok = s.flag[0] != 0;
  }
  if (ok) {
    for (int t = warp; t < g.T; t += kFewThreads / 32) {
      const float* row = g.logits + (size_t)t * g.E;
      if (g.E <= 256) few_route<8>(row, t, g.E, g.k, lane, s);
      else few_route<32>(row, t, g.E, g.k, lane, s);
    }
    __syncthreads();
    if (warp == 0) {  // experts that have tokens, in order, and where their sorted rows start
      int na = 0, rows = 0;
      for (int e0 = 0; e0 < g.E; e0 += 32) {
        const int n = e0 + lane < g.E ? __popcll(s.mask[e0 + lane]) : 0;
        const unsigned any = __ballot_sync(0xffffffffu, n > 0);
        int x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        if (n > 0) {
          const int a = na + __popc(any & ((1u << lane) - 1u));
          s.act[a] = (uint16_t)(e0 + lane);
          s.off[a] = rows + x - n;
          s.slot[e0 + lane] = (uint16_t)a;
        }
        na += __popc(any);
        rows += __shfl_sync(0xffffffffu, x, 31);
      }
      if (lane == 0) {
        s.off[na] = rows;
        *s.n_act = na;
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < g.T * g.k; i += kFewThreads) {
      const int e = s.idx[i], tk = i / g.k;
      const int r = s.off[s.slot[e]] + __popcll(s.mask[e] & ((1ull << tk) - 1));
      s.row[i] = (uint16_t)r;
    }
    __syncthreads();
    const int na = *s.n_act;
    const int UF = g.F / 128, DT = g.d / kFewRows;
    const int KU = g.d / TR::kelems, KD = g.F / TR::kelems;
    const int n_up = round16(g.T);                                  // columns of an up tile

    // This CTA's segments, in order: (phase, cut, tile, first slice, slices).  f returns false to stop.
    auto walk = [&](auto&& f) {
      for (int ph = 0; ph < 2; ++ph) {
        const int K = ph ? KD : KU;
        FewCut cut;
        cut.S = (int64_t)na * (ph ? DT : UF) * K;
        cut.W = (int)min((int64_t)G, cut.S);
        if (cta >= cut.W) continue;
        const int64_t end = cut.start(cta + 1);
        for (int64_t at = cut.start(cta); at < end;) {
          const int u = (int)(at / K), k0 = (int)(at - (int64_t)u * K);
          const int len = (int)min((int64_t)(K - k0), end - at);
          if (!f(ph, cut, u, k0, len)) return false;
          at += len;
        }
      }
      return true;
    };

    if (warp == 0) {
      if (lane == 0 && !g.stall) {
        // -------------------------------------------------------- weights
        const uint64_t pol = policy_evict_first();                  // read once
        uint32_t st = 0, ph = 0, issued = 0, last_par = 0;
        const bool fine = walk([&](int phase, const FewCut&, int u, int k0, int len) {
          const int per = phase ? DT : UF;
          const int a = u / per, tile = u - a * per;
          const int e = s.act[a];
          for (int kb = k0; kb < k0 + len; ++kb) {
            if (!mbar_wait(&s.empty[st], ph ^ 1, wc)) return false;
            mbar_arrive_expect_tx(&s.full[st], kFewABytes + 2 * TR::sf);
            uint8_t* sa = smem + st * stage_bytes;
            uint8_t* sc = sf_base + st * 3 * TR::sf;
            const int x = kQ ? kb * 128 : kb * 64;                  // the maps' unit: bytes or bf16 values
            if (phase == 0) {
              const int row = e * g.F + tile * 128;
              tma_load_2d(sa, &g.mapG, x, row, &s.full[st], pol);
              tma_load_2d(sa + kFewABytes / 2, &g.mapU, x, row, &s.full[st], pol);
              if constexpr (kQ) {
                const size_t at = ((size_t)(row >> 7) * (g.d / TR::atom_k) + (size_t)kb * (TR::kelems / TR::atom_k)) * 512;
                bulk_load_1d(sc, g.sfG + at, TR::sf, &s.full[st]);
                bulk_load_1d(sc + TR::sf, g.sfU + at, TR::sf, &s.full[st]);
              }
            } else {
              const int row = e * g.d + tile * kFewRows;
              tma_load_2d(sa, &g.mapD, x, row, &s.full[st], pol);
              if constexpr (kQ) {
                const size_t kg = g.F / TR::atom_k;
                const size_t at = ((size_t)(row >> 7) * kg + (size_t)kb * (TR::kelems / TR::atom_k)) * 512;
                bulk_load_1d(sc, g.sfD + at, TR::sf, &s.full[st]);
                bulk_load_1d(sc + TR::sf, g.sfD + at + kg * 512, TR::sf, &s.full[st]);
              }
            }
            issued |= 1u << st;
            last_par = (last_par & ~(1u << st)) | (ph << st);
            if (++st == (uint32_t)St) { st = 0; ph ^= 1; }
          }
          return true;
        });
        if (!fine) few_drain(s.full, St, issued, last_par);
      }
    } else if (warp == 1) {
      if (lane == 0) {
        // -------------------------------------------------------- activations
        const uint64_t pol = policy_evict_last();
        uint32_t st = 0, ph = 0, issued = 0, last_par = 0;
        int have = -1;
        bool fine = true;
        if (kQ && !g.Wr) {                                          // the tokens, quantised by all CTAs
          fine = few_wait(g.gate, (unsigned long long)G, wc);
        }
        fence_proxy_async_global();
        fine = fine && walk([&](int phase, const FewCut&, int u, int k0, int len) {
          const int a = u / (phase ? DT : UF);
          if (phase == 1 && a != have) {
            // every epilogue warp that has tokens of the expert counts its part of each tile
            if (!few_wait(g.ready + a, UF * 4 * halves(s.mask[s.act[a]]), wc)) return false;
            fence_proxy_async_global();
            have = a;
          }
          const int n = phase ? round16(TR::per * (s.off[a + 1] - s.off[a])) : n_up;
          const int row0 = phase ? TR::per * s.off[a] : 0;
          const CUtensorMap* m = phase ? &g.mapH : &g.mapX;
          for (int kb = k0; kb < k0 + len; ++kb) {
            if (!mbar_wait(&s.empty[st], ph ^ 1, wc)) return false;
            mbar_arrive_expect_tx(&s.full[st], n * 128 + TR::sf);
            uint8_t* sb = smem + st * stage_bytes + kFewABytes;
            const int x = kQ ? kb * 128 : kb * 64;
            for (int r = 0; r < n; r += 16) tma_load_2d(sb + r * 128, m, x, row0 + r, &s.full[st], pol);
            if constexpr (kQ) {
              const size_t kg = (phase ? g.F : g.d) / TR::atom_k;
              const size_t at = ((size_t)(phase ? a : 0) * kg + (size_t)kb * (TR::kelems / TR::atom_k)) * 512;
              bulk_load_1d(sf_base + st * 3 * TR::sf + 2 * TR::sf, (phase ? g.Hs : g.Xs) + at, TR::sf, &s.full[st]);
            }
            issued |= 1u << st;
            last_par = (last_par & ~(1u << st)) | (ph << st);
            if (++st == (uint32_t)St) { st = 0; ph ^= 1; }
          }
          return true;
        });
        if (!fine) few_drain(s.full, St, issued, last_par);
      }
    } else if (warp == 2) {
      if (lane == 0) {
        // -------------------------------------------------------- products
        uint32_t st = 0, ph = 0, acc = 0, aph = 0;
        const bool fine = walk([&](int phase, const FewCut&, int u, int k0, int len) {
          const int a = u / (phase ? DT : UF);
          const int n = phase ? round16(TR::per * (s.off[a + 1] - s.off[a])) : n_up;
          if (!mbar_wait(&s.tempty[acc], aph ^ 1, wc)) return false;
          tc_fence_after();
          const uint32_t d0 = tmem_base + acc * TR::acc_cols;
          for (int i = 0; i < len; ++i) {
            if (!mbar_wait(&s.full[st], ph, wc)) return false;
            tc_fence_after();
            const uint32_t sa = smem_u32(smem + st * stage_bytes), sb = sa + kFewABytes;
            // descriptors count in 16 bytes: 32 bytes of K, and 512-byte scale atoms, are 2 and 32 further
            const uint64_t da = sdesc_sw128(sa, 16, 1024), db = sdesc_sw128(sb, 16, 1024);
            constexpr int kTile = kFewABytes / 2 / 16;
            if constexpr (FMT == kFmtBf16) {
              const uint32_t id = idesc_bf16(128, n, 0, 0);
#pragma unroll
              for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  umma_bf16(d0 + m * (TR::acc_cols / 2), da + m * kTile + 2 * kk, db + 2 * kk, id, (i | kk) != 0 ? 1u : 0u);
            } else {
              const uint64_t ds = sdesc_plain(smem_u32(sf_base + st * 3 * TR::sf));
              const uint32_t t_sf = tmem_base + 2 * TR::acc_cols + st * TR::sf_cols;
              constexpr int atoms = TR::sf / 512;                   // 1, or 4: one for each product
#pragma unroll
              for (int o = 0; o < 3 * atoms; ++o) tmem_cp_32x128_x4(t_sf + o * 4, ds + o * 32);
              const uint32_t id = FMT == kFmtMx ? 0u : idesc_nvf4(128, n);
#pragma unroll
              for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                  const uint32_t dt = d0 + m * (TR::acc_cols / 2), first = (i | kk) != 0 ? 1u : 0u;
                  if constexpr (FMT == kFmtMx)
                    umma_mxf8(dt, da + m * kTile + 2 * kk, db + 2 * kk, idesc_mxf8(128, n, 0, 0, kk), t_sf + m * 4, t_sf + 8, first);
                  else
                    umma_nvf4(dt, da + m * kTile + 2 * kk, db + 2 * kk, id, t_sf + m * 16 + kk * 4, t_sf + 32 + kk * 4, first);
                }
            }
            umma_commit(&s.empty[st]);
            if (++st == (uint32_t)St) { st = 0; ph ^= 1; }
          }
          umma_commit(&s.tfull[acc]);
          acc ^= 1;
          if (acc == 0) aph ^= 1;
          return true;
        });
        if (!fine) {                                                // products in flight finish before TMEM is freed
          umma_commit(s.drain);
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(s.drain, 0))
            if (globaltimer_ns() - t0 > 50000000ull) break;
        }
      }
    } else if (warp >= 4) {
      // ---------------------------------------------------------- epilogue
      // A warp has 32 rows of both 128-row tiles and every other group of eight columns, and goes its own way: it
      // joins cut tiles with the same warp of the other CTAs, and combines its own columns of a token.
      const int q = warp & 3, half = (warp - 4) >> 2;               // TMEM lane quadrant; which groups of 8 columns
      const int tid = threadIdx.x - 128;
      const int r0 = 32 * q + lane;                                 // row of the first 128-row tile (and of the second)
      const float ts_up = FMT == kFmtNv ? __ldg(g.ts) : 1.0f, ts_dn = FMT == kFmtNv ? __ldg(g.ts + 1) : 1.0f;
      uint32_t acc = 0, aph = 0, turn = 0;
      const bool fine = walk([&](int phase, const FewCut& cut, int u, int k0, int len) {
        const int K = phase ? KD : KU, per = phase ? DT : UF;
        const int a = u / per, tile = u - a * per;
        const int base = s.off[a], n = s.off[a + 1] - base;         // the expert's sorted rows
        const uint64_t mask = s.mask[s.act[a]];
        if (!few_epilogue_wait(&s.tfull[acc], aph, wc, tid, s.flag + 2, turn)) return false;
        tc_fence_after();
        const uint32_t tb = tmem_base + ((uint32_t)(32 * q) << 16) + acc * TR::acc_cols;

        // Where CTA c puts its part of a tile: a range has two cut tiles at most in each phase, one that began
        // before it (`inside`) and one that it leaves unfinished.
        auto part_slot = [&](int c, bool inside) {
          return (size_t)((2 * c + (inside ? 0 : 1)) * 2 + phase) * g.part_rows * kFewRows + r0;
        };
        // One sorted row's two values, finished: h of a column of F, or y of two columns of d.
        auto finish = [&](int r, float v0, float v1) {
          if (phase == 0) {
            if constexpr (FMT == kFmtNv) v0 *= ts_up, v1 *= ts_up;
            const float h = v0 / (1.0f + __expf(-v0)) * v1;
            const int f = tile * 128 + r0;
            if constexpr (FMT == kFmtBf16) {
              __nv_bfloat16* H = reinterpret_cast<__nv_bfloat16*>(g.H) + (size_t)2 * (base + r) * g.F + f;
              const __nv_bfloat16 hi = __float2bfloat16_rn(h);
              H[0] = hi;
              H[g.F] = __float2bfloat16_rn(h - __bfloat162float(hi));
            } else if constexpr (FMT == kFmtMx) {
              const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(h))));
              const int xe = mx_block_exponent(amax);
              const float inv = __int_as_float((127 - xe) << 23);
              g.H[(size_t)(base + r) * g.F + f] = (uint8_t)__nv_cvt_float_to_fp8(h * inv, __NV_SATFINITE, __NV_E4M3);
              if (lane == 0) g.Hs[(size_t)a * (g.F / 128) * 512 + sf_atom_offset(r, f / 32, g.F / 32)] = (uint8_t)(xe + 127);
            } else {
              float amax = fabsf(h);
#pragma unroll
              for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
              const uint8_t sc = (uint8_t)__nv_cvt_float_to_fp8(__fmul_rn(amax, nv_rc(1.0f)), __NV_SATFINITE, __NV_E4M3);
              const float sv = e4m3_value(sc);
              const float x = sv == 0.0f ? 0.0f : __fmul_rn(h, __frcp_rn(sv));
              const float up = __shfl_down_sync(0xffffffffu, x, 1);
              if (!(lane & 1))
                g.H[((size_t)(base + r) * g.F + f) / 2] =
                    sv == 0.0f ? (uint8_t)0 : (uint8_t)__nv_cvt_float2_to_fp4x2(make_float2(x, up), __NV_E2M1, cudaRoundNearest);
              if ((lane & 15) == 0) g.Hs[(size_t)a * (g.F / 64) * 512 + sf_atom_offset(r, f / 16, g.F / 16)] = sc;
            }
          } else {
            if constexpr (FMT == kFmtNv) v0 *= ts_dn, v1 *= ts_dn;
            float* y = g.y + (size_t)(base + r) * g.d + tile * kFewRows + r0;
            __stcg(y, v0);
            __stcg(y + 128, v1);
          }
        };
        // The sorted rows of the eight columns from c on: up, a column is a token, taken where its bit is set; down, a
        // sorted row has TR::per columns.
        auto rows_of = [&](int c, int& r) {
          if (phase == 0) {
            r = __popcll(mask & ((1ull << c) - 1));
            return __popc((uint32_t)(mask >> c) & 0xffu);
          }
          r = c / TR::per;
          return min(8 / TR::per, n - r);
        };
        const bool whole = len == K;
        float* mine = g.part + part_slot(cta, k0 > 0);
        const int cols = phase ? TR::per * n : g.T;
        bool any = false;                                           // this warp has rows of the tile
        for (int c = 8 * half; c < cols; c += 16) {
          int r;
          const int rows = rows_of(c, r);
          if (rows == 0) continue;
          any = true;
          uint32_t v0[8], v1[8];
          tmem_ld8(tb + c, v0);
          tmem_ld8(tb + TR::acc_cols / 2 + c, v1);
          tmem_ld_wait();
          auto take = [&](float x0, float x1) {
            if (whole) {
              finish(r, x0, x1);
            } else {
              __stcg(mine + r * kFewRows, x0);
              __stcg(mine + r * kFewRows + 128, x1);
            }
            ++r;
          };
          if (phase == 0) {
            const uint32_t bits = (uint32_t)(mask >> c) & 0xffu;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if ((bits >> i) & 1) take(__uint_as_float(v0[i]), __uint_as_float(v1[i]));
          } else {
#pragma unroll
            for (int i = 0; i < 8; i += TR::per) {
              float x0 = __uint_as_float(v0[i]), x1 = __uint_as_float(v1[i]);
              if constexpr (TR::per == 2) {
                // an infinite h has left inf - inf behind: its own product stands alone
                x0 = fabsf(x0) < INFINITY ? x0 + __uint_as_float(v0[i + 1]) : x0;
                x1 = fabsf(x1) < INFINITY ? x1 + __uint_as_float(v1[i + 1]) : x1;
              }
              if (r < n) take(x0, x1);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.tempty[acc]);
        acc ^= 1;
        if (acc == 0) aph ^= 1;
        if (!any) return true;

        if (!whole) {
          // the parts of a cut tile: the last warp to bring one adds them up, in the order of the CTAs
          const int first = cut.owner((int64_t)u * K), parts = cut.owner((int64_t)u * K + K - 1) - first + 1;
          __syncwarp();                                             // the lanes' parts come before lane 0's release
          int last = 0;
          if (lane == 0) {
            int* cnt = (phase ? g.cnt_dn : g.cnt_up) + u * kFewEpiWarps + (warp - 4);
            last = atom_add_acq_rel_gpu(cnt, 1) == parts - 1;
            if (last) *cnt = 0;
          }
          if (!__shfl_sync(0xffffffffu, last, 0)) return true;
          __syncwarp();
          for (int c = 8 * half; c < cols; c += 16) {
            int r;
            const int rows = rows_of(c, r);
            if (rows == 0) continue;
            float v0[8], v1[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v0[i] = v1[i] = 0.0f;
#pragma unroll 2
            for (int o = 0; o < parts; ++o) {                       // the first one left the tile unfinished
              const float* p = g.part + part_slot(first + o, o > 0) + r * kFewRows;
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (i < rows) {
                  v0[i] += __ldcg(p + i * kFewRows);
                  v1[i] += __ldcg(p + i * kFewRows + 128);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i < rows) finish(r + i, v0[i], v1[i]);
          }
        }
        if (phase == 0) {
          fence_proxy_async_global();                               // h is read by TMA
          __syncwarp();
          if (lane == 0) red_release_gpu_add(g.ready + a, 1);
        }
        return true;
      });
      // Every CTA's results are on their way; once all CTAs' are there, a warp at a time combines 256 columns of a token.
      // (Combined by whichever warp brought a token's last result, an expert of 16 tokens kept its accumulators waiting:
      // 16 skewed tokens in MXFP8 275 us, 240 like this.)
      if (fine) {
        named_bar(1, 256);
        if (tid == 0) {
          red_release_gpu_add(g.done, 1);
          s.flag[4] = few_wait(g.done, G, wc) ? 1 : 0;
        }
        named_bar(1, 256);
      }
      if (fine && s.flag[4]) {
        for (int i = cta + (warp - 4) * G; i < g.T * DT; i += G * kFewEpiWarps) {
          const int t = i / DT, col = (i - t * DT) * kFewRows + 4 * lane;
          float4 y0 = make_float4(0, 0, 0, 0), y1 = y0;
#pragma unroll 8
          for (int j = 0; j < g.k; ++j) {
            const float4* p = reinterpret_cast<const float4*>(g.y + (size_t)s.row[t * g.k + j] * g.d + col);
            const float w = s.w[t * g.k + j];
            const float4 a0 = __ldcg(p), a1 = __ldcg(p + 32);
            y0.x = fmaf(w, a0.x, y0.x), y0.y = fmaf(w, a0.y, y0.y), y0.z = fmaf(w, a0.z, y0.z), y0.w = fmaf(w, a0.w, y0.w);
            y1.x = fmaf(w, a1.x, y1.x), y1.y = fmaf(w, a1.y, y1.y), y1.z = fmaf(w, a1.z, y1.z), y1.w = fmaf(w, a1.w, y1.w);
          }
          uint2* Y = reinterpret_cast<uint2*>(g.Y + (size_t)t * g.d + col);
          Y[0] = make_uint2(pack_bf16(y0.x, y0.y), pack_bf16(y0.z, y0.w));
          Y[32] = make_uint2(pack_bf16(y1.x, y1.y), pack_bf16(y1.z, y1.w));
        }
      }
    }
  }

  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
  // The last CTA to leave zeroes what the next launch expects to find at zero; after a wait that expired, all of it.
  if (threadIdx.x == 0) {
    __threadfence();
    s.flag[1] = atomicAdd(g.gate + 1, 1ull) == (unsigned long long)G - 1;
    __threadfence();
  }
  __syncthreads();
  if (s.flag[1]) {
    const int na = min(g.E, g.T * g.k);
    for (int i = threadIdx.x; i < na; i += kFewThreads) g.ready[i] = 0;
    if (*reinterpret_cast<volatile int32_t*>(g.status) != 0) {
      for (int i = threadIdx.x; i < g.n_up; i += kFewThreads) g.cnt_up[i] = 0;
      for (int i = threadIdx.x; i < g.n_dn; i += kFewThreads) g.cnt_dn[i] = 0;
    }
    if (threadIdx.x < 2) g.gate[threadIdx.x] = 0;
    if (threadIdx.x == 2) *g.done = 0;
  }
}

template <int FMT>
cudaError_t prepare_one() {
  return cudaFuncSetAttribute(moe_few_kernel<FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
}

template <int FMT>
cudaError_t launch_one(const FewArgs& a, int grid, size_t smem, cudaStream_t st) {
  void* args[] = {const_cast<FewArgs*>(&a)};
  return cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(moe_few_kernel<FMT>), dim3(grid), dim3(kFewThreads),
                                     args, smem, st);
}

}  // namespace

// As many stages as fit (fewer where TMEM has to hold their scales).  A stage holds the activations of a slice:
// all tokens, or one expert's rows of h, twice in bf16.
size_t moe_few_smem(int prec, int T, int E, int k, int* stages, int* b_bytes) {
  const int sf = prec == 0 ? 0 : prec == 1 ? 3 * 512 : 3 * 2048;
  const int rows = ((prec == 0 ? 2 * T : T) + 15) / 16 * 16;
  *b_bytes = rows * 128;
  const size_t tail = few_tail_bytes(T, E, k) + 1024;
  const int most = prec == 2 ? 5 : kFewMaxStages;
  int n = (int)((232448 - tail) / (kFewABytes + *b_bytes + sf));
  *stages = n < most ? n : most;
  return (size_t)*stages * (kFewABytes + *b_bytes + sf) + tail;
}

cudaError_t prepare_moe_few(int prec) {
  return prec == 0 ? prepare_one<kFmtBf16>() : prec == 1 ? prepare_one<kFmtMx>() : prepare_one<kFmtNv>();
}

cudaError_t launch_moe_few(int prec, const FewArgs& a, int grid, size_t smem, cudaStream_t st) {
  return prec == 0   ? launch_one<kFmtBf16>(a, grid, smem, st)
         : prec == 1 ? launch_one<kFmtMx>(a, grid, smem, st)
                     : launch_one<kFmtNv>(a, grid, smem, st);
}

}  // namespace moe
