// head_gemm.cuh -- persistent tcgen05 GEMM of the loss head.
//
// With X [T, d] activations and W [V, d] the head's weight, logits z = X W^T
// are computed tile by tile and consumed in the epilogue:
//   kHeadLse  z tile -> per row (max, sum of exp) of 128 columns, and the
//             logits at the row's target entries; nothing else leaves the SM
//   kHeadDl   z tile again -> D = (softmax - target) * upstream, bf16, one
//             piece of the vocabulary at a time
//   kHeadDX   D . W      (K = vocabulary piece) into fp32 sums
//   kHeadDW   D^T . X    (K = tokens), one bf16 rounding
//
// Roles per CTA (320 threads, 384 with two idle warps): warp 0 TMA producer, warp 1
// TMEM owner and MMA issuer, the last eight warps epilogue (two per TMEM lane
// quadrant, 128 columns each).
// CG = 1: one CTA computes a 128 x 256 tile.  CG = 2: a pair of CTAs computes
// 256 x 256; each holds its 128 rows of A and half of B's 256 columns, so an
// SM fetches 32 KB instead of 48 KB per 64-deep slice of K.
// Two TMEM accumulators of 256 columns overlap a tile's epilogue with the
// next tile's products.  Tiles are handed out statically and every sum has
// one fixed order: bitwise repeatable.
//
// Measured at 2048 tokens, 7168 x 32768 (0.96 TFLOP each): D 546 us, dX 486,
// dW 497, tensor pipe 80, 93 and 87% busy; back to back the power limit holds
// them to 1.65 PFLOP/s, and 4096 tokens' forward at 7168 x 65536 to 1.62.  With
// few tokens reading W bounds the forward (one token, 7168 x 400000: 6.9 TB/s).
// Rows whose byte length is not a multiple of 32 cost the products a quarter
// (width 1000 against 1008): each row of a TMA box then touches one sector more.
//
// The tensor cores add into fp32 accumulators with truncation, which pulls a
// 7168-long dot product towards zero by about 7e-6 of its value (measured
// against 64 bits).  The loss is a difference of logits, and D the difference of
// the softmax and its target, so both logits products end an accumulator every
// kLogitsChunk slices of K and add the parts in registers, rounded to nearest.
// The runs are the same in both directions: D subtracts from the very logits that
// the log-sum-exp was taken of.  With D in one run over K, gradients of tokens
// predicted with 0.997 to 0.9995 at width 7168, from logits of 40, were off by 40%
// (norm of a row of dX); in parts they are off by 0.24%.  The sums dX and dW, of
// entries of D that were rounded to bf16, do not need it.  (D in one run took 514 us.)
#pragma once
#include "head.h"
#include "pdl.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kHBM = 128;                    // rows per CTA
constexpr int kHBK = 64;                     // K slice (128 bytes of bf16)
constexpr int kHeadEpiWarps = 8;
// Adding up a logit's parts takes 128 registers beside what the epilogue needs, and 320 threads get
// 168 each: they spilled 160-220 bytes in kHeadLse.  The kernels with parts have two idle warps more,
// so that the first four make a warpgroup that hands registers to the epilogue's two.
constexpr int kLaunchRegs = 168, kFewRegs = 56, kEpiRegs = 224;
template <int KIND, bool PARTS>
constexpr bool head_regs = KIND == kHeadLse || (KIND == kHeadDl && PARTS);
template <int KIND, bool PARTS>
constexpr int head_threads = (head_regs<KIND, PARTS> ? 4 : 2) * 32 + kHeadEpiWarps * 32;
static_assert(4 * kFewRegs + kHeadEpiWarps * kEpiRegs <= 12 * kLaunchRegs, "the shares come out of the launch's registers");
constexpr int kLogitsChunk = 16;             // K slices per accumulator of the logits products (1024), and
constexpr int kLogitsChunkFew = 8;           // of up to 64 tokens (512), whose epilogues have the time
constexpr int logits_chunk(int arows) { return arows == kHBM ? kLogitsChunk : kLogitsChunkFew; }

// AR rows of A are fetched per CTA: 128, or 16 or 64 when the call has no more
// tokens.  The product still covers 128 rows -- those past AR read whatever
// follows in shared memory, and no one reads their results -- but the stages get
// smaller, and more of W is on its way, which is what a call of few tokens waits
// for.  Epilogue warps of rows past 64 then only hand the accumulator back.  In dX: backward
// of 64 tokens, 2048 x 32768, 3.6 us less with 64 rows of D per stage than with 128.
template <int KIND, int CG, int AR>
struct HeadTraits {
  static_assert(AR == kHBM || (CG == 1 && KIND <= kHeadDX));
  static constexpr bool a_mn = KIND == kHeadDW;
  static constexpr bool b_mn = KIND == kHeadDX || KIND == kHeadDW;
  static constexpr int a_bytes = AR * kHBK * 2;               // 16 KB for 128 rows
  static constexpr int b_rows = kHeadBN / CG;
  static constexpr int b_bytes = b_rows * kHBK * 2;           // 32 / 16 KB
  static constexpr int stage_bytes = a_bytes + b_bytes;
  // staging per epilogue warp: 32 rows of 128 bytes
  static constexpr int staging = KIND == kHeadLse ? 0 : 4096;
  static constexpr int staging_warps = AR == kHBM ? kHeadEpiWarps : kHeadEpiWarps / 2;
  static constexpr int spare = staging_warps * staging + 1024 + 256;
  static constexpr int stages = AR == kHBM ? (CG == 2 ? 6 : 4) : (232448 - spare) / stage_bytes;
  static constexpr int smem_bytes = stages * stage_bytes + spare;
};

struct HeadTile {
  int64_t row0;    // first row of the tile (compact rows, or vocabulary rows of the piece)
  int64_t col0;    // first column (vocabulary inside the piece, or d)
  int kb0, nkb;    // K slices
  int split;
};

// Columns of a tile: 256; up to 64 tokens' logits products take what the call
// says (64, 128, 192 or 256).  dX's tiles stay 256 wide: its copies of W are whole
// groups of four 64-column boxes, which the stage's byte count has to match.
template <int KIND, int AR>
__device__ __forceinline__ int head_bn(const HeadArgs& g) {
  return AR == kHBM || KIND > kHeadDl ? kHeadBN : g.bn;
}

template <int KIND, int CG, int AR>
__device__ __forceinline__ int64_t head_tiles(const HeadArgs& g, int na, int& MT, int& NT) {
  constexpr int TM = kHBM * CG;
  const int64_t mrows = KIND == kHeadDW ? g.vlen : na;
  const int64_t ncols = KIND <= kHeadDl ? g.vlen : g.d;
  const int bn = head_bn<KIND, AR>(g);
  MT = (int)((mrows + TM - 1) / TM);
  NT = (int)((ncols + bn - 1) / bn);
  return (int64_t)MT * NT * (KIND == kHeadDX ? g.nsplit : 1);
}

template <int KIND, int CG, int AR>
__device__ __forceinline__ HeadTile head_tile(const HeadArgs& g, int na, int MT, int NT, int64_t w) {
  HeadTile t;
  t.split = 0;
  int64_t mt, nt;
  if (KIND == kHeadDW) {
    // d tiles fastest: the piece's D^T block is read by neighbours, X stays in L2
    mt = w / NT;
    nt = w - mt * NT;
  } else {
    // row tiles fastest: a W tile is read by neighbours, X (or D) stays in L2
    const int64_t per = (int64_t)MT * NT;
    t.split = (int)(w / per);
    const int64_t local = w - t.split * per;
    nt = local / MT;
    mt = local - nt * MT;
  }
  t.row0 = mt * (kHBM * CG);
  t.col0 = nt * head_bn<KIND, AR>(g);
  t.kb0 = 0;
  if (KIND == kHeadDX) {
    const int nkb = (int)((g.vlen + kHBK - 1) / kHBK);
    const int base = nkb / g.nsplit, rem = nkb % g.nsplit;
    t.nkb = base + (t.split < rem ? 1 : 0);
    t.kb0 = t.split * base + min(t.split, rem);
  } else {
    t.nkb = ((KIND == kHeadDW ? na : g.d) + kHBK - 1) / kHBK;
  }
  return t;
}

// Accumulators (TMEM phases) of one tile.
template <int KIND, int AR, bool PARTS>
__device__ __forceinline__ int head_phases(int nkb) {
  return KIND == kHeadLse || (KIND == kHeadDl && PARTS) ? (nkb + logits_chunk(AR) - 1) / logits_chunk(AR) : 1;
}

// ---------------------------------------------------------------- pair (cta_group::2) pieces
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t mapa_u32(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* m, int32_t x, int32_t y,
                                                 uint32_t bar_cluster, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar_cluster), "l"(policy)
      : "memory");
}
template <int CG>
__device__ __forceinline__ void head_tmem_alloc(uint32_t* slot) {
  if constexpr (CG == 1) {
    tmem_alloc(slot, 512);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void head_tmem_free(uint32_t taddr) {
  if constexpr (CG == 1)
    tmem_dealloc(taddr, 512);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(512) : "memory");
}
template <int CG>
__device__ __forceinline__ void head_mma(uint32_t d_tmem, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t accum) {
  if constexpr (CG == 1)
    umma_bf16(d_tmem, ad, bd, idesc, accum);
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(ad), "l"(bd), "r"(idesc), "r"(accum)
        : "memory");
}
// Arrive on `bar` of this CTA (and of its peer, CG = 2) once the MMAs issued so far completed.
template <int CG>
__device__ __forceinline__ void head_commit(uint64_t* bar) {
  if constexpr (CG == 1)
    umma_commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
// An epilogue warp's lanes hold one row each; rows are transposed through 32
// x 128 bytes of shared memory so that eight lanes write a row's 128 bytes
// together.  (TMA stores of the same blocks cost a proxy fence and a wait per block:
// the fences alone were a fifth of these warps' time.)  16-byte chunk c
// of row r sits at c ^ (r & 7).
__device__ __forceinline__ void stage_put(uint8_t* buf, int lane, int c, uint4 v) {
  *reinterpret_cast<uint4*>(buf + lane * 128 + ((c ^ (lane & 7)) << 4)) = v;
}
__device__ __forceinline__ uint4 stage_get(const uint8_t* buf, int r, int c) {
  return *reinterpret_cast<const uint4*>(buf + r * 128 + ((c ^ (r & 7)) << 4));
}

// What an epilogue lane needs to know about its row and the row's target
// entries inside its 128 columns.  The next tile's are fetched while the
// current one is worked on, in the three dependent steps below.
template <bool TEACHER>
struct HeadRow {
  int tok;             // token, -1 past the rows that count
  int cnt;             // TEACHER: entries in use; else the label
  float rl, gr;        // kHeadDl: log-sum-exp, upstream gradient over the common factor
  int e;               // next entry
  int id0, id1;        // next two entries' vocabulary ids, INT_MAX past the list
  float p0, p1;

  template <bool DIRECT>
  __device__ __forceinline__ void fetch_record(const HeadArgs& g, int64_t row, int na) {
    int4 q = make_int4(-1, 0, 0, 0);
    if (DIRECT && !g.n_active) {
      if (row < na) {
        const int64_t n = TEACHER ? (int64_t)__ldg(g.cnt + row)
                          : g.ids64 ? __ldg(reinterpret_cast<const long long*>(g.labels) + row)
                                    : (int64_t)__ldg(reinterpret_cast<const int*>(g.labels) + row);
        if (TEACHER ? n > 0 : n >= 0 && n < g.V) q = make_int4((int)row, (int)n, 0, 0);
      }
    } else if (row < na) {
      q = __ldg(g.rec + row);
    }
    tok = q.x;
    cnt = q.y;
    rl = __int_as_float(q.z);
    gr = __int_as_float(q.w);
  }
  __device__ __forceinline__ void find_first(const HeadArgs& g, int64_t vcol) {
    if constexpr (TEACHER)
      e = tok >= 0 ? (int)__ldg(g.first + (int64_t)tok * g.blocks + min(vcol / 128, g.blocks - 1)) : 0;
  }
  __device__ __forceinline__ void load(const HeadArgs& g, int i, int& id, float& p) {
    const bool in = tok >= 0 && i < cnt;
    id = in ? __ldg(g.ids + (int64_t)tok * g.K + i) : INT_MAX;
    p = in ? __ldg(g.probs + (int64_t)tok * g.K + i) : 0.0f;
  }
  __device__ __forceinline__ void fetch_entries(const HeadArgs& g, int64_t vcol) {
    if constexpr (TEACHER) {
      load(g, e, id0, p0);
      load(g, e + 1, id1, p1);
      while (id0 < vcol) next(g);        // the table's block may start before the column
    } else {
      e = 0;
      id0 = tok >= 0 && cnt >= vcol ? cnt : INT_MAX;
      p0 = 1.0f;
    }
  }
  __device__ __forceinline__ void next(const HeadArgs& g) {
    ++e;
    if constexpr (TEACHER) {
      id0 = id1;
      p0 = p1;
      load(g, e + 1, id1, p1);
    } else {
      id0 = INT_MAX;
    }
  }
};

// v[col] of 32 registers: 31 selections by the bits of col.
__device__ __forceinline__ float pick32(const float* v, int col) {
  float t[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) t[i] = (col & 1) ? v[2 * i + 1] : v[2 * i];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = (col & 2) ? t[2 * i + 1] : t[2 * i];
#pragma unroll
  for (int i = 0; i < 4; ++i) t[i] = (col & 4) ? t[2 * i + 1] : t[2 * i];
  t[0] = (col & 8) ? t[1] : t[0];
  t[2] = (col & 8) ? t[3] : t[2];
  return (col & 16) ? t[2] : t[0];
}

// PARTS (kHeadDl): a logit has several parts.  Widths with one (up to 1024, or 512 for up to 64 tokens) have
// a kernel of their own, without the registers for more: distillation backward of 2048 tokens, 512 x
// 32768, K = 64, 196 us against 204 with one kernel for all widths.
template <int KIND, int CG, bool TEACHER, int AR, bool PARTS>
__global__ void __launch_bounds__(head_threads<KIND, PARTS>, 1) head_gemm_kernel(const __grid_constant__ HeadArgs g) {
  using TR = HeadTraits<KIND, CG, AR>;
  constexpr int kSt = TR::stages;
  extern __shared__ uint8_t smem_raw[];
  // every CTA of a launch has the same dynamic shared-memory base, so a pair's layouts coincide
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* stage_base = smem;
  uint8_t* staging_base = smem + kSt * TR::stage_bytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging_base + TR::staging_warps * TR::staging);
  uint64_t* full = bars;                 // used in the leader CTA
  uint64_t* empty = bars + kSt;
  uint64_t* tfull = bars + 2 * kSt;
  uint64_t* tempty = bars + 2 * kSt + 2; // used in the leader CTA
  uint64_t* drain = bars + 2 * kSt + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kSt + 5);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kSt; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], kHeadEpiWarps * CG);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&g.mapA0);
    tma_prefetch_desc(&g.mapB0);
  }
  if (warp == 1) {
    head_tmem_alloc<CG>(tmem_slot);
    tc_fence_before();
  }
  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // dW behind dX reads nothing that dX writes, and dX let it start only after
  // everything earlier was complete: the two overlap, and dW waits at its end,
  // so that whatever follows finds both complete.
  const bool beside = KIND == kHeadDW && g.beside;
  if (!beside) {
    pdl_wait();
    pdl_release();
  }
  WaitCtl wc{g.status, abort_flag, g.timeout_ns};

  const int na = KIND == kHeadLse && !g.n_active ? g.T : *g.n_active;
  int MT, NT;
  const int64_t nwork = head_tiles<KIND, CG, AR>(g, na, MT, NT);
  const int bn = head_bn<KIND, AR>(g);
  const int64_t w0 = blockIdx.x / CG;
  const int64_t wstep = gridDim.x / CG;

  constexpr int kEpi0 = head_threads<KIND, PARTS> / 32 - kHeadEpiWarps;      // the epilogue's first warp
  if (warp < kEpi0) {
    if constexpr (head_regs<KIND, PARTS>) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    if (warp == 0) {
      if (lane == 0) {
        // ------------------------------------------------------------ producer
        fence_proxy_async_global();                       // the predecessors' plain stores, read by TMA below
        const uint64_t pol = policy_evict_last();
        const uint64_t pol_b = (KIND == kHeadLse || KIND == kHeadDX) && g.T <= kHBM * CG ? policy_evict_first() : pol;
        const bool all = na == g.T;                       // no row skipped: X is read in place
        const CUtensorMap* mA = (KIND <= kHeadDl && !all) ? &g.mapA1 : &g.mapA0;
        const CUtensorMap* mB = (KIND == kHeadDW && !all) ? &g.mapB1 : &g.mapB0;
        uint32_t s = 0, ph = 0, issued = 0, last_par = 0;
        bool ok = true;
        for (int64_t w = w0; w < nwork && ok && !g.stall; w += wstep) {
          const HeadTile t = head_tile<KIND, CG, AR>(g, na, MT, NT, w);
          const int64_t arow = t.row0 + rank * kHBM;          // this CTA's rows of A
          const int64_t bcol = t.col0 + rank * TR::b_rows;    // and columns of B
          for (int kb = 0; kb < t.nkb; ++kb) {
            if (!mbar_wait(&empty[s], ph ^ 1, wc)) { ok = false; break; }
            if (leader) mbar_arrive_expect_tx(&full[s], TR::a_bytes * CG + bn * kHBK * 2);
            uint8_t* sa = stage_base + s * TR::stage_bytes;
            uint8_t* sb = sa + TR::a_bytes;
            const int32_t k0 = (t.kb0 + kb) * kHBK;
            const uint32_t bar_c = CG == 2 ? mapa_u32(smem_u32(&full[s]), 0) : 0;
            auto load = [&](uint8_t* dst, const CUtensorMap* m, int64_t x, int64_t y, uint64_t pol) {
              if constexpr (CG == 1) tma_load_2d(dst, m, (int32_t)x, (int32_t)y, &full[s], pol);
              else tma_load_2d_pair(dst, m, (int32_t)x, (int32_t)y, bar_c, pol);
            };
            if (KIND == kHeadDW) {
  #pragma unroll
              for (int j = 0; j < kHBM / 64; ++j) load(sa + j * 8192, mA, arow + j * 64, k0, pol);
            } else {
              load(sa, mA, k0, arow, pol);
            }
            if (KIND == kHeadDX || KIND == kHeadDW) {
              const int64_t krow = (KIND == kHeadDX ? g.v0 : 0) + k0;
  #pragma unroll
              for (int j = 0; j < TR::b_rows / 64; ++j) load(sb + j * 8192, mB, bcol + j * 64, krow, pol_b);
            } else {
              load(sb, mB, k0, g.v0 + bcol, pol_b);
            }
            issued |= 1u << s;
            last_par = (last_par & ~(1u << s)) | (ph << s);
            if (++s == kSt) { s = 0; ph ^= 1; }
          }
        }
        if (!ok) {
          // abort: give every issued copy time to land before the CTA may exit
          // (the barriers are the leader's; its peer waits a fixed time)
          const uint64_t t0 = globaltimer_ns();
          if (leader) {
            for (int st = 0; st < kSt; ++st) {
              if (!(issued & (1u << st))) continue;
              while (!mbar_try_wait(&full[st], (last_par >> st) & 1u))
                if (globaltimer_ns() - t0 > 50000000ull) break;
            }
          } else {
            while (globaltimer_ns() - t0 < 5000000ull) __nanosleep(1000);
          }
        }
      }
    } else if (warp == 1) {
      if (lane == 0 && leader) {
        // ------------------------------------------------------------ MMA issuer
        const uint32_t idesc = idesc_bf16(kHBM * CG, bn, TR::a_mn ? 1 : 0, TR::b_mn ? 1 : 0);
        uint32_t s = 0, ph = 0, acc = 0, aph = 0;
        bool ok = true;
        for (int64_t w = w0; w < nwork && ok; w += wstep) {
          const HeadTile t = head_tile<KIND, CG, AR>(g, na, MT, NT, w);
          if (t.nkb == 0) continue;
          const int phases = head_phases<KIND, AR, PARTS>(t.nkb);
          const int len = t.nkb / phases, longer = t.nkb - len * phases;
          int k_hi = 0;
          for (int p = 0; p < phases && ok; ++p) {
            const int k_lo = k_hi;
            k_hi += len + (p < longer ? 1 : 0);
            if (!mbar_wait(&tempty[acc], aph ^ 1, wc)) { ok = false; break; }
            tc_fence_after();
            const uint32_t d_tmem = tmem_base + acc * kHeadBN;
            for (int kb = k_lo; kb < k_hi; ++kb) {
              if (!mbar_wait(&full[s], ph, wc)) { ok = false; break; }
              tc_fence_after();
              const uint32_t sa = smem_u32(stage_base + s * TR::stage_bytes);
              const uint32_t sb = sa + TR::a_bytes;
  #pragma unroll
              for (int kk = 0; kk < kHBK / 16; ++kk) {
                const uint64_t ad =
                    TR::a_mn ? sdesc_sw128(sa + kk * 2048, 8192, 1024) : sdesc_sw128(sa + kk * 32, 16, 1024);
                const uint64_t bd =
                    TR::b_mn ? sdesc_sw128(sb + kk * 2048, 8192, 1024) : sdesc_sw128(sb + kk * 32, 16, 1024);
                head_mma<CG>(d_tmem, ad, bd, idesc, (kb > k_lo || kk) ? 1u : 0u);
              }
              head_commit<CG>(&empty[s]);
              if (++s == kSt) { s = 0; ph ^= 1; }
            }
            if (!ok) break;
            head_commit<CG>(&tfull[acc]);
            acc ^= 1;
            if (acc == 0) aph ^= 1;
          }
        }
        if (!ok) {  // abort: let the products in flight finish before TMEM is freed
          head_commit<CG>(drain);
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(drain, 0))
            if (globaltimer_ns() - t0 > 50000000ull) break;
        }
      }
    }
  } else {
    // -------------------------------------------------------------- epilogue
    if constexpr (head_regs<KIND, PARTS>) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    const int q = warp & 3;                 // TMEM lane quadrant of this warp
    const int h = (warp - kEpi0) >> 2;      // column half
    const bool idle = AR != kHBM && q >= 2; // rows past 64 of a call with no more
    uint8_t* stg = staging_base + (AR == kHBM ? warp - kEpi0 : 2 * h + (q & 1)) * TR::staging;
    uint32_t acc = 0, aph = 0;
    [[maybe_unused]] const float c2 = g.inv_temp * 1.4426950408889634f;   // logits to base-2 exponents
    auto release = [&](uint32_t a) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 1) mbar_arrive(&tempty[a]);
        else mbar_arrive_cluster(mapa_u32(smem_u32(&tempty[a]), 0));
      }
    };
    const uint32_t lane_off = (uint32_t)(32 * q) << 16;
    const int sub = lane >> 3, chunk = lane & 7;                  // coalesced writes: row within 4, 16-byte chunk
    [[maybe_unused]] const float sc = KIND >= kHeadDX ? *g.scale * g.out_scale : 1.0f;
    [[maybe_unused]] HeadRow<TEACHER> cur, nxt;
    const int half = bn / 2;                                      // columns of a warp: 32, 64, 96 or 128
    if constexpr (KIND <= kHeadDl) {
      if (w0 < nwork && !idle) {
        const HeadTile t = head_tile<KIND, CG, AR>(g, na, MT, NT, w0);
        const int64_t vcol = g.v0 + t.col0 + h * half;
        nxt.template fetch_record<KIND == kHeadLse>(g, t.row0 + rank * kHBM + 32 * q + lane, na);
        nxt.find_first(g, vcol);
        nxt.fetch_entries(g, vcol);
      }
    }
    for (int64_t w = w0; w < nwork; w += wstep) {
      const HeadTile t = head_tile<KIND, CG, AR>(g, na, MT, NT, w);
      if (idle) {
        bool ok = true;
        const int phases = t.nkb > 0 ? head_phases<KIND, AR, PARTS>(t.nkb) : 0;
        for (int p = 0; p < phases && ok; ++p) {
          ok = mbar_wait(&tfull[acc], aph, wc);
          if (!ok) break;
          tc_fence_after();
          release(acc);
          acc ^= 1;
          if (acc == 0) aph ^= 1;
        }
        if (!ok) break;
        continue;
      }
      const int64_t rowq = t.row0 + rank * kHBM + 32 * q;         // the warp's first row
      const int64_t row = rowq + lane;                            // this lane's row
      const int64_t colh = t.col0 + h * half;                     // the warp's first column

      if constexpr (KIND <= kHeadDl) {
        cur = nxt;
        const int64_t vcol = g.v0 + colh;                         // vocabulary id of the first column
        const bool more = w + wstep < nwork;
        int64_t nvcol = 0;
        if (more) {
          const HeadTile n = head_tile<KIND, CG, AR>(g, na, MT, NT, w + wstep);
          nvcol = g.v0 + n.col0 + h * half;
          nxt.template fetch_record<KIND == kHeadLse>(g, n.row0 + rank * kHBM + 32 * q + lane, na);
        }
        const int64_t left = min((int64_t)half, g.vlen - colh);   // its columns inside the vocabulary
        const int last = (int)vcol + half;                        // ids below it are this block's
        // the row's 128 logits; kHeadDl takes the last part as it goes, 32 columns at a time
        float z[128] = {};
        const int phases = head_phases<KIND, AR, PARTS>(t.nkb);
        const int whole = KIND == kHeadLse ? phases : phases - 1;   // 0 without PARTS
        bool ok = true;
        for (int p = 0; p < whole; ++p) {
          if (!mbar_wait(&tfull[acc], aph, wc)) { ok = false; break; }
          tc_fence_after();
          const uint32_t tb = tmem_base + lane_off + acc * kHeadBN + h * half;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c * 32 >= half) break;
            uint32_t r[32];
            tmem_ld32(tb + c * 32, r);
            tmem_ld_wait();
            if (p == 0) {
#pragma unroll
              for (int i = 0; i < 32; ++i) z[c * 32 + i] = __uint_as_float(r[i]);
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) z[c * 32 + i] += __uint_as_float(r[i]);
            }
          }
          release(acc);
          acc ^= 1;
          if (acc == 0) aph ^= 1;
        }
        if (!ok) break;
        if constexpr (KIND == kHeadLse) {
          if (more) nxt.find_first(g, nvcol);
          // logits at this row's target entries inside these 128 columns
          while (__any_sync(0xffffffffu, cur.id0 < last)) {
            const int col = (cur.id0 - (int)vcol) & 127;
            float v[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = pick32(z + c * 32, col);
            const float lo = (col & 32) ? v[1] : v[0], hi = (col & 32) ? v[3] : v[2];
            if (cur.id0 < last) {
              g.zt[(int64_t)cur.tok * g.K + cur.e] = (col & 64) ? hi : lo;
              cur.next(g);
            }
          }
          if (more) nxt.fetch_entries(g, nvcol);
          if (left < 128) {
#pragma unroll
            for (int i = 0; i < 128; ++i)
              if (i >= left) z[i] = -INFINITY;
          }
          float m4[4] = {z[0], z[1], z[2], z[3]};
#pragma unroll
          for (int i = 4; i < 128; ++i) m4[i & 3] = fmaxf(m4[i & 3], z[i]);
          const float m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          const float mb = m == -INFINITY ? 0.0f : m * c2;        // a block without columns sums to 0
          const float md = m == -INFINITY ? 0.0f : fmaf(m, c2, -mb);   // the sum is taken about m, not about mb
          float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int i = 0; i < 128; ++i) s4[i & 3] += ex2_approx(fmaf(z[i], c2, -mb));
          g.part[(2 * (t.col0 / bn) + h) * g.Tp + row] =
              make_float2(m * g.inv_temp, ((s4[0] + s4[1]) + (s4[2] + s4[3])) * ex2_approx(-md));
        } else {
          if (!mbar_wait(&tfull[acc], aph, wc)) break;
          tc_fence_after();
          const uint32_t tb = tmem_base + lane_off + acc * kHeadBN + h * half;
          uint32_t r[32];
          tmem_ld32(tb, r);
          __nv_bfloat16* out = g.dl + (rowq + sub) * g.ldl + colh + chunk * 8;
#pragma unroll
          for (int c = 0; c < 4; ++c) {                           // 32 columns at a time, stored by 64
            if (c * 32 >= half) break;
            tmem_ld_wait();
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
            if (whole > 0) {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = z[c * 32 + i] + v[i];
            }
            if (c * 32 + 32 < half) tmem_ld32(tb + (c + 1) * 32, r);
            else release(acc);
            // the difference first: near the log-sum-exp it is exact, and its size sets the rounding
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = ex2_approx(fmaf(v[i], g.inv_temp, -cur.rl) * 1.4426950408889634f);
            const int until = (int)vcol + c * 32 + 32;
            while (__any_sync(0xffffffffu, cur.id0 < until)) {
              const bool hit = cur.id0 < until;
              const int col = hit ? cur.id0 - (int)vcol - c * 32 : -1;
              const float p = cur.p0;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i == col) v[i] -= p;
              if (hit) cur.next(g);
            }
            if (c == 0 && more) nxt.find_first(g, nvcol);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= cur.gr;
            if (left < half || rowq + 32 > na) {                   // zeros past the vocabulary and the rows that count
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (c * 32 + i >= left || cur.tok < 0) v[i] = 0.0f;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) stage_put(stg, lane, (c & 1) * 4 + k, pack8(v + 8 * k));
            if ((c & 1) || c * 32 + 32 >= half) {
              __syncwarp();
              const int x = (c & ~1) * 32 + chunk * 8;
              if (x < half && colh + x < g.ldl) {
#pragma unroll
                for (int it = 0; it < 8; ++it)
                  *reinterpret_cast<uint4*>(out + (int64_t)(4 * it) * g.ldl + (c & ~1) * 32) =
                      stage_get(stg, 4 * it + sub, chunk);
              }
              __syncwarp();
            }
          }
          if (more) nxt.fetch_entries(g, nvcol);
          acc ^= 1;
          if (acc == 0) aph ^= 1;
        }
      } else {
        const bool has = t.nkb > 0;
        const bool final_dx = KIND == kHeadDX && g.dX != nullptr;
        int tok = -1;
        if (final_dx && row < na) tok = __ldg(g.rec + row).x;
        if (has) {
          if (!mbar_wait(&tfull[acc], aph, wc)) break;
          tc_fence_after();
        }
        const uint32_t tb = tmem_base + lane_off + acc * kHeadBN + h * 128;
        uint32_t r[32];
        if (has) {
          tmem_ld32(tb, r);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) r[i] = 0u;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (has) tmem_ld_wait();
          const int64_t col = colh + c * 32;
          if (KIND == kHeadDX && !final_dx) {
            // fp32 sums, 32 columns at a time
#pragma unroll
            for (int k = 0; k < 8; ++k)
              stage_put(stg, lane, k, make_uint4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]));
            if (has) {
              if (c < 3) tmem_ld32(tb + (c + 1) * 32, r);
              else release(acc);
            }
            __syncwarp();
            if (col + chunk * 4 < g.d) {
              float* out = g.acc + (t.split * g.Tp + rowq + sub) * g.d + col + chunk * 4;
              float4 old[8];
              if (g.add) {
#pragma unroll
                for (int it = 0; it < 8; ++it)
                  old[it] = *reinterpret_cast<const float4*>(out + (int64_t)(4 * it) * g.d);
              }
#pragma unroll
              for (int it = 0; it < 8; ++it) {
                const uint4 u = stage_get(stg, 4 * it + sub, chunk);
                float4 v = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z),
                                       __uint_as_float(u.w));
                if (g.add) v.x += old[it].x, v.y += old[it].y, v.z += old[it].z, v.w += old[it].w;
                *reinterpret_cast<float4*>(out + (int64_t)(4 * it) * g.d) = v;
              }
            }
            __syncwarp();
            continue;
          }
          // bf16 results, stored 64 columns at a time
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
          if (has) {
            if (c < 3) tmem_ld32(tb + (c + 1) * 32, r);
            else release(acc);
          }
          if (KIND == kHeadDX && g.add && tok >= 0) {             // the earlier pieces' sums
            const float4* src = reinterpret_cast<const float4*>(g.acc + row * g.d + col);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (col + 4 * k < g.d) {
                const float4 o = src[k];
                v[4 * k] += o.x, v[4 * k + 1] += o.y, v[4 * k + 2] += o.z, v[4 * k + 3] += o.w;
              }
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] *= sc;
#pragma unroll
          for (int k = 0; k < 4; ++k) stage_put(stg, lane, (c & 1) * 4 + k, pack8(v + 8 * k));
          if (!(c & 1)) continue;
          __syncwarp();
          const int64_t x = col - 32 + chunk * 8;
#pragma unroll
          for (int it = 0; it < 8; ++it) {
            const int rr = 4 * it + sub;
            const uint4 u = stage_get(stg, rr, chunk);
            if constexpr (KIND == kHeadDX) {
              const int to = __shfl_sync(0xffffffffu, tok, rr);
              if (to >= 0 && x < g.d) *reinterpret_cast<uint4*>(g.dX + (int64_t)to * g.d + x) = u;
            } else {
              if (rowq + rr < g.vlen && x < g.d)
                __stcs(reinterpret_cast<uint4*>(g.dW + (g.v0 + rowq + rr) * g.d + x), u);
            }
          }
          __syncwarp();
        }
        if (has) {
          acc ^= 1;
          if (acc == 0) aph ^= 1;
        }
      }
    }
  }

  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();   // no arrival or copy may target a CTA that has left
  if (warp == 1) {
    tc_fence_after();
    head_tmem_free<CG>(tmem_base);
  }
  if (beside) pdl_wait();
}

}  // namespace moe
