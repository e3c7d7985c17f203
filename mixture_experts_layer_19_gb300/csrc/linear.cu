// linear.cu -- a projection shared by many requests, each with a low-rank adapter
// of its own or none:
//   y_t = W x_t + scale_a B_a (A_a x_t),   a = adapter of token t
//
// Launches: the adapters' low side u_t = scale_a A_a x_t, then the product with W, to which
// each adapter of a block of tokens adds slices of K, 32 columns of B_a (16 for ranks up to 16) against u.  u is an fp32
// sum, held as a bf16 value and what its rounding left (2^-16 of it at most is lost, 2.5e-6 as a rule), and for fp32
// results what that left (2^-24).
//
// The tokens are the A operand of the tensor cores, up to 128 of them to a CTA, and so lanes of the accumulator: an
// adapter's products leave the lanes of other adapters' tokens alone.  The rows of W are the B operand, 256 of them to a
// tile (of one CTA or of a pair: on_pairs), or 128 for up to 64 tokens, whose calls wait for W and B: there u comes from dot products, and the adapters of
// the call are found by the kernel itself.  Where the low side is large (kDotWork) u comes from the same kernel with the
// stacked A in the place of W (only the row tiles of adapters that a block of tokens has), from lists made by the launch
// before.  All adapters of a block meet the same u, in other lanes, so a stage holds several adapters' B; up to 64 tokens
// fetch u once (64 tokens, 2048 x 32768, 32 adapters of rank 32: 47 us; 12 us more with u beside each adapter's B), more
// tokens once per stage (777 x 1000 x 5001, 200 adapters of rank 16 in turn: 54 us, 83 with one adapter to a stage).
// (With the tokens as columns and W as lanes, 128 tokens' products read as much shared memory as an SM
// gives: a slice of K took 0.47 us instead of 0.37.  And an adapter's products then need zeros in the rows of the others.)
//
// What does not fill a wave of tiles is cut along K into shares of equal bytes, where that pays; the CTAs take them first.
// A cut tile's parts go to memory; each of its CTAs adds up, in order, a share of its columns, while
// the products of its whole tiles go on.  A CTA whose tile is not complete after kPatience leaves its share to the one that
// completes it, so no CTA depends on another's being on the GPU at the same time (on streams of other priorities, two
// calls can each hold SMs that the other still needs).
// The tensor cores add into fp32 with truncation (8e-6 of a 7168-long sum), so fp32 results end
// an accumulator every 512 products and add the parts in registers: 5e-7 (1024 products: 1.7e-6; fp32 multiply-adds:
// 1e-7 to 4e-7).  bf16 results do not need it.
// Every sum has one fixed order: bitwise repeatable.
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>
#include <string>

#include "few.cuh"
#include "kernels.h"
#include "moe.h"
#include "pair.cuh"
#include "pdl.cuh"

namespace {

using namespace moe;

constexpr int kMaxRank = 256;
constexpr int kFew = 64;             // up to so many tokens: tiles of 128 rows of W, u by dot products
constexpr int kBlock = 128;          // most tokens of a tile
constexpr int kRowsFew = 128, kRowsWide = 256;                 // rows of W of a tile
constexpr int kRowsLow = 128;                                  // rows of the stacked A of a tile: a block has few adapters
constexpr int kMaxStages = 12;
// Up to so many multiply-adds of the low side go to dot products (always up to kFew tokens), with two launches in the
// place of three; twice as many where the stacked A is more than one tile, as products of whole tiles then do more than is
// needed, from lists.  (1024 x 2048, 8 adapters of rank 16, 34M multiply-adds: 26 us against 28 with products; 2048 tokens, 67M: 33
// against 31.  1024 x 7168, 64 adapters, 117M: 78 against 94; 512 x 7168, 8 adapters of rank 64, 235M: 76 against 63.)
constexpr int64_t kDotWork = 64 << 20;
constexpr uint64_t kPatience = 50000;                          // ns; parts of a tile come within a few us of each other
constexpr int kShares = kRowsWide / 32;                        // most CTAs that share a tile's join
constexpr int kLowRegs = 56, kHighRegs = 224, kLaunch = 168;   // registers of the warps, as in head_gemm.cuh

// More tokens: the adapters of a tile's tokens (of one block, or of a pair's two), and the lanes that have each.
template <int CG>
struct BlockList {
  int n, unused[3];
  int adapter[CG * kBlock];
  uint4 lanes[CG * kBlock][CG];
};
static_assert(sizeof(BlockList<1>) % 16 == 0 && sizeof(BlockList<2>) % 16 == 0, "copied in units of 16 bytes");

struct LinArgs {
  CUtensorMap mapW, mapX;            // boxes of a tile's rows, 64 columns
  CUtensorMap mapB;                  // [n, N, r]: boxes of a tile's rows of one adapter, `pc` columns
  CUtensorMap mapU, mapU3;           // [T, 3 pc per 32 of the rank]: boxes of two parts, and of the third
  const void* ids;                   // [T]
  const float* scale;                // [n] or null
  uint4* u;                          // [T][rank / 32]: pc columns of u as bf16, what their rounding left, and what that left
  void* out;                         // [T, N]
  float4* part;                      // [2 per CTA] parts of cut tiles
  int* cnt;                          // [tiles cut along K] parts that have come, and << 16 the shares that were left
  const int2* tiles;                 // low side: (row tile, token block) of each tile, and how many there are
  const int* n_tiles;
  const void* lists;                 // more tokens: a BlockList of each block, or of two
  int32_t* status;
  uint64_t timeout_ns;
  int64_t N;
  int T, d, n, r, nt, blocks;        // nt: tokens of a CTA's tile; blocks of them
  int pairs, groups;                 // the product runs on pairs of CTAs; blocks, or pairs of them
  int stages, chunk, least;          // K slices per accumulator; at least so many per part of a tile
  int out_f32, ids64, high, stall;   // high: adapters are added
  int all;                           // low side: the stacked A is one tile, which every block takes
  uint64_t patience;
  int u_bytes;                       // few tokens: room for u, 6 pc bytes per token and 32 of the rank
  int pc;                            // columns of a slice of the rank: 32, or 16 where there are no more
};

__device__ __forceinline__ int adapter_of(const LinArgs& g, int t) {
  if (t >= g.T) return -1;
  const int64_t a = g.ids64 ? (int64_t)__ldg(static_cast<const long long*>(g.ids) + t)
                            : (int64_t)__ldg(static_cast<const int*>(g.ids) + t);
  return a >= 0 && a < g.n ? (int)a : -1;
}
__device__ __forceinline__ int rank_slices(const LinArgs& g) { return (g.r + 31) / 32; }

// v as a bf16 value, and what that leaves.  A finite v beyond the largest bf16 value takes that one; an infinite one
// leaves nothing (inf - inf would make NaN of its products).
__device__ __forceinline__ float bf16_part(float v) {
  constexpr float kMost = 3.38953139e38f;
  const float b = __bfloat162float(__float2bfloat16_rn(v));
  return fabsf(v) < INFINITY ? fminf(fmaxf(b, -kMost), kMost) : b;
}
__device__ __forceinline__ float bf16_rest(float v, float b) { return fabsf(b) < INFINITY ? v - b : 0.0f; }

// u of one token and rank index: three bf16 values, pc columns apart.  A rank that ends inside a product's 16
// columns has zeros behind it (they meet zeros of B, but must not be NaN).
__device__ __forceinline__ __nv_bfloat16* u_at(const LinArgs& g, int t, int j) {
  return reinterpret_cast<__nv_bfloat16*>(g.u) + ((size_t)t * rank_slices(g) + j / 32) * (3 * g.pc) + j % 32;
}
__device__ __forceinline__ void put_u(const LinArgs& g, int t, int j, float v) {
  __nv_bfloat16* p = u_at(g, t, j);
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const float b = bf16_part(v);
    p[g.pc * i] = __float2bfloat16_rn(b);
    v = bf16_rest(v, b);
    if (g.r % 16 && j >= g.r - 8) p[g.pc * i + 8] = __float2bfloat16_rn(0.0f);
  }
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* m, int32_t x, int32_t y, int32_t z, uint64_t* bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
// As sdesc_sw128, for rows of 32, 64 or 128 bytes swizzled over their width: the upper half of the descriptor, and
// the whole.
__device__ __forceinline__ uint32_t sdesc_kind(int row_bytes) {
  return (uint32_t)(8 * row_bytes >> 4) | 1u << 14 | (row_bytes == 128 ? 2u : row_bytes == 64 ? 4u : 6u) << 29;
}
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr, uint32_t kind) {
  return (uint64_t)kind << 32 | ((saddr >> 4) & 0x3FFFu) | 1u << 16;
}
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* m, int32_t x, int32_t y, int32_t z,
                                                 uint32_t bar_cluster, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar_cluster), "l"(policy)
      : "memory");
}
// pair_mma that adds to the accumulator's lanes with a bit in `on` only (of a pair: 128 lanes of each CTA in turn).
template <int CG>
__device__ __forceinline__ void umma_lanes(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, const uint4 (&on)[CG]) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, 1, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%4, %5, %6, %7}, p;\n}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(~on[0].x), "r"(~on[0].y), "r"(~on[0].z), "r"(~on[0].w)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, 1, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, {%4, %5, %6, %7, %8, %9, %10, %11}, p;\n}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(~on[0].x), "r"(~on[0].y), "r"(~on[0].z), "r"(~on[0].w),
        "r"(~on[CG - 1].x), "r"(~on[CG - 1].y), "r"(~on[CG - 1].z), "r"(~on[CG - 1].w)
        : "memory");
}

// One CTA's segments in order: its share of the slices of the tiles that are cut, then whole tiles, one in each wave.
// A tile has K slices of the width and A slices of adapters, which cost kBase and `unit`; worker c of W starts at
// the slice in which cost start(c) falls.  The cut tiles follow the whole ones.
constexpr int kBase = 4;
// What joining the parts of cut tiles costs, in slices.
constexpr int kJoinFew = 8, kJoinWide = 24, kBesideFew = 2, kBesideWide = 8;
struct Walk {
  int K, A, unit, whole, S, W;       // S: cost of all cut tiles
  int tile, at, end;                 // next whole tile; next slice and end of the cut share
  // Cutting costs its joins, in slices of W: `join` of them where nothing else goes on meanwhile, else `beside`.
  __device__ __forceinline__ void init(int tiles, int least, int join, int beside, int G, int cta) {
    tile = cta;
    whole = tiles / G * G;
    S = (tiles - whole) * cost();
    W = min(G, max(1, S / (least * kBase)));
    if (S / W + (whole ? beside : join) * kBase >= cost()) whole = tiles, S = 0;
    const bool mine = S > 0 && cta < W;
    at = mine ? start(cta) : 0;
    end = mine ? start(cta + 1) : 0;
  }
  __device__ __forceinline__ int cost() const { return kBase * K + unit * A; }
  __device__ __forceinline__ int start(int c) const {
    const int64_t x = (int64_t)S * c / W;
    const int t = (int)(x / cost()), y = (int)(x - (int64_t)t * cost());
    return t * (K + A) + (y < kBase * K ? y / kBase : K + (y - kBase * K) / unit);
  }
  // The worker that has slice s: the last one whose start lies before the slice's end.
  __device__ __forceinline__ int owner(int s) const {
    const int t = s / (K + A), j = s - t * (K + A) + 1;
    const int64_t end_cost = (int64_t)t * cost() + (j <= K ? kBase * j : kBase * K + unit * (j - K));
    return (int)((end_cost * W - 1) / S);
  }
  // The tile, which of the cut tiles it is (-1: whole), first slice, slices.
  __device__ __forceinline__ bool next(int step, int& t, int& c, int& k0, int& len) {
    if (at < end) {
      c = at / (K + A);
      t = whole + c;
      k0 = at - c * (K + A);
      len = min(K + A - k0, end - at);
      at += len;
      return true;
    }
    if (tile >= whole) return false;
    t = tile;
    c = -1;
    k0 = 0;
    len = K + A;
    tile += step;
    return true;
  }
};

struct LinSmem {
  uint64_t full[kMaxStages], empty[kMaxStages], tfull[4], tempty[4], list_full[2], list_empty[2], drain, u_full;
  uint32_t tmem_slot;
  int abort_flag, n_list, ready[2], todo[2], left[2];
  int id[kFew], list[kFew];          // few tokens: their adapters, and the distinct ones in the order of first tokens,
  uint2 lanes[kFew];                 //   with their lanes
  float turn[kFewEpiWarps][16][33];  // an epilogue warp's 32 tokens x 16 columns, on their way to rows of the output
};

template <int CG>
__device__ __forceinline__ void lin_setup(const LinArgs& g, LinSmem& s, uint32_t rank) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < g.stages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s.tfull[i], 1);
      mbar_init(&s.tempty[i], CG * kFewEpiWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.list_full[i], 1);
      mbar_init(&s.list_empty[i], rank == 0 ? 2 : 1);               // the threads that load and that issue products
    }
    mbar_init(&s.drain, 1);
    mbar_init(&s.u_full, 1);
    s.abort_flag = 0;
    s.n_list = 0;
    fence_mbar_init();
    tma_prefetch_desc(&g.mapW);
    tma_prefetch_desc(&g.mapX);
    if (g.high) tma_prefetch_desc(&g.mapB);
  }
  if (threadIdx.x / 32 == 2) {
    pair_tmem_alloc<CG>(&s.tmem_slot);
    tc_fence_before();
  }
}

// Products in flight finish before TMEM is freed.
template <int CG>
__device__ __forceinline__ void lin_drain(LinSmem& s) {
  pair_commit<CG>(&s.drain);
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(&s.drain, 0))
    if (globaltimer_ns() - t0 > 50000000ull) break;
}

// Clears the accumulator of 128 lanes and kRowsFew columns: zeros times zeros (rows of 32 bytes).
__device__ __forceinline__ void umma_clear(uint32_t d_tmem, uint32_t zeros) {
  const uint64_t z = sdesc(zeros, sdesc_kind(32));
  umma_bf16(d_tmem, z, z, idesc_bf16(128, kRowsFew, 0, 0), 0);
}
constexpr int kZeroBytes = 128 * 32;

// BN: rows of W of a tile (128: the call's up to 64 tokens are one block).  PC: columns of a slice of the rank
// (constants here: the threads that issue loads and products are a bottleneck for few tokens).  LOW: the adapters' low side.
// CG = 2: pairs of CTAs, each with 128 tokens and half of the tile's rows of W.
template <int BN, int PC, bool LOW, int CG>
__global__ void __launch_bounds__(kFewThreads, 1) lin_kernel(const __grid_constant__ LinArgs g) {
  constexpr bool kOne = BN == kRowsFew && !LOW;
  // 64 columns of K at a time, two of them to a slice of 128-row tiles: 32 KB of W per
  // slice either way.  (With 16 KB, the single threads that issue loads and products took longer than the loads.)
  constexpr int kSub = kOne ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int St = g.stages;
  const int kX = g.nt * 128;                                        // products read 128 rows: those past nt read W, for no one
  // Accumulators in TMEM: with two of 128 columns, products waited for the epilogue every 512 of them (one token,
  // 7168 x 65536: 150 us against 143).
  constexpr int kAccs = 512 / BN;
  constexpr int kRows = BN / CG;                                    // rows of W of a CTA
  constexpr int kWt = kRows * 128;
  const int sub_bytes = kX + kWt, stage_bytes = kSub * sub_bytes;
  uint8_t* u_base = smem + St * stage_bytes;                        // kOne only, as are the zeros
  uint8_t* zeros = u_base + (kOne ? g.u_bytes : 0);
  using List = BlockList<CG>;                                       // more tokens: those of two segments, or of one
  constexpr int kLists = 2 / CG;
  List* lists = reinterpret_cast<List*>(u_base);
  LinSmem& s = *reinterpret_cast<LinSmem*>(kOne ? zeros + kZeroBytes : reinterpret_cast<uint8_t*>(lists + kLists));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = gridDim.x / CG, cta = blockIdx.x / CG;              // of pairs, the pair: they share a walk
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  const bool high = !LOW && g.high;
  const int RS = rank_slices(g);
  // Adapters' slices of the rank to a stage: as many as W's room holds, beside the third part of u where 32 columns wide
  // (one to a stage, whose latency the stages in flight then do not cover: 0.48 us each).
  constexpr int kRoom = (kOne ? 128 : 64) / PC;
  const int kHigh = kOne || PC == 16 || !g.out_f32 ? kRoom : kRoom / 2;
  constexpr int b_bytes = kRows * PC * 2;
  const int u_pair = g.nt * PC * 4;          // of an adapter's slice of B, and of two parts of u
  const int u_third = PC == 16 ? u_pair : kX + b_bytes;             // more tokens: where the third part is in a stage

  lin_setup<CG>(g, s, rank);
  // What the caller wrote may be read at once: a call's first launch lets the next start only after it has itself
  // waited for everything earlier.  What the launches before this one write (u, lists, counters) is read after the wait.
  if constexpr (!kOne) {
    if (LOW && !g.all) pdl_wait();
    pdl_release();
  }
  if constexpr (kOne) {
    if (high) {
      if (threadIdx.x < kFew) s.id[threadIdx.x] = adapter_of(g, threadIdx.x);
      if (threadIdx.x < kZeroBytes / 16) reinterpret_cast<uint4*>(zeros)[threadIdx.x] = make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncthreads();
      if (warp == 0) {
        // the first token of each adapter, and the lanes of tokens 0 to 31 and 32 to 63 that have it
        const int lo = s.id[lane], hi = s.id[32 + lane];
        const uint32_t lo_lo = __match_any_sync(0xffffffffu, lo), hi_hi = __match_any_sync(0xffffffffu, hi);
        uint32_t lo_hi = 0, hi_lo = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          if (__shfl_sync(0xffffffffu, hi, j) == lo) lo_hi |= 1u << j;
          if (__shfl_sync(0xffffffffu, lo, j) == hi) hi_lo |= 1u << j;
        }
        const bool first_lo = lo >= 0 && __ffs(lo_lo) - 1 == lane, first_hi = hi >= 0 && hi_lo == 0 && __ffs(hi_hi) - 1 == lane;
        const uint32_t all_lo = __ballot_sync(0xffffffffu, first_lo), all_hi = __ballot_sync(0xffffffffu, first_hi);
        const uint32_t before = (1u << lane) - 1u;
        if (first_lo) {
          const int i = __popc(all_lo & before);
          s.list[i] = lo;
          s.lanes[i] = make_uint2(lo_lo, lo_hi);
        }
        if (first_hi) {
          const int i = __popc(all_lo) + __popc(all_hi & before);
          s.list[i] = hi;
          s.lanes[i] = make_uint2(0, hi_hi);
        }
        const int n = __popc(all_lo) + __popc(all_hi);
        if (lane == 0) s.n_list = n;
      }
    }
  }
  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = s.tmem_slot;
  WaitCtl wc{g.status, &s.abort_flag, g.timeout_ns};
  Walk w0;
  w0.K = (g.d + 64 * kSub - 1) / (64 * kSub);
  const int high_subs = kOne ? s.n_list * RS : 0;
  w0.A = (high_subs + kHigh - 1) / kHigh;                           // few tokens: their adapters' slices count
  w0.unit = kBase;                                                  // as many bytes as a slice of W
  w0.init(LOW ? (g.all ? g.blocks : __ldcg(g.n_tiles)) : (int)((g.N + BN - 1) / BN) * g.groups, g.least, kOne ? kJoinFew : kJoinWide,
          kOne ? kBesideFew : kBesideWide, G, cta);
  // Tiles of one row tile follow each other: its rows of W are read by neighbours.
  auto place = [&](int tile, int& row0, int& block) {
    if (LOW) {
      const int2 p = g.all ? make_int2(0, tile) : __ldcg(g.tiles + tile);
      row0 = p.x * BN;
      block = p.y;
    } else if (kOne) {
      row0 = tile * BN;
      block = 0;
    } else {
      const int rt = tile / g.groups;
      row0 = rt * BN;
      block = (tile - rt * g.groups) * CG + rank;
    }
  };
  // Blocks of tokens: the segment that begins a tile also takes the slices of its block's adapters, behind its own: in
  // the last of its accumulators, which products of every lane have begun.  Their list is fetched when the segment
  // begins.
  auto listed = [&](int k0) { return !kOne && high && k0 == 0; };
  // Slices of W in a segment; the others are adapters'.
  auto base_of = [&](int k0, int len) { return kOne ? min(max(w0.K - k0, 0), len) : len; };
  int tile, c, k0, len, row0, block;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLowRegs));
    if (warp == 0) {
      if (lane == 0 && !g.stall) {
        // ---------------------------------------------------------- loads
        const uint64_t keep = policy_evict_last();
        const uint64_t pol_w = g.groups == 1 && !LOW ? policy_evict_first() : keep;
        uint32_t st = 0, ph = 0, issued = 0, last_par = 0, lst = 0, lph = 0, list_issued = 0, list_par = 0;
        bool fine = true, waited = false;
        for (Walk w = w0; fine && w.next(G, tile, c, k0, len);) {
          place(tile, row0, block);
          int ai = 0, rs = 0;                                       // next adapter of the list, which 32 of its rank
          if (kOne && k0 > w0.K) ai = (k0 - w0.K) * kHigh / RS, rs = (k0 - w0.K) * kHigh % RS;
          auto next_stage = [&](uint8_t*& sx) {
            if (!mbar_wait(&s.empty[st], ph ^ 1, wc)) return false;
            sx = smem + st * stage_bytes;
            return true;
          };
          auto sent = [&]() {
            issued |= 1u << st;
            last_par = (last_par & ~(1u << st)) | (ph << st);
            if (++st == (uint32_t)St) { st = 0; ph ^= 1; }
          };
          // a pair's loads all arrive at the leader's barrier
          auto expect = [&](int bytes) {
            if (rank == 0) mbar_arrive_expect_tx(&s.full[st], CG * bytes);
          };
          auto load = [&](void* dst, const CUtensorMap& m, int x, int y, uint64_t pol) {
            if constexpr (CG == 1) tma_load_2d(dst, &m, x, y, &s.full[st], pol);
            else tma_load_2d_pair(dst, &m, x, y, mapa_u32(smem_u32(&s.full[st]), 0), pol);
          };
          auto load_b = [&](void* dst, int x, int y, int a) {
            if constexpr (CG == 1) tma_load_3d(dst, &g.mapB, x, y, a, &s.full[st], pol_w);
            else tma_load_3d_pair(dst, &g.mapB, x, y, a, mapa_u32(smem_u32(&s.full[st]), 0), pol_w);
          };
          const int rows = row0 + rank * kRows;                     // this CTA's rows of W and B
          uint8_t* sx;
          // The slice before which the list is asked for: not before the stages went round, when the list before it is used up,
          // and at the end where that still has to wait for the launch before this one.
          const int fetch = !listed(k0) ? -1 : waited ? min(St, len - 1) : len - 1;
          for (int i = 0; i < len; ++i) {
            if (!kOne && i == fetch) {
              if (!waited) {
                pdl_wait();
                fence_proxy_async_global();                         // of u too
                waited = true;
              }
              if (!mbar_wait(&s.list_empty[lst], lph ^ 1, wc)) { fine = false; break; }
              mbar_arrive_expect_tx(&s.list_full[lst], sizeof(List));
              bulk_load_1d(lists + lst, static_cast<const List*>(g.lists) + block / CG, sizeof(List), &s.list_full[lst]);
              list_issued |= 1u << lst;
              list_par = (list_par & ~(1u << lst)) | (lph << lst);
            }
            if (!next_stage(sx)) { fine = false; break; }
            const int kb = k0 + i;
            if (!kOne || kb < w0.K) {
              expect(stage_bytes);
#pragma unroll
              for (int u = 0; u < kSub; ++u) {
                load(sx + u * sub_bytes, g.mapX, (kb * kSub + u) * 64, block * kBlock, keep);
                load(sx + u * sub_bytes + kX, g.mapW, (kb * kSub + u) * 64, rows, pol_w);
              }
            } else {
              if (!waited) {
                // u, once for all adapters: parts one and two side by side in rows of 128 bytes, then part three
                pdl_wait();
                fence_proxy_async_global();
                waited = true;
                mbar_arrive_expect_tx(&s.u_full, g.u_bytes);
                for (int j = 0; j < RS; ++j) {
                  uint8_t* su = u_base + j * (u_pair + u_pair / 2);
                  tma_load_2d(su, &g.mapU, j * 3 * PC, 0, &s.u_full, keep);
                  tma_load_2d(su + u_pair, &g.mapU3, j * 3 * PC + 2 * PC, 0, &s.u_full, keep);
                }
              }
              const int subs = min(kHigh, high_subs - (kb - w0.K) * kHigh);
              expect(subs * b_bytes);
              for (int u = 0; u < subs; ++u) {
                load_b(sx + u / (kRoom / 2) * sub_bytes + kX + u % (kRoom / 2) * b_bytes, rs * 32, rows, s.list[ai]);
                if (++rs == RS) ++ai, rs = 0;
              }
            }
            sent();
          }
          if (!fine) break;
          if (listed(k0)) {
            if (!mbar_wait(&s.list_full[lst], lph, wc)) { fine = false; break; }
            const List& list = lists[lst];
            for (int j = 0, n = list.n; fine && j < RS; ++j)
              for (int a = 0; a < n; a += kHigh) {
                if (!next_stage(sx)) { fine = false; break; }
                const int m = min(kHigh, n - a);
                expect(u_pair + m * b_bytes + (g.out_f32 ? u_pair / 2 : 0));
                load(sx, g.mapU, j * 3 * PC, block * kBlock, keep);
                if (g.out_f32) load(sx + u_third, g.mapU3, j * 3 * PC + 2 * PC, block * kBlock, keep);
                for (int u = 0; u < m; ++u) load_b(sx + kX + u * b_bytes, j * 32, rows, list.adapter[a + u]);
                sent();
              }
            if (fine) mbar_arrive(&s.list_empty[lst]);
            if (++lst == kLists) lst = 0, lph ^= 1;
          }
        }
        if (!fine) {
          if (rank == 0) {
            few_drain(s.full, St, issued, last_par);
          } else {                                                  // the barriers are the leader's: a fixed time
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 5000000ull) __nanosleep(1000);
          }
          if (kOne && waited) few_drain(&s.u_full, 1, 1, 0);
          if (!kOne) few_drain(s.list_full, 2, list_issued, list_par);
        }
      }
    } else if (warp == 2) {
      if (lane == 0 && rank == 0) {
        // ---------------------------------------------------------- products
        constexpr uint32_t id = idesc_bf16(CG * 128, BN, 0, 0);
        uint32_t st = 0, ph = 0, acc = 0, aph = 0, lst = 0, lph = 0;
        bool fine = true, have_u = false;
        const uint32_t kind_u = sdesc_kind(4 * PC), kind_b = sdesc_kind(2 * PC);
        for (Walk w = w0; fine && w.next(G, tile, c, k0, len);) {
          place(tile, row0, block);
          // slices of W, an accumulator every g.chunk of them; the adapters' go into the last (or one of their own)
          const int base = base_of(k0, len), more = kOne ? len - base : 0;
          const int high0 = max(k0 - w0.K, 0);                      // few tokens: first of the adapters' slices here
          int ai = 0, rs = 0;
          if (kOne) ai = high0 * kHigh / RS, rs = high0 * kHigh % RS;
          auto stage = [&](uint32_t& sx) {
            if (!mbar_wait(&s.full[st], ph, wc)) return false;
            tc_fence_after();
            sx = smem_u32(smem + st * stage_bytes);
            return true;
          };
          auto used = [&]() {
            pair_commit<CG>(&s.empty[st]);
            if (++st == (uint32_t)St) { st = 0; ph ^= 1; }
          };
          // 32 of the rank: 16 columns of B_a meet the parts of u, in the lanes of the adapter's tokens
          auto adapter = [&](uint32_t d0, uint32_t sb, uint32_t su, uint32_t su3, int j, const uint4 (&on)[CG]) {
            const uint64_t du = sdesc(su, kind_u), du3 = sdesc(su3, kind_b), db = sdesc(sb, kind_b);
            const int second = PC / 8;                              // the second part, in 16 bytes
            const int steps = g.r - 32 * j > 16 ? 2 : 1;
            for (int kk = 0; kk < steps; ++kk) {
              umma_lanes<CG>(d0, du + 2 * kk, db + 2 * kk, id, on);
              umma_lanes<CG>(d0, du + second + 2 * kk, db + 2 * kk, id, on);
              if (g.out_f32) umma_lanes<CG>(d0, du3 + 2 * kk, db + 2 * kk, id, on);
            }
          };
          for (int done = 0; (done == 0 || done < base) && fine; done += g.chunk) {
            const int n = min(g.chunk, base - done);
            const bool last = done + n == base;
            if (!mbar_wait(&s.tempty[acc], aph ^ 1, wc)) { fine = false; break; }
            tc_fence_after();
            const uint32_t d0 = tmem_base + acc * BN;
            uint32_t sx;
            if (kOne && base == 0) umma_clear(d0, smem_u32(zeros));
            for (int i = 0; i < n; ++i) {
              if (!stage(sx)) { fine = false; break; }
#pragma unroll
              for (int u = 0; u < kSub; ++u) {
                const uint64_t dx = sdesc_sw128(sx + u * sub_bytes, 16, 1024), dw = sdesc_sw128(sx + u * sub_bytes + kX, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)                      // 32 bytes further each time
                  pair_mma<CG>(d0, dx + 2 * kk, dw + 2 * kk, id, (i | u | kk) != 0 ? 1u : 0u);
              }
              used();
            }
            if (!fine) break;
            if (kOne && last && more > 0) {
              if (!have_u) {
                if (!mbar_wait(&s.u_full, 0, wc)) { fine = false; break; }
                tc_fence_after();
                have_u = true;
              }
              for (int i = 0; i < more; ++i) {
                if (!stage(sx)) { fine = false; break; }
                const int subs = min(kHigh, high_subs - (high0 + i) * kHigh);
                for (int u = 0; u < subs; ++u) {
                  const uint4 on[CG] = {make_uint4(s.lanes[ai].x, s.lanes[ai].y, 0, 0)};
                  const uint32_t su = smem_u32(u_base) + rs * (u_pair + u_pair / 2);
                  adapter(d0, sx + u / (kRoom / 2) * sub_bytes + kX + u % (kRoom / 2) * b_bytes, su, su + u_pair, rs, on);
                  if (++rs == RS) ++ai, rs = 0;
                }
                used();
              }
            }
            if (last && listed(k0)) {
              if (!mbar_wait(&s.list_full[lst], lph, wc)) { fine = false; break; }
              const List& list = lists[lst];
              for (int j = 0, m = list.n; fine && j < RS; ++j)
                for (int a = 0; a < m; a += kHigh) {
                  if (!stage(sx)) { fine = false; break; }
                  for (int u = 0; u < min(kHigh, m - a); ++u) {
                    uint4 on[CG];
#pragma unroll
                    for (int x = 0; x < CG; ++x) on[x] = list.lanes[a + u][x];
                    adapter(d0, sx + kX + u * b_bytes, sx, sx + u_third, j, on);
                  }
                  used();
                }
              if (fine) mbar_arrive(&s.list_empty[lst]);
              if (++lst == kLists) lst = 0, lph ^= 1;
            }
            if (!fine) break;
            pair_commit<CG>(&s.tfull[acc]);
            if (++acc == kAccs) acc = 0, aph ^= 1;
          }
        }
        if (!fine) lin_drain<CG>(s);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kHighRegs));
    // ------------------------------------------------------------ epilogue: lane = token, register = row of W
    constexpr int kHalf = BN / 2;
    const int q = warp & 3, h = (warp - 4) >> 2;                    // TMEM lane quadrant; half of the columns
    const int tid = threadIdx.x - 128;
    float(*turned)[33] = s.turn[warp - 4];
    const bool live = kOne ? 32 * q < g.T : true;                   // the quadrant has tokens
    // rows of the output whose 16 columns begin and end on 16 bytes are written by their lanes
    const bool vectors = (g.N * (g.out_f32 ? 4 : 2) & 15) == 0 && (reinterpret_cast<uintptr_t>(g.out) & 15) == 0;
    uint32_t acc = 0, aph = 0, turn = 0;
    int mine_id = -1;                                               // LOW: the adapter of this lane's token
    pdl_wait();
    // 16 columns of this warp's 32 tokens, from column `col` of a tile on
    auto finish = [&](int row0_, int block_, int col, const float (&v)[16]) {
      const int64_t n0 = (int64_t)row0_ + col;
      const int t0 = block_ * kBlock + 32 * q;
      if constexpr (LOW) {
#pragma unroll
        for (int e = 0; e < 16; e += 8) {                           // eight rows of the stacked A have one adapter
          const int a = (int)((n0 + e) / g.r), j = (int)(n0 + e - (int64_t)a * g.r);
          if (mine_id >= 0 && a == mine_id) {
            const float sc = g.scale ? __ldg(g.scale + a) : 1.0f;
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = sc * v[e + i];
            uint4* p = reinterpret_cast<uint4*>(u_at(g, t0 + lane, j));
#pragma unroll
            for (int o = 0; o < 3; ++o) {
              float b[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) b[i] = bf16_part(x[i]);
              p[g.pc / 8 * o] = make_uint4(pack_bf16(b[0], b[1]), pack_bf16(b[2], b[3]), pack_bf16(b[4], b[5]), pack_bf16(b[6], b[7]));
              if (g.r % 16 && j == g.r - 8) p[g.pc / 8 * o + 1] = make_uint4(0, 0, 0, 0);
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i] = bf16_rest(x[i], b[i]);
            }
          }
        }
      } else if (vectors) {
        if (t0 + lane < g.T) {
          if (g.out_f32) {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(g.out) + (size_t)(t0 + lane) * g.N + n0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (n0 + 4 * i < g.N) o[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          } else {
            uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(g.out) + (size_t)(t0 + lane) * g.N + n0);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (n0 + 8 * i < g.N)
                o[i] = make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                                  pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
          }
        }
      } else {
        // through shared memory, so that lanes write neighbouring columns of a row, whatever its alignment (bf16 columns
        // two at a time where they share a word: 777 x 1000 x 5001 31 us against 26)
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i) turned[i][lane] = v[i];
        __syncwarp();
        const int64_t n = n0 + lane % 16;
        const int rows = min(32, g.T - t0);
        if (n < g.N) {
          const size_t at = (size_t)(t0 + lane / 16) * g.N + n;
          if (g.out_f32) {
            float* o = static_cast<float*>(g.out) + at;
#pragma unroll 8
            for (int r = lane / 16; r < rows; r += 2, o += 2 * g.N) *o = turned[lane % 16][r];
          } else {
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(g.out) + at;
#pragma unroll 8
            for (int r = lane / 16; r < rows; r += 2, o += 2 * g.N) *o = __float2bfloat16_rn(turned[lane % 16][r]);
          }
        }
      }
    };
    // A part of a cut tile: [column / 4][token] of four columns.  A share has two cut tiles at most: one that began before
    // it, and one that it leaves unfinished.
    const int part_rows = kOne ? g.nt : kBlock;
    const size_t slot = (size_t)BN / 4 * part_rows;
    const bool stored = 32 * q + lane < part_rows;
    // The cut tiles' sums, once this CTA's own parts are on their way: groups of 32 columns, in turn by a tile's CTAs.
    // While weights stream, a load takes 2 us and more, so both tiles are waited for at once and two groups are
    // fetched at a time.
    auto join = [&]() {
      int jt[2] = {0, 0}, js[2] = {0, 0}, jf[2] = {0, 0}, jp[2] = {1, 1};   // tile, index, first CTA, parts
      int tiles_cut = 0;
      for (Walk w = w0; w.at < w.end;) {
        w.next(G, tile, c, k0, len);
        if (len == w0.K + w0.A) continue;
        const int s0 = c * (w0.K + w0.A), first = w0.owner(s0), parts = w0.owner(s0 + w0.K + w0.A - 1) - first + 1;
        // at most two: static indexing keeps them in registers
        if (tiles_cut == 0) jt[0] = tile, js[0] = c, jf[0] = first, jp[0] = parts;
        else jt[1] = tile, js[1] = c, jf[1] = first, jp[1] = parts;
        ++tiles_cut;
      }
      if (tiles_cut == 0) return;
      // One word has the parts that came and the shares that were left: either this CTA finds its tile complete, or
      // the CTA that completes it finds this one's share.
      if (lane == 0 && warp - 4 < 2) {
        const bool second = warp - 4 == 1;
        int m = 0;
        if (!second || tiles_cut == 2) {
          const int share = cta - (second ? jf[1] : jf[0]), parts = second ? jp[1] : jp[0];
          int* word = g.cnt + (second ? js[1] : js[0]) * CG + rank;
          if (share < min(parts, BN / 32)) {
            const uint64_t t0 = globaltimer_ns();
            bool there;
            while (!(there = (ld_acquire_gpu(word) & 0xffff) >= parts) && globaltimer_ns() - t0 < g.patience) __nanosleep(20);
            if (!there) there = (atom_or_acq_rel_gpu(word, 1 << (16 + share)) & 0xffff) >= parts;
            if (there) m = 1 << share;
          }
        }
        s.todo[second ? 1 : 0] = m;
      }
      named_bar(1, 256);
      __threadfence();
      // the groups of the shares: bits 0.. of the first tile, kShares.. of the second
      uint32_t todo = 0;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int m = x < tiles_cut ? s.todo[x] | s.left[x] : 0;
        for (int i = 0, share = 0; i < BN / 32; ++i) {
          todo |= ((uint32_t)(m >> share) & 1u) << (x * kShares + i);
          if (++share == jp[x]) share = 0;
        }
      }
      if (!live) return;
      while (todo) {
        float v[2][16];
        const float4* p[2];
        int r0[2], bl[2], col[2], parts[2], most = 0;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = todo ? __ffs(todo) - 1 : 0;
          const bool second = i >= kShares;
          parts[e] = todo ? (second ? jp[1] : jp[0]) : 0;
          todo &= todo - 1;
          place(second ? jt[1] : jt[0], r0[e], bl[e]);
          col[e] = (i - (second ? kShares : 0)) * 32 + 16 * h;
          p[e] = g.part + (size_t)(2 * (CG * (second ? jf[1] : jf[0]) + rank) + 1) * slot + (size_t)col[e] / 4 * part_rows + 32 * q + lane;
          most = max(most, parts[e]);
#pragma unroll
          for (int k = 0; k < 16; ++k) v[e][k] = 0.0f;
        }
#pragma unroll 2
        for (int o = 0; o < most; ++o) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (o >= parts[e] || !stored) continue;
            // the first CTA left the tile unfinished: its second slot; the others began inside it: their first
            const float4* x = o == 0 ? p[e] : p[e] + (size_t)(2 * CG * o - 1) * slot;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float4 y = __ldcg(x + (size_t)k * part_rows);
              v[e][4 * k] += y.x;
              v[e][4 * k + 1] += y.y;
              v[e][4 * k + 2] += y.z;
              v[e][4 * k + 3] += y.w;
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (parts[e] == 0) continue;
          if (LOW) mine_id = adapter_of(g, bl[e] * kBlock + 32 * q + lane);
          finish(r0[e], bl[e], col[e], v[e]);
        }
      }
    };
    bool joined = w0.at >= w0.end, fine = true;
    int cuts = 0;                                                   // cut tiles so far
    for (Walk w = w0; fine && w.next(G, tile, c, k0, len);) {
      // The join goes before the first whole tile, whose products go on meanwhile; after it where such a tile takes several
      // accumulators, which would be kept waiting (tiles of 128 rows; those of 256 take longer than the join).
      if (c < 0 && !joined && (!kOne || g.chunk >= w0.K)) {
        const int keep_tile = tile, keep_len = len;
        join();
        joined = true;
        tile = keep_tile, len = keep_len, c = -1, k0 = 0;
      }
      place(tile, row0, block);
      float z[kHalf];
      const int base = base_of(k0, len);
      for (int done = 0; done == 0 || done < base; done += g.chunk) {
        if (!few_epilogue_wait(&s.tfull[acc], aph, wc, tid, s.ready, turn)) { fine = false; break; }
        tc_fence_after();
        const uint32_t tb = tmem_base + ((uint32_t)(32 * q) << 16) + acc * BN + kHalf * h;
        if (live) {
#pragma unroll
          for (int i = 0; i < kHalf; i += 16) {
            uint32_t v[16];
            tmem_ld16(tb + i, v);
            tmem_ld_wait();
            if (done == 0) {
#pragma unroll
              for (int e = 0; e < 16; ++e) z[i + e] = __uint_as_float(v[e]);
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) z[i + e] += __uint_as_float(v[e]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 1) mbar_arrive(&s.tempty[acc]);
          else mbar_arrive_cluster(mapa_u32(smem_u32(&s.tempty[acc]), 0));
        }
        if (++acc == kAccs) acc = 0, aph ^= 1;
      }
      if (!fine) break;
      if (LOW) mine_id = adapter_of(g, block * kBlock + 32 * q + lane);
      const bool whole = len == w0.K + w0.A;
      float4* mine = g.part + (size_t)(2 * blockIdx.x + (k0 > 0 ? 0 : 1)) * slot + 32 * q + lane;
      if (live) {
#pragma unroll
        for (int i = 0; i < kHalf; i += 16) {
          if (whole) {
            float v[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = z[i + e];
            finish(row0, block, kHalf * h + i, v);
          } else if (stored) {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              __stcg(mine + (size_t)(kHalf * h + i + e) / 4 * part_rows, make_float4(z[i + e], z[i + e + 1], z[i + e + 2], z[i + e + 3]));
          }
        }
      }
      if (!whole) {
        __threadfence();
        named_bar(1, 256);
        if (tid == 0) {
          const int s0 = c * (w0.K + w0.A), parts = w0.owner(s0 + w0.K + w0.A - 1) - w0.owner(s0) + 1;
          const int old = atom_add_acq_rel_gpu(g.cnt + c * CG + rank, 1);
          s.left[cuts] = (old & 0xffff) == parts - 1 ? old >> 16 : 0;   // complete: with what others left
        }
        ++cuts;
      } else if (c < 0 && !joined) {
        join();
        joined = true;
      }
    }
    if (fine && !joined) join();
  }

  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();                        // no arrival or copy may target a CTA that has left
  if (warp == 2) {
    tc_fence_after();
    pair_tmem_free<CG>(tmem_base);
  }
  // every thread has waited when the grid is done, so that whatever follows finds the launch before this one complete
  pdl_wait();
}

// ------------------------------------------------------------------ the launch before the product
struct LowArgs {
  const __nv_bfloat16 *X, *A;        // [T, d], [n, r, d]
  int* cnt;                          // zeroed: n_cnt counters
  int2* tiles;                       // more tokens than kFew: the low side's tiles
  int* n_tiles;
  void* lists;                       // and each block's adapters, or each two blocks'
  int n_cnt, row_tiles;              // row tiles of the stacked A (0: no adapters)
  int list_ctas;                     // low_dot_kernel: CTAs that make the lists
};

// The adapters of a block of tokens, or two (a warp's), in increasing order, from bit sets of 1024.
template <int CG>
struct BlockIds {
  static constexpr int kIds = CG * kBlock / 32;
  int id[kIds];
  bool lead[kIds];                                                  // the first of a run
  __device__ __forceinline__ BlockIds(const LinArgs& g, int b, int lane) {
#pragma unroll
    for (int i = 0; i < kIds; ++i) {
      id[i] = adapter_of(g, b * CG * kBlock + 32 * i + lane);
      const int left = __shfl_up_sync(0xffffffffu, id[i], 1);
      lead[i] = id[i] >= 0 && (lane == 0 || left != id[i]);
    }
  }
  // The members of [x0, x0 + 1024) that mark() sets, in order: put(position, member); returns how many.
  template <class Mark, class Put>
  __device__ __forceinline__ int members(uint32_t* set, int lane, int x0, Mark&& mark, Put&& put) const {
    set[lane] = 0;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kIds; ++i)
      if (lead[i]) mark(id[i]);
    __syncwarp();
    uint32_t bits = set[lane];
    const int n = __popc(bits);
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    for (int at = x - n; bits; bits &= bits - 1) put(at++, x0 + 32 * lane + __ffs(bits) - 1);
    __syncwarp();
    return __shfl_sync(0xffffffffu, x, 31);
  }
  static __device__ __forceinline__ void add(uint32_t* set, int x0, int v) {
    if (v >= x0 && v < x0 + 1024) atomicOr(&set[(v - x0) >> 5], 1u << (v & 31));
  }
  // List b, with the lanes that have each adapter.
  __device__ __forceinline__ void write(const LinArgs& g, const LowArgs& l, uint32_t* set, int* found, int b, int lane) const {
    BlockList<CG>& list = static_cast<BlockList<CG>*>(l.lists)[b];
    int n = 0;
    for (int x0 = 0; x0 < g.n; x0 += 1024)
      n += members(set, lane, x0, [&](int a) { add(set, x0, a); }, [&](int at, int a) { found[n + at] = a; });
    for (int i = 0; i < n; ++i) {
      const int a = found[i];
      uint32_t on[kIds];
#pragma unroll
      for (int k = 0; k < kIds; ++k) on[k] = __ballot_sync(0xffffffffu, id[k] == a);
      if (lane == 0) {
        list.adapter[i] = a;
#pragma unroll
        for (int k = 0; k < CG; ++k) list.lanes[i][k] = make_uint4(on[4 * k], on[4 * k + 1], on[4 * k + 2], on[4 * k + 3]);
      }
    }
    if (lane == 0) list.n = n;
  }
};

__device__ __forceinline__ void write_list(const LinArgs& g, const LowArgs& l, uint32_t* set, int* found, int b, int lane) {
  if (g.pairs) BlockIds<2>(g, b, lane).write(g, l, set, found, b, lane);
  else BlockIds<1>(g, b, lane).write(g, l, set, found, b, lane);
}

// Zeroes the counters; u with a warp per token and row of A (few tokens, and more where that is less work than
// products of whole tiles); the lists of blocks of tokens in the first CTAs, where there are such blocks.
constexpr int kDotWarps = 8;
__global__ void __launch_bounds__(kDotWarps * 32) low_dot_kernel(const __grid_constant__ LinArgs g, const __grid_constant__ LowArgs l) {
  __shared__ uint32_t set[kDotWarps][32];
  __shared__ int found[kDotWarps][2 * kBlock];
  pdl_wait();
  pdl_release();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < l.n_cnt; i += kDotWarps * 32) l.cnt[i] = 0;
  if (!g.high) return;
  if ((int)blockIdx.x < l.list_ctas) {
    const int b = blockIdx.x * kDotWarps + warp;
    if (blockIdx.y == 0 && b < g.groups) write_list(g, l, set[warp], found[warp], b, lane);
    return;
  }
  const int t = blockIdx.x - l.list_ctas, j = blockIdx.y * kDotWarps + warp;
  const int a = adapter_of(g, t);
  if (a < 0) return;
  const uint4* x = reinterpret_cast<const uint4*>(l.X + (size_t)t * g.d);
  const uint4* w = reinterpret_cast<const uint4*>(l.A + ((size_t)a * g.r + j) * g.d);
  float sum[2] = {0.0f, 0.0f};
#pragma unroll 8
  for (int v = lane; v < g.d / 8; v += 32) {
    const uint4 p = __ldg(x + v), o = __ldg(w + v);
    const uint32_t pp[4] = {p.x, p.y, p.z, p.w}, oo[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sum[0] = fmaf(__uint_as_float(pp[i] << 16), __uint_as_float(oo[i] << 16), sum[0]);
      sum[1] = fmaf(__uint_as_float(pp[i] & 0xffff0000u), __uint_as_float(oo[i] & 0xffff0000u), sum[1]);
    }
  }
  float s = sum[0] + sum[1];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) put_u(g, t, j, (g.scale ? __ldg(g.scale + a) : 1.0f) * s);
}

// More tokens: the 128-row tiles of the stacked A that each block of tokens has adapters in (the low side's
// tiles, in increasing order), and each block's adapters with their tokens' lanes.  A warp per block.
constexpr int kListWarps = 32;
__global__ void __launch_bounds__(kListWarps * 32) low_list_kernel(const __grid_constant__ LinArgs g, const __grid_constant__ LowArgs l) {
  __shared__ uint32_t set[kListWarps][32];
  __shared__ int count[kListWarps];
  __shared__ int found[kListWarps][2 * kBlock];
  pdl_wait();
  pdl_release();
  for (int i = threadIdx.x; i < l.n_cnt; i += kListWarps * 32) l.cnt[i] = 0;
  if (!g.high) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int base = 0;
  for (int b0 = 0; b0 < g.blocks; b0 += kListWarps) {
    const int b = b0 + warp;
    if (b < g.groups) write_list(g, l, set[warp], found[warp], b, lane);
    const BlockIds<1> ids(g, b, lane);
    // the tiles, in the order of the blocks: first how many, then where
    auto tiles_of = [&](int x0, auto&& put) {
      return ids.members(set[warp], lane, x0, [&](int a) {
        const int last_tile = (int)(((int64_t)a * g.r + g.r - 1) / kRowsLow);
        for (int x = (int)((int64_t)a * g.r / kRowsLow); x <= last_tile; ++x) BlockIds<1>::add(set[warp], x0, x);
      }, put);
    };
    int n = 0;
    if (b < g.blocks)
      for (int x0 = 0; x0 < l.row_tiles; x0 += 1024) n += tiles_of(x0, [](int, int) {});
    if (lane == 0) count[warp] = n;
    __syncthreads();
    int at = base;
    for (int w = 0; w < kListWarps; ++w) {
      if (w < warp) at += count[w];
      base += count[w];
    }
    if (b < g.blocks)
      for (int x0 = 0; x0 < l.row_tiles; x0 += 1024)
        at += tiles_of(x0, [&](int i, int tile) { l.tiles[at + i] = make_int2(tile, b); });
    __syncthreads();
  }
  if (threadIdx.x == 0) *l.n_tiles = base;
}

// ------------------------------------------------------------------ host side
moe_status_t bad(const std::string& what, moe_status_t s = MOE_ERR_INVALID_ARG) {
  set_error_detail(("moe_linear: " + what).c_str());
  return s;
}
moe_status_t cuda_bad(const char* what, cudaError_t e) {
  return bad(std::string(what) + ": " + cudaGetErrorString(e), MOE_ERR_CUDA);
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}
CUtensorMapSwizzle swizzle_of(int box_cols) {
  return box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : box_cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
}
// bf16 [rows, cols]: boxes of 64, 32 or 16 columns, swizzled over their width; reads past the edges give zeros
bool map_rows(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int box, int box_cols = 64) {
  auto enc = encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)cols * 2};
  cuuint32_t boxes[2] = {(cuuint32_t)box_cols, (cuuint32_t)box}, es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, boxes, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle_of(box_cols), CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [n, N, r]: boxes of `cols` columns and `rows` rows of one adapter
bool map_adapters(CUtensorMap* m, const void* base, int64_t r, int64_t N, int64_t n, int rows, int cols) {
  auto enc = encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)r, (cuuint64_t)N, (cuuint64_t)n};
  cuuint64_t strides[2] = {(cuuint64_t)r * 2, (cuuint64_t)(N * r) * 2};
  cuuint32_t boxes[3] = {(cuuint32_t)cols, (cuuint32_t)rows, 1}, es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, boxes, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle_of(cols), CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kTail = sizeof(LinSmem) + 1024;
constexpr int kMaxSmem = 232448;

template <int BN, int PC, bool LOW, int CG>
cudaError_t prepare_one() {
  cudaFuncAttributes a;    // a launch with fewer registers than the warps' shares would wait for them without end
  const cudaError_t e = cudaFuncGetAttributes(&a, lin_kernel<BN, PC, LOW, CG>);
  if (e != cudaSuccess) return e;
  if (a.numRegs < kLaunch) return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(lin_kernel<BN, PC, LOW, CG>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
}

moe_status_t facts(int* sms) {
  constexpr int kMax = 64;
  static int known[kMax];
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaSetDevice(dev);      // binds the context: the tensor-map encoder is a driver call
  if (e != cudaSuccess) return cuda_bad("no usable current device", e);
  if (dev < 0 || dev >= kMax) return bad("device ordinal out of range", MOE_ERR_UNSUPPORTED);
  std::lock_guard<std::mutex> lock(mu);
  if (!known[dev]) {
    int major = 0, minor = 0, n = 0;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (major != 10 || minor != 3) return bad("this library is built for sm_103a (GB300) only", MOE_ERR_UNSUPPORTED);
    if ((e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
        (e = prepare_one<kRowsFew, 16, false, 1>()) != cudaSuccess || (e = prepare_one<kRowsFew, 32, false, 1>()) != cudaSuccess ||
        (e = prepare_one<kRowsWide, 16, false, 1>()) != cudaSuccess || (e = prepare_one<kRowsWide, 32, false, 1>()) != cudaSuccess ||
        (e = prepare_one<kRowsWide, 16, false, 2>()) != cudaSuccess || (e = prepare_one<kRowsWide, 32, false, 2>()) != cudaSuccess ||
        (e = prepare_one<kRowsLow, 16, true, 1>()) != cudaSuccess)
      return cuda_bad("kernel attributes", e);
    known[dev] = n;
  }
  *sms = known[dev];
  return MOE_OK;
}

int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

struct Layout {
  int nt, blocks, groups, row_tiles;
  bool adapters, wide, pairs;
  size_t part, cnt, u, tiles, n_tiles, lists, total;
};

// Pairs of CTAs read half as much of W into each SM, and every second block of tokens reads W once less.  They pay for
// bf16 results (fp32: an accumulator changes every 512 products, and a pair waits for both epilogues: 4096 x 2048 x 7168
// 121 us against 114; bf16: 73 against 81), where waves of tiles are filled (4096 x 7168 x 2048: 79 against 85; 1024 tokens: 37
// against 36) and long, and for two blocks where W is large (200 x 7168 x 8192: 39 against 53; 256 x 2048 x 7168: 20 against 19).  A
// pair's list holds both blocks' adapters: with many, each on few tokens, it is twice as long (1000 x 4096 x 7168, 300
// adapters in turn: 186 against 128; 64 adapters: alike).
bool on_pairs(const moe_linear_config_t& c, int blocks, int sms) {
  if (c.out_f32 || c.n > 64) return false;
  if (blocks == 2) return (int64_t)c.N * c.d >= 1 << 25;
  return blocks >= 8 && c.d >= 1024 && (c.N + kRowsWide - 1) / kRowsWide * blocks >= 3 * sms / 2;
}

Layout layout(const moe_linear_config_t& c, int sms) {
  Layout L{};
  L.adapters = c.n > 0;
  L.wide = c.T > kFew;
  L.nt = L.wide ? kBlock : (int)up(c.T, 16);
  L.blocks = (int)((c.T + L.nt - 1) / L.nt);
  L.pairs = L.wide && on_pairs(c, L.blocks, sms);
  L.groups = L.pairs ? (L.blocks + 1) / 2 : L.blocks;
  L.row_tiles = L.adapters ? (int)(((int64_t)c.n * c.r + kRowsLow - 1) / kRowsLow) : 0;
  size_t o = 0;
  auto take = [&o](size_t n) {
    const size_t at = o;
    o += (n + 255) & ~size_t(255);
    return at;
  };
  L.part = take((size_t)2 * sms * L.nt * (L.wide ? kRowsWide : kRowsFew) * 4);
  L.cnt = take((size_t)2 * sms * 4);                           // fewer tiles than SMs are cut, of either side
  L.u = take(L.adapters ? (size_t)c.T * ((c.r + 31) / 32) * 192 : 0);
  const bool lists = L.adapters && L.wide;
  // a block of tokens has at most as many adapters as tokens, each in one to three tiles
  L.tiles = take(lists ? (size_t)L.blocks * std::min(L.row_tiles, 3 * kBlock) * 8 : 0);
  L.n_tiles = take(4);
  L.lists = take(lists ? std::max(L.blocks * sizeof(BlockList<1>), (L.blocks + 1) / 2 * sizeof(BlockList<2>)) : 0);
  L.total = o;
  return L;
}

moe_status_t check(const moe_linear_config_t* c) {
  if (!c) return bad("null config");
  if (c->T < 0 || c->T > (1 << 20)) return bad("T must be in [0, 2^20]");
  if (c->N < 1 || c->N > (1 << 24)) return bad("N must be in [1, 2^24]");
  if (c->d < 8 || c->d > (1 << 16) || c->d % 8) return bad("d must be a multiple of 8 in [8, 2^16]", MOE_ERR_UNSUPPORTED);
  if (c->n < 0 || c->n > (1 << 16)) return bad("n must be in [0, 2^16]");
  if (c->n > 0 && (c->r < 8 || c->r > kMaxRank || c->r % 8))
    return bad("r must be a multiple of 8 in [8, 256]", MOE_ERR_UNSUPPORTED);
  if (c->wait_timeout_ns < 0) return bad("wait_timeout_ns must not be negative");
  return MOE_OK;
}

bool at16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <int BN, int PC, bool LOW, int CG>
cudaError_t launch_one(LinArgs& g, int sms, cudaStream_t st) {
  constexpr bool one = BN == kRowsFew && !LOW;
  const int stage = (one ? 2 : 1) * (g.nt + BN / CG) * 128;
  g.u_bytes = one && g.high ? (g.r + 31) / 32 * g.nt * 6 * g.pc : 0;
  const int rest = kTail + (one ? kZeroBytes + g.u_bytes : 2 / CG * (int)sizeof(BlockList<CG>));
  g.stages = std::min(kMaxStages, (kMaxSmem - rest) / stage);
  return launch_pdl(lin_kernel<BN, PC, LOW, CG>, dim3(sms / CG * CG), dim3(kFewThreads), (size_t)g.stages * stage + rest, st, CG, g);
}

template <int BN, int CG>
cudaError_t launch_high(LinArgs& g, int sms, cudaStream_t st) {
  return g.pc == 16 ? launch_one<BN, 16, false, CG>(g, sms, st) : launch_one<BN, 32, false, CG>(g, sms, st);
}
cudaError_t launch_wide(LinArgs& g, int sms, cudaStream_t st) {
  return g.pairs ? launch_high<kRowsWide, 2>(g, sms, st) : launch_high<kRowsWide, 1>(g, sms, st);
}

}  // namespace

extern "C" moe_status_t moe_linear_workspace_bytes(const moe_linear_config_t* cfg, size_t* bytes) {
  if (!bytes) return bad("null argument");
  moe_status_t s = check(cfg);
  int sms = 0;
  if (s == MOE_OK) s = facts(&sms);
  if (s != MOE_OK) return s;
  *bytes = cfg->T ? layout(*cfg, sms).total : 0;
  return MOE_OK;
}

extern "C" moe_status_t moe_linear(const moe_linear_config_t* cfg, const void* X, const void* W, const void* A,
                                   const void* B, const void* ids, const float* scale, void* out, void* workspace,
                                   size_t workspace_bytes, int32_t* status, moe_stream_t stream) {
  moe_status_t s = check(cfg);
  if (s != MOE_OK) return s;
  const moe_linear_config_t& c = *cfg;
  if (c.T == 0) return MOE_OK;
  if (!at16(X) || !at16(W)) return bad("X and W are required, 16-byte aligned");
  if (!out || reinterpret_cast<uintptr_t>(out) & (c.out_f32 ? 3 : 1)) return bad("out is required, aligned to its type");
  if (c.n > 0) {
    if (!at16(A) || !at16(B)) return bad("A and B are required, 16-byte aligned");
    if (!ids || reinterpret_cast<uintptr_t>(ids) & (c.ids_int64 ? 7 : 3)) return bad("ids are required, aligned to their type");
    if (reinterpret_cast<uintptr_t>(scale) & 3) return bad("scale: misaligned");
  }
  if (reinterpret_cast<uintptr_t>(status) & 3) return bad("status: misaligned");
  const uintptr_t o0 = reinterpret_cast<uintptr_t>(out), o1 = o0 + (size_t)c.T * c.N * (c.out_f32 ? 4 : 2);
  auto meets = [&](const void* p, size_t bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(p);
    return p && x < o1 && o0 < x + bytes;
  };
  const size_t na = c.n > 0 ? (size_t)c.n * c.r * 2 : 0;
  if (meets(X, (size_t)c.T * c.d * 2) || meets(W, (size_t)c.N * c.d * 2) || (na && (meets(A, na * c.d) || meets(B, na * c.N) ||
      meets(ids, (size_t)c.T * (c.ids_int64 ? 8 : 4)) || meets(scale, (size_t)c.n * 4))))
    return bad("out overlaps an input");
  int sms = 0;
  if ((s = facts(&sms)) != MOE_OK) return s;
  const Layout L = layout(c, sms);
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) & 255) return bad("workspace is required, 256-byte aligned");
  if (workspace_bytes < L.total) return bad("workspace too small");
  char* w = static_cast<char*>(workspace);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);

  LinArgs g{};
  g.ids = ids;
  g.scale = scale;
  g.u = reinterpret_cast<uint4*>(w + L.u);
  g.out = out;
  g.part = reinterpret_cast<float4*>(w + L.part);
  g.cnt = reinterpret_cast<int*>(w + L.cnt);
  g.tiles = reinterpret_cast<const int2*>(w + L.tiles);
  g.n_tiles = reinterpret_cast<const int*>(w + L.n_tiles);
  g.lists = w + L.lists;
  g.pairs = L.pairs;
  g.groups = L.groups;
  g.status = status;
  g.patience = (c.debug_flags & MOE_DEBUG_NO_PATIENCE) ? 0 : kPatience;
  g.timeout_ns = c.wait_timeout_ns > 0 ? (uint64_t)c.wait_timeout_ns : 2000000000ull;
  g.N = c.N;
  g.T = (int)c.T;
  g.d = c.d;
  g.n = c.n;
  g.r = c.n > 0 ? c.r : 8;
  g.nt = L.nt;
  g.pc = g.r <= 16 ? 16 : 32;
  g.blocks = L.blocks;
  g.least = L.nt <= 16 ? 2 : L.wide ? 8 : 4;
  g.out_f32 = c.out_f32;
  g.ids64 = c.ids_int64;
  g.high = L.adapters;
  g.stall = (c.debug_flags & MOE_DEBUG_STALL_TEST) != 0;
  const int chunk = L.wide ? 8 : 4, whole = 1 << 20;     // 512 products
  LowArgs l{};
  l.X = static_cast<const __nv_bfloat16*>(X);
  l.A = static_cast<const __nv_bfloat16*>(A);
  l.cnt = g.cnt;
  l.tiles = reinterpret_cast<int2*>(w + L.tiles);
  l.n_tiles = reinterpret_cast<int*>(w + L.n_tiles);
  l.lists = w + L.lists;
  l.n_cnt = 2 * sms;
  l.row_tiles = L.row_tiles;
  const int rows = L.wide ? kRowsWide / (L.pairs ? 2 : 1) : kRowsFew, RS = (g.r + 31) / 32;
  if (!map_rows(&g.mapX, X, c.d, c.T, L.nt)) return bad("tensor map of X", MOE_ERR_CUDA);
  if (!map_rows(&g.mapW, W, c.d, c.N, rows)) return bad("tensor map of W", MOE_ERR_CUDA);
  if (L.adapters && !map_adapters(&g.mapB, B, c.r, c.N, c.n, rows, g.pc)) return bad("tensor map of B", MOE_ERR_CUDA);
  if (L.adapters && (!map_rows(&g.mapU, g.u, 3 * g.pc * RS, c.T, L.nt, 2 * g.pc) ||
                     !map_rows(&g.mapU3, g.u, 3 * g.pc * RS, c.T, L.nt, g.pc)))
    return bad("tensor map of u", MOE_ERR_CUDA);
  g.chunk = c.out_f32 ? chunk : whole;

  cudaError_t e;
  const bool dots = L.adapters && (int64_t)c.T * c.r * c.d <= kDotWork * (L.row_tiles == 1 ? 1 : 2);
  if (L.wide && !dots) {
    e = launch_pdl(low_list_kernel, dim3(1), dim3(kListWarps * 32), 0, st, 1, g, l);
    if (e != cudaSuccess) return cuda_bad("adapter list launch", e);
    if (L.adapters) {
      LinArgs a = g;
      if (!map_rows(&a.mapW, A, c.d, (int64_t)c.n * c.r, kRowsLow)) return bad("tensor map of A", MOE_ERR_CUDA);
      a.cnt = g.cnt + sms;
      a.chunk = chunk;
      a.high = 0;
      a.all = L.row_tiles == 1;
      e = launch_one<kRowsLow, 16, true, 1>(a, sms, st);
      if (e != cudaSuccess) return cuda_bad("adapter product launch", e);
    }
    e = launch_wide(g, sms, st);
  } else {
    l.list_ctas = L.wide ? (L.groups + kDotWarps - 1) / kDotWarps : 0;
    const dim3 grid = L.adapters ? dim3((unsigned)(l.list_ctas + c.T), c.r / 8) : dim3(1);
    e = launch_pdl(low_dot_kernel, grid, dim3(kDotWarps * 32), 0, st, 1, g, l);
    if (e != cudaSuccess) return cuda_bad("adapter dot launch", e);
    e = L.wide ? launch_wide(g, sms, st) : launch_high<kRowsFew, 1>(g, sms, st);
  }
  if (e != cudaSuccess) return cuda_bad("launch", e);
  return MOE_OK;
}
