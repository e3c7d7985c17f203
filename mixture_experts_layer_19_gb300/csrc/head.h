// head.h -- internal interface of the loss head (cross entropy and
// distillation over logits = X W^T that are never stored whole): the GEMM
// kinds of head_gemm.cuh and the row kernels of head_rows.cu, as head.cu
// launches them.  Not part of the public ABI.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

namespace moe {

constexpr int kHeadRowPad = 256;    // compact row buffers are padded to this many rows
constexpr int kHeadBN = 256;        // vocabulary (or d) columns of one tile
constexpr int kHeadMaxEntries = 1024;

enum HeadKind { kHeadLse = 0, kHeadDl = 1, kHeadDX = 2, kHeadDW = 3 };

// Arguments of one head GEMM launch.  "Compact" rows are the rows with a loss
// (and, in the backward, a nonzero upstream gradient), in token order.
struct HeadArgs {
  CUtensorMap mapA0;         // A operand; X itself when every row is active
  CUtensorMap mapA1;         // kHeadLse / kHeadDl: the compacted copy of X
  CUtensorMap mapB0;         // B operand; kHeadDW: X itself
  CUtensorMap mapB1;         // kHeadDW: the compacted copy of X
  const int32_t* n_active;   // [1] compact rows; NULL: every token has its own row (kHeadLse, one row tile),
                             //   and what counts is read from labels or cnt
  const void* labels;        // [T] int32, or int64 with ids64
  const int32_t* cnt;        // [T] distillation: entries in use
  int ids64;
  int64_t V;
  const int4* rec;           // [Tp] of each compact row: token, label (or teacher entries in use), and, as float
                             //   bits for kHeadDl, log-sum-exp and upstream gradient / *scale
  const int32_t* ids;        // distillation: [T, K] entries in use of each token, ids ascending
  const float* probs;        // [T, K] their probabilities
  const uint16_t* first;     // [T, blocks] first entry at or past vocabulary column 128 * block; NULL: labels
  int64_t blocks;
  const float* scale;        // [1] common factor of dloss, taken out of D and applied to the sums
  float2* part;              // kHeadLse: [2 * NT, Tp] (max, sum of exp) of 128 columns of one row
  float* zt;                 // kHeadLse: [T, K] logits at the target entries
  __nv_bfloat16* dl;         // kHeadDl: [Tp, ldl] this piece of D
  int64_t ldl;
  float* acc;                // kHeadDX: [nsplit, Tp, d] fp32 sums
  __nv_bfloat16* dX;         // kHeadDX: [T, d], written instead of the sums (last piece, nsplit = 1); else NULL
  __nv_bfloat16* dW;         // kHeadDW: [V, d]
  int32_t* status;
  uint64_t timeout_ns;
  int64_t Tp;                // padded rows of the compact buffers
  int64_t v0, vlen;          // this piece of the vocabulary (kHeadLse: all of it)
  int T, d, K;
  int bn;                    // kHeadLse, kHeadDl: columns of a tile, 64, 128, 192 or 256 (arows < 128)
  int nsplit;                // kHeadDX: the vocabulary piece is split over this many tiles
  int add;                   // kHeadDX: add into the fp32 sums (0: first piece, overwrite)
  float inv_temp;            // 1 / temperature
  float out_scale;           // temperature, multiplied with *scale
  int beside;                // kHeadDW: the launch before is this call's dX
  int stall;                 // test hook: the producer issues nothing
};

cudaError_t head_gemm_prepare();
// pair: two CTAs work on one 256-row tile (cta_group::2); otherwise one CTA on 128 rows.
// arows (without pairs, not kHeadDW): rows of A per tile, 16, 64 or 128.
cudaError_t head_gemm_launch(int kind, bool pair, int arows, const HeadArgs& a, int grid, cudaStream_t st);
cudaError_t head_gemm_max_pairs(int* pairs);

// ---- row kernels (head_rows.cu)
struct HeadRows {
  int32_t* n_active;   // [4]
  float* scale;        // [1] common factor of the upstream gradients (backward)
  int4* rec;           // [Tp] see HeadArgs
  int32_t* inv;        // [T] compact row of each token, -1 = inactive
  int32_t* ids;        // [T, K] (distillation)
  float* probs;        // [T, K] (distillation)
  uint16_t* first;     // [T, blocks] (distillation)
  int64_t blocks;
  int32_t* cnt;        // [T]    (distillation)
  float* plogp;        // [T]    (distillation, forward) sum p log p
  void* Xc;            // [Tp, d] bf16
  float2* part;        // [2 * NT, Tp]
  float* zt;           // [T, K]
  void* dl;            // [Tp, piece] bf16
  float* acc;          // [S, Tp, d]
};

cudaError_t launch_head_entries(const void* teacher, bool teacher_bf16, const void* ids, bool ids64, int T, int K,
                                int64_t V, float inv_temp, const HeadRows& r, cudaStream_t st);
// The list of rows that count and, when some do not, their compact copy of X.
// labels != NULL: cross entropy; otherwise r.cnt says which rows count.
// dX != NULL: rows of tokens that do not count are zeroed.
cudaError_t launch_head_prep(const void* labels, bool ids64, const float* dloss, const float* lse, const void* X,
                             int T, int d, int64_t V, const HeadRows& r, void* dX, int num_sms, cudaStream_t st);
// r.inv == NULL: no list of rows was made; token t has row t, and labels (or r.cnt) say whether it counts.
cudaError_t launch_head_loss(const void* labels, bool ids64, int T, int64_t V, int K, int np, int64_t Tp,
                             float temperature, bool distill, const HeadRows& r, float* loss, float* lse,
                             cudaStream_t st);
// dX rows of the tokens that count, from the splits' sums.
cudaError_t launch_head_dx(int T, int d, int nsplit, int64_t Tp, float out_scale, const HeadRows& r, void* dX,
                           int num_sms, cudaStream_t st);

}  // namespace moe
