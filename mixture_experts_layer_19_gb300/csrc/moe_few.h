// moe_few.h -- the layer for few tokens: what the C ABI (api.cu) hands to the kernel (moe_few.cu).
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int kFewTokens = 64;   // a token is a bit of an expert's 64-bit mask

struct FewArgs {
  CUtensorMap mapG, mapU, mapD;   // weights: Wg, Wu in boxes of 128 rows, Wd of 256 (128 bytes wide)
  CUtensorMap mapX, mapH;         // tokens; rows of h sorted by expert (boxes of 16 rows)
  const __nv_bfloat16* X;
  const __nv_bfloat16* Wr;        // router weight, or null: `logits` is the input
  const float* logits;            // [T, E] (with Wr: workspace, written here)
  float* logits_out;
  // block-scaled plans: scale atoms of the weights, the quantised tokens and h
  const uint8_t *sfG, *sfU, *sfD;
  uint8_t *Xq, *Xs, *Hs;
  const float* ts;                // NVFP4: tensor scales [Wg and Wu, Wd]
  uint8_t* H;                     // [2 T k, F] bf16 (h and what its rounding left), or [T k, F] quantised
  float* y;                       // [T k, d] the experts' results
  float* part;                    // [4 CTAs][part_rows][256] parts of sums cut between CTAs
  int *cnt_up, *cnt_dn;           // arrivals of parts, per tile and epilogue warp; zero between launches, as are
  int* ready;                     //   finished parts of h per expert,
  int* done;                      //   epilogue warps that are done,
  unsigned long long* gate;       //   and CTAs that have passed the prologue / left
  __nv_bfloat16* Y;
  int32_t* status;
  uint64_t timeout_ns;
  int T, d, F, E, k;
  int part_rows;                  // most tokens that the plan's calls have, 64 at most
  int stages, b_bytes;            // ring stages, bytes of activations per stage
  int n_up, n_dn;                 // how many tile counters there are
  int stall;                      // test hook: no weights are loaded, every wait expires
};

// prec: moe_precision_t
cudaError_t prepare_moe_few(int prec);
size_t moe_few_smem(int prec, int T, int E, int k, int* stages, int* b_bytes);
cudaError_t launch_moe_few(int prec, const FewArgs& a, int grid, size_t smem, cudaStream_t st);

}  // namespace moe
