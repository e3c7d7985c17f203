// head_gemm.cu -- instantiations and launches of the loss head's GEMMs.
#include "head_gemm.cuh"

namespace moe {

namespace {

template <int KIND, int CG, bool TEACHER, int AR = kHBM, bool PARTS = false>
cudaError_t prepare_one() {
  auto kernel = head_gemm_kernel<KIND, CG, TEACHER, AR, PARTS>;
  if constexpr (head_regs<KIND, PARTS>) {
    // a launch with fewer registers than the warps' shares would wait for them without end
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, kernel);
    if (e != cudaSuccess) return e;
    if (a.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;
  }
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, HeadTraits<KIND, CG, AR>::smem_bytes);
}

template <int KIND, int CG, bool TEACHER, int AR = kHBM, bool PARTS = false>
cudaError_t launch_one(const HeadArgs& a, int grid, cudaStream_t st) {
  return launch_pdl(head_gemm_kernel<KIND, CG, TEACHER, AR, PARTS>, dim3(grid), dim3(head_threads<KIND, PARTS>),
                    HeadTraits<KIND, CG, AR>::smem_bytes, st, CG, a);
}

template <int KIND, int CG, int AR>
cudaError_t launch_targets(const HeadArgs& a, int grid, cudaStream_t st) {
  if (KIND == kHeadDl && a.d > logits_chunk(AR) * kHBK)
    return a.first ? launch_one<KIND, CG, true, AR, KIND == kHeadDl>(a, grid, st)
                   : launch_one<KIND, CG, false, AR, KIND == kHeadDl>(a, grid, st);
  return a.first ? launch_one<KIND, CG, true, AR>(a, grid, st) : launch_one<KIND, CG, false, AR>(a, grid, st);
}

template <int KIND>
cudaError_t launch_logits(bool pair, int arows, const HeadArgs& a, int grid, cudaStream_t st) {
  if (pair) return launch_targets<KIND, 2, kHBM>(a, grid, st);
  if (arows == 16) return launch_targets<KIND, 1, 16>(a, grid, st);
  if (arows == 64) return launch_targets<KIND, 1, 64>(a, grid, st);
  return launch_targets<KIND, 1, kHBM>(a, grid, st);
}

template <int KIND, bool PARTS>
cudaError_t prepare_logits() {
  cudaError_t e = prepare_one<KIND, 2, false, kHBM, PARTS>();
  if (e == cudaSuccess) e = prepare_one<KIND, 2, true, kHBM, PARTS>();
  if (e == cudaSuccess) e = prepare_one<KIND, 1, false, kHBM, PARTS>();
  if (e == cudaSuccess) e = prepare_one<KIND, 1, true, kHBM, PARTS>();
  if (e == cudaSuccess) e = prepare_one<KIND, 1, false, 16, PARTS>();
  if (e == cudaSuccess) e = prepare_one<KIND, 1, true, 16, PARTS>();
  if (e == cudaSuccess) e = prepare_one<KIND, 1, false, 64, PARTS>();
  if (e == cudaSuccess) e = prepare_one<KIND, 1, true, 64, PARTS>();
  return e;
}

}  // namespace

cudaError_t head_gemm_prepare() {
  cudaError_t e = prepare_logits<kHeadLse, false>();
  if (e == cudaSuccess) e = prepare_logits<kHeadDl, false>();
  if (e == cudaSuccess) e = prepare_logits<kHeadDl, true>();
  if (e == cudaSuccess) e = prepare_one<kHeadDX, 1, false>();
  if (e == cudaSuccess) e = prepare_one<kHeadDX, 1, false, 16>();
  if (e == cudaSuccess) e = prepare_one<kHeadDX, 1, false, 64>();
  if (e == cudaSuccess) e = prepare_one<kHeadDX, 2, false>();
  if (e == cudaSuccess) e = prepare_one<kHeadDW, 1, false>();
  if (e == cudaSuccess) e = prepare_one<kHeadDW, 2, false>();
  return e;
}

cudaError_t head_gemm_launch(int kind, bool pair, int arows, const HeadArgs& a, int grid, cudaStream_t st) {
  switch (kind) {
    case kHeadLse: return launch_logits<kHeadLse>(pair, arows, a, grid, st);
    case kHeadDl: return launch_logits<kHeadDl>(pair, arows, a, grid, st);
    case kHeadDX:
      if (pair) return launch_one<kHeadDX, 2, false>(a, grid, st);
      if (arows == 16) return launch_one<kHeadDX, 1, false, 16>(a, grid, st);
      if (arows == 64) return launch_one<kHeadDX, 1, false, 64>(a, grid, st);
      return launch_one<kHeadDX, 1, false>(a, grid, st);
    default: return pair ? launch_one<kHeadDW, 2, false>(a, grid, st) : launch_one<kHeadDW, 1, false>(a, grid, st);
  }
}

// How many CTA pairs the device holds at once: the static schedule's grid.
cudaError_t head_gemm_max_pairs(int* pairs) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(head_threads<kHeadDl, true>);
  cfg.dynamicSmemBytes = HeadTraits<kHeadDl, 2, kHBM>::smem_bytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(pairs, head_gemm_kernel<kHeadDl, 2, false, kHBM, true>, &cfg);
}

}  // namespace moe
