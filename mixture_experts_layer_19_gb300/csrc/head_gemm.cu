// head_gemm.cu -- instantiations and launches of the loss head's GEMMs.
#include "head_gemm.cuh"

namespace moe {

namespace {

template <int KIND, int CG, bool TEACHER>
cudaError_t prepare_one() {
  return cudaFuncSetAttribute(head_gemm_kernel<KIND, CG, TEACHER>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              HeadTraits<KIND, CG>::smem_bytes);
}

template <int KIND, int CG, bool TEACHER>
cudaError_t launch_one(const HeadArgs& a, int grid, cudaStream_t st) {
  return launch_pdl(head_gemm_kernel<KIND, CG, TEACHER>, dim3(grid), dim3(kHeadThreads), HeadTraits<KIND, CG>::smem_bytes, st,
                    CG, a);
}

template <int CG>
cudaError_t launch_kind(int kind, const HeadArgs& a, int grid, cudaStream_t st) {
  const bool teacher = a.first != nullptr;
  switch (kind) {
    case kHeadLse:
      return teacher ? launch_one<kHeadLse, CG, true>(a, grid, st) : launch_one<kHeadLse, CG, false>(a, grid, st);
    case kHeadDl:
      return teacher ? launch_one<kHeadDl, CG, true>(a, grid, st) : launch_one<kHeadDl, CG, false>(a, grid, st);
    case kHeadDX: return launch_one<kHeadDX, CG, false>(a, grid, st);
    default: return launch_one<kHeadDW, CG, false>(a, grid, st);
  }
}

template <int CG>
cudaError_t prepare_kinds() {
  cudaError_t e = prepare_one<kHeadLse, CG, false>();
  if (e == cudaSuccess) e = prepare_one<kHeadLse, CG, true>();
  if (e == cudaSuccess) e = prepare_one<kHeadDl, CG, false>();
  if (e == cudaSuccess) e = prepare_one<kHeadDl, CG, true>();
  if (e == cudaSuccess) e = prepare_one<kHeadDX, CG, false>();
  if (e == cudaSuccess) e = prepare_one<kHeadDW, CG, false>();
  return e;
}

}  // namespace

cudaError_t head_gemm_prepare() {
  cudaError_t e = prepare_kinds<1>();
  return e == cudaSuccess ? prepare_kinds<2>() : e;
}

cudaError_t head_gemm_launch(int kind, bool pair, const HeadArgs& a, int grid, cudaStream_t st) {
  return pair ? launch_kind<2>(kind, a, grid, st) : launch_kind<1>(kind, a, grid, st);
}

// How many CTA pairs the device holds at once: the static schedule's grid.
cudaError_t head_gemm_max_pairs(int* pairs) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(kHeadThreads);
  cfg.dynamicSmemBytes = HeadTraits<kHeadDl, 2>::smem_bytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(pairs, head_gemm_kernel<kHeadDl, 2, false>, &cfg);
}

}  // namespace moe
