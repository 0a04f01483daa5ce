// Instantiations of the split kernel for sequences behind a shared prefix.
#include "pa_split.cuh"

namespace pa {
namespace {

using Kernel = void (*)(CUtensorMap, CUtensorMap, SplitParams);

Kernel kernel_of(int d, bool fp8) {
  if (d == 128)
    return fp8 ? pa_split_kernel<128, true, false, false, Walk::kOwn>
               : pa_split_kernel<128, false, false, false, Walk::kOwn>;
  if (d == 64)
    return fp8 ? pa_split_kernel<64, true, false, false, Walk::kOwn>
               : pa_split_kernel<64, false, false, false, Walk::kOwn>;
  return nullptr;
}

}  // namespace

cudaError_t launch_split_own(int head_dim, bool fp8, const CUtensorMap& tk, const CUtensorMap& tv,
                              const SplitParams& p, int grid, int threads, int smem, bool pdl, cudaStream_t stream) {
  const Kernel k = kernel_of(head_dim, fp8);
  if (k == nullptr) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k, tk, tv, p);
}

cudaError_t set_split_smem_limits_own(int smem) {
  for (int d = 64; d <= 128; d += 64)
    for (int fp8 = 0; fp8 < 2; ++fp8) {
      const Kernel k = kernel_of(d, fp8 != 0);
      const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(k),
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

}  // namespace pa
