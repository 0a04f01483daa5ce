// Instantiations of the split kernel for sliding windows with first tokens that stay visible.
#include "pa_split.cuh"

namespace pa {
namespace {

using Kernel = void (*)(CUtensorMap, CUtensorMap, SplitParams);

Kernel kernel_of(int d, bool fp8, bool tok) {
  if (d == 128)
    return tok ? pa_split_kernel<128, true, true, true, Walk::kFirst>
               : fp8 ? pa_split_kernel<128, true, true, false, Walk::kFirst>
                     : pa_split_kernel<128, false, true, false, Walk::kFirst>;
  if (d == 64)
    return tok ? pa_split_kernel<64, true, true, true, Walk::kFirst>
               : fp8 ? pa_split_kernel<64, true, true, false, Walk::kFirst>
                     : pa_split_kernel<64, false, true, false, Walk::kFirst>;
  return nullptr;
}

}  // namespace

cudaError_t launch_split_first(int head_dim, bool fp8, const CUtensorMap& tk, const CUtensorMap& tv,
                              const SplitParams& p, int grid, int threads, int smem, bool pdl, cudaStream_t stream) {
  const Kernel k = kernel_of(head_dim, fp8, p.k_tok != nullptr);
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

cudaError_t set_split_smem_limits_first(int smem) {
  for (int d = 64; d <= 128; d += 64)
    for (int form = 0; form < 3; ++form) {
      const Kernel k = kernel_of(d, form > 0, form == 2);
      const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(k),
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

}  // namespace pa
