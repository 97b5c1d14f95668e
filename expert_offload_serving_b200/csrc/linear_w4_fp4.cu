// The dense 4-bit linear over MXFP4 and NVFP4 weights (linear_w4.cuh).
#include "linear_w4.cuh"

namespace moe {

cudaError_t launch_linear_fp4(const LinearParams& P, int fmt, bool bf16, const DeviceInfo& dev, cudaStream_t s) {
  if (fmt == MOE_W_MXFP4)
    return bf16 ? w4::launch_tokens<MOE_W_MXFP4, 32, true>(P, dev, s) : w4::launch_tokens<MOE_W_MXFP4, 32, false>(P, dev, s);
  return bf16 ? w4::launch_tokens<MOE_W_NVFP4, 16, true>(P, dev, s) : w4::launch_tokens<MOE_W_NVFP4, 16, false>(P, dev, s);
}

}  // namespace moe
