// The dense 4-bit linear over MXFP4 and NVFP4 weights on the 5th-generation tensor cores (linear_w4_tc.cuh).
#include "linear_w4_tc.cuh"

namespace moe {

cudaError_t launch_linear_tc_fp4(const LinearParams& P, int fmt, bool bf16, const DeviceInfo& dev, int32_t* status,
                                 cudaStream_t s) {
  if (fmt == MOE_W_MXFP4)
    return bf16 ? w4tc::launch_tokens<MOE_W_MXFP4, 32, true>(P, dev, status, s) : w4tc::launch_tokens<MOE_W_MXFP4, 32, false>(P, dev, status, s);
  return bf16 ? w4tc::launch_tokens<MOE_W_NVFP4, 16, true>(P, dev, status, s) : w4tc::launch_tokens<MOE_W_NVFP4, 16, false>(P, dev, status, s);
}

}  // namespace moe
