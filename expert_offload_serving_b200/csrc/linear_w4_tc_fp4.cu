// The dense 4-bit linear over MXFP4 and NVFP4 weights on the 5th-generation tensor cores (linear_w4_tc.cuh,
// linear_w4_tc16.cuh).
#include "linear_w4_tc16.cuh"

namespace moe {
namespace {

// MXFP4: up to 16 tokens the narrow kernel, which is the faster one for it.
template <bool BF16>
cudaError_t launch_mxfp4(const LinearParams& P, const DeviceInfo& dev, int32_t* status, cudaStream_t s) {
  return P.T <= w4t16::NT ? w4t16::launch<MOE_W_MXFP4, 32, BF16>(P, dev, status, s)
                          : w4tc::launch_tokens<MOE_W_MXFP4, 32, BF16>(P, dev, status, s);
}

}  // namespace

cudaError_t launch_linear_tc_fp4(const LinearParams& P, int fmt, bool bf16, const DeviceInfo& dev, int32_t* status,
                                 cudaStream_t s) {
  if (fmt == MOE_W_MXFP4)
    return bf16 ? launch_mxfp4<true>(P, dev, status, s) : launch_mxfp4<false>(P, dev, status, s);
  return bf16 ? w4tc::launch_tokens<MOE_W_NVFP4, 16, true>(P, dev, status, s)
              : w4tc::launch_tokens<MOE_W_NVFP4, 16, false>(P, dev, status, s);
}

}  // namespace moe
