// The dense 4-bit linear over INT4 weights on the 5th-generation tensor cores (linear_w4_tc.cuh,
// linear_w4_tc16.cuh).
#include "linear_w4_tc16.cuh"

namespace moe {
namespace {

// Up to 16 tokens the narrow kernel, for the groups that it is the faster one for.
template <int GROUP, bool BF16>
cudaError_t launch(const LinearParams& P, const DeviceInfo& dev, int32_t* status, cudaStream_t s) {
  if constexpr (GROUP >= 64) {
    if (P.T <= w4t16::NT) return w4t16::launch<MOE_W_INT4, GROUP, BF16>(P, dev, status, s);
  }
  if constexpr (BF16) {
    if (scales_outside(P, MOE_W_INT4, true)) return w4tc::launch_tokens<MOE_W_INT4, GROUP, true, true>(P, dev, status, s);
  }
  return w4tc::launch_tokens<MOE_W_INT4, GROUP, BF16>(P, dev, status, s);
}

}  // namespace

cudaError_t launch_linear_tc_int4(const LinearParams& P, int group, bool bf16, const DeviceInfo& dev, int32_t* status,
                                 cudaStream_t s) {
  switch (group) {
    case 32: return bf16 ? launch<32, true>(P, dev, status, s)
                         : launch<32, false>(P, dev, status, s);
    case 64: return bf16 ? launch<64, true>(P, dev, status, s)
                         : launch<64, false>(P, dev, status, s);
    default: return bf16 ? launch<128, true>(P, dev, status, s)
                         : launch<128, false>(P, dev, status, s);
  }
}

}  // namespace moe
