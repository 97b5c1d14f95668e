// The dense 4-bit linear over INT4 weights (linear_w4.cuh).
#include "linear_w4.cuh"

namespace moe {

cudaError_t launch_linear_int4(const LinearParams& P, int group, bool bf16, const DeviceInfo& dev, cudaStream_t s) {
  switch (group) {
    case 32: return bf16 ? w4::launch_tokens<MOE_W_INT4, 32, true>(P, dev, s)
                         : w4::launch_tokens<MOE_W_INT4, 32, false>(P, dev, s);
    case 64: return bf16 ? w4::launch_tokens<MOE_W_INT4, 64, true>(P, dev, s)
                         : w4::launch_tokens<MOE_W_INT4, 64, false>(P, dev, s);
    default: return bf16 ? w4::launch_tokens<MOE_W_INT4, 128, true>(P, dev, s)
                         : w4::launch_tokens<MOE_W_INT4, 128, false>(P, dev, s);
  }
}

}  // namespace moe
