// Gradient of the gate-weighted combine (combine.cu):
//   dgate[t][j] = <dout[t], y_perm[q]>,   dy_perm[q] = gate[t][j] * dout[t],   q = inv_perm[t*k+j]
// for the pairs the combine adds; the others get dgate = 0 and keep their
// dy_perm row.
//
// A CTA per pair: it reads the pair's y row and writes its dy row, and reads its
// token's dout row, which the token's other pairs find in L2.  Bound by HBM: per
// token (k + 1) rows read and k written.  Against a CTA per token with 8 pairs at
// once (dout read once, 128 registers): 104 against 121 us at T = 4096, k = 6,
// d = 4096 (6.1 against 5.2 TB/s of the 631 MB; HBM bounds it; without dy 64.5 us, 5.4
// TB/s of 349 MB), 2.4 against 7.3 us at T = 16, k = 8, d = 2048 (the launch and three
// dependent loads).  y and dy pass through the caches once and are marked so.  A
// dot is summed in fp32: per thread over its columns, then over the lanes of a
// warp, then over the warps -- a fixed order.
#include "common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;         // at most

__global__ void __launch_bounds__(kThreads) combine_backward_kernel(
    const float* __restrict__ y_perm, const int32_t* __restrict__ idx, const float* __restrict__ gate,
    const int32_t* __restrict__ inv_perm, const int32_t* __restrict__ slot, const float* __restrict__ dout, int k,
    int d, int E_bound, int pairs, float* __restrict__ dgate, float* __restrict__ dy_perm) {
  __shared__ float part[kThreads / 32];
  const int p = blockIdx.x, threads = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  const int q = __ldg(inv_perm + p);
  bool use = q >= 0 && q < pairs;
  if (slot != nullptr && use) {
    const int e = __ldg(idx + p);
    use = e >= 0 && e < E_bound && __ldg(slot + e) >= 0;
  }
  if (!use) {                          // the same for the whole CTA
    if (threadIdx.x == 0) dgate[p] = 0.f;
    return;
  }
  const float4* o = reinterpret_cast<const float4*>(dout + static_cast<size_t>(p / k) * d);
  const float4* y = reinterpret_cast<const float4*>(y_perm + static_cast<size_t>(q) * d);
  float4* dy = dy_perm == nullptr ? nullptr : reinterpret_cast<float4*>(dy_perm + static_cast<size_t>(q) * d);
  const float g = dy_perm == nullptr ? 0.f : __ldg(gate + p);
  float dot = 0.f;
#pragma unroll 4
  for (int c = threadIdx.x; c < d / 4; c += threads) {
    const float4 a = __ldg(o + c), b = __ldcs(y + c);
    dot = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, dot))));
    if (dy != nullptr) __stcs(dy + c, make_float4(g * a.x, g * a.y, g * a.z, g * a.w));
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(kFull, dot, off);
  if (lane == 0) part[warp] = dot;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < threads >> 5; ++w) dot += part[w];
    dgate[p] = dot;
  }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_combine_backward(const float* y_perm, const int32_t* idx, const float* gate,
                                           const int32_t* inv_perm, const int32_t* slot_of_expert, const float* dout,
                                           int T, int k, int d, int E, float* dgate, float* dy_perm,
                                           cudaStream_t stream) {
  clear_error();
  MOE_REQUIRE(T >= 0 && k >= 1 && k <= 32 && d >= 4 && d % 4 == 0, "T=%d, k=%d, d=%d", T, k, d);
  MOE_REQUIRE(E >= 1 && E <= 1024, "E=%d outside [1, 1024]", E);
  MOE_REQUIRE(static_cast<long long>(T) * k <= (1 << 24), "T*k too large");
  if (T == 0) return MOE_OK;
  MOE_REQUIRE(y_perm && idx && inv_perm && dout && dgate, "null pointer");
  MOE_REQUIRE(dy_perm == nullptr || gate != nullptr, "dy_perm needs gate");
  MOE_REQUIRE(aligned(y_perm, 16) && aligned(dout, 16) && (!dy_perm || aligned(dy_perm, 16)),
              "y_perm, dout and dy_perm must be 16-byte aligned");
  MOE_REQUIRE(aligned(idx, 4) && aligned(gate, 4) && aligned(inv_perm, 4) && aligned(dgate, 4) &&
                  aligned(slot_of_expert, 4), "misaligned pointer");
  DeviceInfo dev;
  const moe_status st = current_device(&dev);
  if (st != MOE_OK) return st;
  const int threads = d / 4 >= kThreads ? kThreads : (d / 4 + 31) / 32 * 32;
  MOE_CUDA_TRY(launch_pdl(combine_backward_kernel, dim3(T * k), dim3(threads), 0, stream, y_perm, idx, gate, inv_perm,
                          slot_of_expert, dout, k, d, E, T * k, dgate, dy_perm));
  MOE_LAUNCH_CHECK("combine_backward_kernel");
  return MOE_OK;
}
