// Gradient of the gate-weighted combine (combine.cu):
//   dgate[t][j] = <dout[t], y_perm[q]>,   dy_perm[q] = gate[t][j] * dout[t],   q = inv_perm[t*k+j]
// for the pairs the combine adds; the others get dgate = 0 and keep their
// dy_perm row.
//
// One pass: a CTA takes a token and up to 8 of its pairs at once, or one pair
// where the tokens are too few to fill the SMs; it reads its dout row once for
// them, and each pair's y row is read where its dy row is written.  y and dy pass
// through the caches once and are marked so.  Bound by HBM: per token (k + 1)
// rows read and k written.  A dot is summed in fp32: per thread over its columns,
// then over the lanes of a warp, then over the warps -- a fixed order.
#include "common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

template <int PAIRS>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(
    const float* __restrict__ y_perm, const int32_t* __restrict__ idx, const float* __restrict__ gate,
    const int32_t* __restrict__ inv_perm, const int32_t* __restrict__ slot, const float* __restrict__ dout, int T,
    int k, int d, int E_bound, int nq, float* __restrict__ dgate, float* __restrict__ dy_perm) {
  __shared__ float part[kThreads / 32][PAIRS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = PAIRS == 1 ? blockIdx.x / k : blockIdx.x;
  const int first = PAIRS == 1 ? blockIdx.x % k : 0, last = PAIRS == 1 ? first + 1 : k;
  pdl_wait();
  pdl_trigger();
  const float4* drow = reinterpret_cast<const float4*>(dout + static_cast<size_t>(t) * d);
  for (int j0 = first; j0 < last; j0 += PAIRS) {
    int q[PAIRS];
    float g[PAIRS], dot[PAIRS];
#pragma unroll
    for (int jj = 0; jj < PAIRS; ++jj) {
      const int p = t * k + j0 + jj;
      q[jj] = j0 + jj < last ? __ldg(inv_perm + p) : -1;
      g[jj] = (dy_perm != nullptr && j0 + jj < last) ? __ldg(gate + p) : 0.f;
      if (q[jj] >= nq) q[jj] = -1;
      if (slot != nullptr && q[jj] >= 0) {
        const int e = __ldg(idx + p);
        if (e < 0 || e >= E_bound || __ldg(slot + e) < 0) q[jj] = -1;
      }
      dot[jj] = 0.f;
    }
    for (int c = threadIdx.x; c * 4 < d; c += kThreads) {
      const float4 o = __ldg(drow + c);
      float4 y[PAIRS];
#pragma unroll
      for (int jj = 0; jj < PAIRS; ++jj)
        if (q[jj] >= 0) y[jj] = __ldcs(reinterpret_cast<const float4*>(y_perm + static_cast<size_t>(q[jj]) * d) + c);
#pragma unroll
      for (int jj = 0; jj < PAIRS; ++jj) {
        if (q[jj] < 0) continue;
        dot[jj] = fmaf(o.x, y[jj].x, fmaf(o.y, y[jj].y, fmaf(o.z, y[jj].z, fmaf(o.w, y[jj].w, dot[jj]))));
        if (dy_perm != nullptr)
          __stcs(reinterpret_cast<float4*>(dy_perm + static_cast<size_t>(q[jj]) * d) + c,
                 make_float4(g[jj] * o.x, g[jj] * o.y, g[jj] * o.z, g[jj] * o.w));
      }
    }
#pragma unroll
    for (int jj = 0; jj < PAIRS; ++jj) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) dot[jj] += __shfl_xor_sync(kFull, dot[jj], off);
      if (lane == 0) part[warp][jj] = dot[jj];
    }
    __syncthreads();
    if (threadIdx.x < PAIRS && j0 + static_cast<int>(threadIdx.x) < last) {
      float s = 0.f;
      for (int w = 0; w < kThreads / 32; ++w) s += part[w][threadIdx.x];
      dgate[static_cast<size_t>(t) * k + j0 + threadIdx.x] = s;
    }
    __syncthreads();
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
  const bool few = T < 4 * dev.sm_count;
  MOE_CUDA_TRY(launch_pdl(few ? combine_backward_kernel<1> : combine_backward_kernel<8>, dim3(few ? T * k : T),
                          dim3(kThreads), 0, stream, y_perm, idx, gate, inv_perm, slot_of_expert, dout, T, k, d, E, T * k,
                          dgate, dy_perm));
  MOE_LAUNCH_CHECK("combine_backward_kernel");
  return MOE_OK;
}
