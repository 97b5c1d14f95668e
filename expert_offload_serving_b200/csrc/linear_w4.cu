// moe_linear_w4: argument checks and dispatch (the kernel: linear_w4.cuh).
#include <cstdlib>
#include <cstring>

#include "linear_w4.cuh"

namespace moe {
namespace {

// Which kernel: warp-level MMAs (linear_w4.cuh) or tcgen05 (linear_w4_tc.cuh,
// linear_w4_tc16.cuh).  A tcgen05 tile of 128 rows is a chain of stages that takes
// 0.5 to 1 us a 1024 of K however few tokens it serves.  Above 16 tokens clusters
// share that chain where tiles are few; up to 16, enough tiles to fill the SMs pay
// for it.  Device time in us, warp / tcgen05, K = 4096 (weights of N <= 16384 in L2):
//   T = 8    N = 16384   INT4/128 14.9 / 17.9   INT4/32 22.9 / 30.7  MXFP4 24.2 / 26.3  NVFP4 23.2 / 29.5
//   T = 16   N = 4096    INT4/128  8.6 / 17.6   INT4/32 10.9 / 12.1  MXFP4 10.9 / 26.0  NVFP4  9.6 / 11.6
//            N = 16384   INT4/128 23.2 / 18.0   INT4/32 28.1 / 31.0  MXFP4 29.6 / 26.4  NVFP4 28.3 / 29.5
//            N = 131072  INT4/128  146 / 114    INT4/32  193 / 200   MXFP4  195 / 170   NVFP4  192 / 190
//   T = 17   N = 1024    INT4/128 17.4 /  7.6   INT4/32 21.1 /  8.9  MXFP4 21.6 /  7.6  NVFP4 19.0 /  8.6
//            N = 16384   INT4/128 26.9 / 23.2   INT4/32 30.8 / 30.8  MXFP4 32.0 / 25.6  NVFP4 30.6 / 29.6
//   T = 64   N = 16384   INT4/128 52.1 / 26.8   INT4/32 84.3 / 38.5  MXFP4 86.0 / 27.4  NVFP4 76.2 / 31.7
//   T = 512  N = 4096    INT4/128 90.8 / 38.5   INT4/32  148 / 51.8  MXFP4  150 / 32.1  NVFP4  133 / 38.0
// MOE_LINEAR=warp|tc, read at every call, forces one.
bool use_tc(const LinearParams& P, int fmt, int group, const DeviceInfo& dev) {
  const char* force = getenv("MOE_LINEAR");
  if (force != nullptr) return strcmp(force, "tc") == 0;
  if (P.T > 16) return true;
  const bool fills = P.N >= 77 * dev.sm_count;                 // 0.6 tiles of 128 rows for each SM
  return P.T > 8 && fills && (fmt == MOE_W_MXFP4 || (fmt == MOE_W_INT4 && group >= 64));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_linear_w4(moe_linear_shape s, const void* codes, const void* scales, const uint8_t* zeros,
                                    float tensor_scale, const void* x, int x_type, int64_t ldx, int T, void* y,
                                    int y_type, int64_t ldy, int flags, int32_t* dev_status,
                                    cudaStream_t stream) {
  clear_error();
  MOE_REQUIRE(s.N >= 1 && s.N <= (1 << 24), "N=%d outside [1, %d]", s.N, 1 << 24);
  MOE_REQUIRE(s.K >= 32 && s.K <= (1 << 17) && s.K % 32 == 0, "K=%d: a multiple of 32 up to %d", s.K, 1 << 17);
  const bool int4 = s.fmt == MOE_W_INT4;
  MOE_REQUIRE(int4 || s.fmt == MOE_W_MXFP4 || s.fmt == MOE_W_NVFP4, "unknown weight format %d", s.fmt);
  if (int4) {
    MOE_REQUIRE(s.group == 32 || s.group == 64 || s.group == 128, "INT4 group %d: 32, 64 or 128", s.group);
    MOE_REQUIRE(s.scale_type >= MOE_DT_F32 && s.scale_type <= MOE_DT_F16, "scale type %d", s.scale_type);
  } else {
    MOE_REQUIRE(s.group == (s.fmt == MOE_W_MXFP4 ? 32 : 16), "group %d: 32 (MXFP4) or 16 (NVFP4)", s.group);
    MOE_REQUIRE(zeros == nullptr, "zeros belong to INT4");
  }
  MOE_REQUIRE(T >= 0 && T <= (1 << 20), "T=%d outside [0, %d]", T, 1 << 20);
  MOE_REQUIRE(x_type == MOE_DT_BF16 || x_type == MOE_DT_F16, "x type %d: bf16 or f16", x_type);
  MOE_REQUIRE(y_type == MOE_DT_F32 || y_type == x_type, "y type %d: f32 or the x type", y_type);
  MOE_REQUIRE((flags & ~(MOE_LINEAR_SWIGLU | MOE_LINEAR_ACCUMULATE)) == 0, "flags %d", flags);
  const bool swiglu = (flags & MOE_LINEAR_SWIGLU) != 0;
  MOE_REQUIRE(!swiglu || s.N % 2 == 0, "SwiGLU needs an even N, got %d", s.N);
  if (T == 0) return MOE_OK;
  MOE_REQUIRE(codes && scales && x && y, "null pointer");
  MOE_REQUIRE(aligned(codes, 16) && aligned(x, 16), "codes and x must be 16-byte aligned");
  const int ssize = !int4 ? 1 : s.scale_type == MOE_DT_F32 ? 4 : 2;
  MOE_REQUIRE(aligned(scales, ssize) && aligned(y, y_type == MOE_DT_F32 ? 4 : 2), "misaligned pointer");
  MOE_REQUIRE(ldx >= s.K && ldx % 8 == 0, "ldx=%lld: at least K, a multiple of 8", static_cast<long long>(ldx));
  MOE_REQUIRE(ldy >= (swiglu ? s.N / 2 : s.N), "ldy=%lld is shorter than a row", static_cast<long long>(ldy));
  DeviceInfo dev;
  const moe_status st = current_device(&dev);
  if (st != MOE_OK) return st;
  LinearParams P{};
  P.codes = static_cast<const uint8_t*>(codes);
  P.scales = scales;
  P.zeros = zeros;
  P.x = x;
  P.y = y;
  P.ldx = ldx;
  P.ldy = ldy;
  P.N = s.N;
  P.K = s.K;
  P.T = T;
  P.groups = (s.K + s.group - 1) / s.group;
  P.scale_type = s.scale_type;
  P.y_f32 = y_type == MOE_DT_F32;
  P.swiglu = swiglu;
  P.accumulate = (flags & MOE_LINEAR_ACCUMULATE) != 0;
  P.tensor_scale = tensor_scale;
  const bool bf16 = x_type == MOE_DT_BF16;
  const bool tc = use_tc(P, s.fmt, s.group, dev);
  const cudaError_t e = tc ? (int4 ? launch_linear_tc_int4(P, s.group, bf16, dev, dev_status, stream)
                                   : launch_linear_tc_fp4(P, s.fmt, bf16, dev, dev_status, stream))
                           : (int4 ? launch_linear_int4(P, s.group, bf16, dev, stream)
                                   : launch_linear_fp4(P, s.fmt, bf16, dev, stream));
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "linear_w4 launch: %s", cudaGetErrorString(e));
  return MOE_OK;
}
