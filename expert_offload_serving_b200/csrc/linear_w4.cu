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
// for it.  Groups of 32 whose sums are scaled (f16 x; fp32 scales with an fp32 y) have
// four hand-overs a stage, which 32 tokens do not pay for either.  Device time in us,
// warp / tcgen05, fp32 y, K = 4096 (weights of N <= 16384 in L2):
//   bf16 x               INT4/128      INT4/32       MXFP4         NVFP4         f16 x: INT4/32
//   T = 8   N = 16384   14.5 / 17.8   22.7 / 25.7   24.3 / 26.4   22.9 / 25.5   22.7 / 44.5
//   T = 16  N = 4096     9.0 / 17.6   10.9 / 10.6   10.8 / 26.0   10.0 / 10.1   10.8 / 15.5
//           N = 16384   22.9 / 18.0   28.0 / 25.7   29.7 / 26.4   28.0 / 24.9   28.0 / 43.9
//           N = 131072   146 / 114     193 / 167     195 / 170     192 / 162     193 / 304
//   T = 17  N = 1024    17.5 /  7.5   21.1 /  7.8   21.8 /  7.6   19.0 /  7.4
//           N = 4096    17.5 / 10.0   21.1 / 10.6   21.9 / 10.1   19.3 / 10.1   21.3 / 15.4
//           N = 16384   26.9 / 22.7   30.7 / 25.5   32.2 / 24.7   30.4 / 24.8   30.5 / 43.9
//           N = 131072   168 / 144     265 / 167     211 / 158     192 / 162     266 / 303
//   T = 64  N = 16384   52.4 / 26.2   84.4 / 31.4   85.9 / 26.3   76.4 / 26.1    ..  / 60.5
//   T = 512 N = 4096    91.0 / 37.4    148 / 42.6    151 / 30.9    133 / 31.4
// MOE_LINEAR=warp|tc, read at every call, forces one.
bool use_tc(const LinearParams& P, int fmt, int group, bool bf16, const DeviceInfo& dev) {
  const char* force = getenv("MOE_LINEAR");
  if (force != nullptr) return strcmp(force, "tc") == 0;
  const bool fills = P.N >= 77 * dev.sm_count;                 // 0.6 tiles of 128 rows for each SM
  const bool sums32 = scales_outside(P, fmt, bf16) && group == 32 &&
                      !(fmt == MOE_W_MXFP4 && P.T <= 16);      // (those have a kernel)
  if (P.T > 16) return !(sums32 && fills && P.T <= 32);
  return P.T > 8 && fills && !sums32;
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
  const bool tc = use_tc(P, s.fmt, s.group, bf16, dev);
  const cudaError_t e = tc ? (int4 ? launch_linear_tc_int4(P, s.group, bf16, dev, dev_status, stream)
                                   : launch_linear_tc_fp4(P, s.fmt, bf16, dev, dev_status, stream))
                           : (int4 ? launch_linear_int4(P, s.group, bf16, dev, stream)
                                   : launch_linear_fp4(P, s.fmt, bf16, dev, stream));
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "linear_w4 launch: %s", cudaGetErrorString(e));
  return MOE_OK;
}
