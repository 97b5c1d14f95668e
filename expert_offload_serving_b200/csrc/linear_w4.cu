// Dense 4-bit linear: y[t][n] = sum_k w[n][k] x[t][k], w from 4-bit codes and a
// scale per group of K.
//
// One warp multiplies 16 rows of W by 8 * NT tokens with mma.sync (m16n8k16,
// fp32 accumulators).  The codes arrive through a private ring of cp.async
// stages; a thread turns 8 codes of a row (one 32-bit word) into two operand
// pairs a piece, in the x type, exactly:
//   INT4   code - zero            an integer of at most 4 bits
//   MXFP4  the E2M1 value          2 significant bits
//   NVFP4  E2M1 * E4M3 block scale 6 significant bits
// INT4 and MXFP4 scales multiply the fp32 sum of their group, so every product
// is exact and only the fp32 sums round.
//
// K order.  A word holds the codes k = 8j .. 8j+7 with k + i in nibble i, and
// masking a 16-bit half's nibble yields the pair (k+i, k+i+4).  The MMA's k
// slots may hold any 16 elements as long as both operands agree, so x is
// permuted the same way: the four pairs (0,4), (1,5), (2,6), (3,7) of a thread's
// 8 elements are the operand registers of two MMAs (32 elements of K).
//
// The CTA's warps split K and add their sums through shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kRows = 16;             // rows of W per warp tile
constexpr int kStageK = 256;          // codes of a row per stage
constexpr int kPitch = 144;           // bytes of a row in a stage: 128 + 16, so that 8 rows x 4 words hit 32 banks
constexpr int kStages = 3;
constexpr int kStageBytes = kRows * kPitch;
constexpr int kUnit = 128;            // K is split between warps in units of the largest group

struct LinearParams {
  const uint8_t* codes;
  const void* scales;
  const uint8_t* zeros;
  const void* x;
  void* y;
  int64_t ldx, ldy;
  int N, K, T, groups, scale_type, y_f32, swiglu, accumulate;
  float tensor_scale;
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool BF16>
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
  if constexpr (BF16) {
    const __nv_bfloat162 r = __hsub2(reinterpret_cast<__nv_bfloat162&>(a), reinterpret_cast<__nv_bfloat162&>(b));
    return reinterpret_cast<const uint32_t&>(r);
  } else {
    const __half2 r = __hsub2(reinterpret_cast<__half2&>(a), reinterpret_cast<__half2&>(b));
    return reinterpret_cast<const uint32_t&>(r);
  }
}
template <bool BF16>
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  if constexpr (BF16) {
    const __nv_bfloat162 r = __hmul2(reinterpret_cast<__nv_bfloat162&>(a), reinterpret_cast<__nv_bfloat162&>(b));
    return reinterpret_cast<const uint32_t&>(r);
  } else {
    const __half2 r = __hmul2(reinterpret_cast<__half2&>(a), reinterpret_cast<__half2&>(b));
    return reinterpret_cast<const uint32_t&>(r);
  }
}

// The pair (code i, code i + 4) of a word as two exact values.  INT4: `c` holds
// the pair (M + zero, M + zero) with M = 128 (bf16) or 1024 (f16), at which the
// type's step is 1, and a code is OR-ed into M's low bits.  E2M1: sign and
// (exponent, mantissa) go to their places in the x type; as the format's
// subnormals are the type's, the bits read as a number are the value times a
// fixed power of two, which `c` (a multiplier) takes back, with the block scale
// where there is one.
template <int FMT, bool BF16, int I>
__device__ __forceinline__ uint32_t pair_of(uint32_t w, uint32_t c) {
  if constexpr (FMT == MOE_W_INT4) {
    constexpr uint32_t M = BF16 ? 0x43004300u : 0x64006400u;
    return sub2<BF16>(((w >> (4 * I)) & 0x000F000Fu) | M, c);
  } else {
    constexpr int SIGN = 12 - 4 * I;                       // left shift that takes bit 4I+3 to bit 15
    constexpr int MAG = (BF16 ? 6 : 9) - 4 * I;            // left shift that takes bit 4I to the mantissa's top bit
    constexpr uint32_t MASK = BF16 ? 0x01C001C0u : 0x0E000E00u;
    const uint32_t s = (w << SIGN) & 0x80008000u;
    const uint32_t m = (MAG >= 0 ? w << (MAG >= 0 ? MAG : 0) : w >> (MAG < 0 ? -MAG : 0)) & MASK;
    return mul2<BF16>(s | m, c);
  }
}

__device__ __forceinline__ float scale_value(const void* p, size_t i, int type) {
  if (type == MOE_DT_F32) return __ldg(static_cast<const float*>(p) + i);
  const uint16_t b = __ldg(static_cast<const uint16_t*>(p) + i);
  return type == MOE_DT_BF16 ? __uint_as_float(static_cast<uint32_t>(b) << 16) : __half2float(__ushort_as_half(b));
}

// E8M0: 2^(b - 127); 0 is a subnormal of fp32, 255 is NaN.
__device__ __forceinline__ float e8m0_value(uint8_t b) {
  return __uint_as_float(b == 255 ? 0x7FC00000u : (b == 0 ? 0x00400000u : static_cast<uint32_t>(b) << 23));
}

// E4M3 block scale as a multiplier of the raw E2M1 pair (exact: 4 significant
// bits).  bf16: raw is the value * 2^-126; the multiplier brings 2^110 of it
// back and the epilogue the rest, since scale * 2^126 can overflow.
template <bool BF16>
__device__ __forceinline__ uint32_t e4m3_mult(uint8_t b) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(b, __NV_E4M3);
  if constexpr (BF16) {
    const float f = __half2float(__half(h)) * 1.298074214633707e33f;   // 2^110
    const uint32_t u = __float_as_uint(f) >> 16;
    return u | (u << 16);
  } else {
    const uint32_t u = __half_as_ushort(__half(h));
    return u | (u << 16);
  }
}
constexpr float kNvBackBf16 = 65536.f;      // 2^16
constexpr float kNvBackF16 = 16384.f;       // 2^14: raw f16 pairs are the value * 2^-14

// ROW of W held by tile row r (0..15) of tile `tile`: with SwiGLU rows 0-7 are
// gate rows and 8-15 the up rows of the same outputs.
__device__ __forceinline__ int weight_row(const LinearParams& P, int tile, int r) {
  const int half = P.N >> 1;
  if (P.swiglu) {
    const int i = min(tile * 8 + (r & 7), half - 1);
    return r < 8 ? i : half + i;
  }
  return min(tile * kRows + r, P.N - 1);
}

__device__ __forceinline__ void store_y(const LinearParams& P, int BF16x, int t, int n, float v) {
  const int64_t at = static_cast<int64_t>(t) * P.ldy + n;
  if (P.y_f32) {
    float* y = static_cast<float*>(P.y) + at;
    *y = P.accumulate ? *y + v : v;
  } else if (BF16x) {
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(P.y) + at;
    *y = __float2bfloat16_rn(P.accumulate ? __bfloat162float(*y) + v : v);
  } else {
    __half* y = static_cast<__half*>(P.y) + at;
    *y = __float2half_rn(P.accumulate ? __half2float(*y) + v : v);
  }
}

// GB: 32-element blocks per INT4 group (1, 2, 4).
template <int FMT, int GB, bool BF16, int NT>
__global__ void __launch_bounds__(kThreads) linear_w4_kernel(const __grid_constant__ LinearParams P) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
  const int tile = blockIdx.x, tok0 = blockIdx.y * (8 * NT);
  unsigned char* ring = smem + warp * (kStages * kStageBytes);
  const int units = (P.K + kUnit - 1) / kUnit;
  const int k0 = static_cast<int>(static_cast<int64_t>(units) * warp / kWarps) * kUnit;
  const int k1 = min(P.K, static_cast<int>(static_cast<int64_t>(units) * (warp + 1) / kWarps) * kUnit);
  const int nstages = (k1 - k0 + kStageK - 1) / kStageK;

  // this lane's 16-byte chunk of four rows of each stage
  const int ch = lane & 7;
  const uint8_t* src[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    src[i] = P.codes + static_cast<size_t>(weight_row(P, tile, i * 4 + (lane >> 3))) * (P.K / 2) + ch * 16;
  auto issue = [&](int st) {
    if (st < nstages) {
      const int k = k0 + st * kStageK;
      unsigned char* dst = ring + (st % kStages) * kStageBytes + (lane >> 3) * kPitch + ch * 16;
      if (k + ch * 32 < k1)
#pragma unroll
        for (int i = 0; i < 4; ++i) cp_async16(dst + i * 4 * kPitch, src[i] + k / 2);
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);

  const int row0 = weight_row(P, tile, g), row1 = weight_row(P, tile, g + 8);
  const size_t s0 = static_cast<size_t>(row0) * P.groups, s1 = static_cast<size_t>(row1) * P.groups;
  const uint16_t* xrow[NT];
  bool xok[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int t = tok0 + nt * 8 + g;
    xok[nt] = t < P.T;
    xrow[nt] = static_cast<const uint16_t*>(P.x) + static_cast<int64_t>(xok[nt] ? t : 0) * P.ldx + t4 * 8;
  }
  float acc[NT][4], part[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[nt][i] = part[nt][i] = 0.f;

  for (int st = 0; st < nstages; ++st) {
    cp_wait<kStages - 2>();
    __syncwarp();
    issue(st + kStages - 1);
    const unsigned char* sp = ring + (st % kStages) * kStageBytes + g * kPitch + t4 * 4;
    const int kb = k0 + st * kStageK;
    const int blocks = min(kStageK, k1 - kb) / 32;
    for (int b = 0; b < blocks; ++b) {
      const int k = kb + b * 32;
      const uint32_t w0 = *reinterpret_cast<const uint32_t*>(sp + b * 16);
      const uint32_t w1 = *reinterpret_cast<const uint32_t*>(sp + 8 * kPitch + b * 16);
      uint32_t c0, c1;
      float f0 = 1.f, f1 = 1.f;
      if constexpr (FMT == MOE_W_INT4) {
        constexpr uint32_t M = BF16 ? 0x4300u : 0x6400u;
        const int gi = k / (32 * GB);
        c0 = (M | (P.zeros != nullptr ? __ldg(P.zeros + s0 + gi) & 15u : 8u)) * 0x10001u;
        c1 = (M | (P.zeros != nullptr ? __ldg(P.zeros + s1 + gi) & 15u : 8u)) * 0x10001u;
      } else if constexpr (FMT == MOE_W_MXFP4) {
        c0 = c1 = BF16 ? 0x7E807E80u : 0x74007400u;        // 2^126, 2^14
        f0 = e8m0_value(__ldg(static_cast<const uint8_t*>(P.scales) + s0 + k / 32));
        f1 = e8m0_value(__ldg(static_cast<const uint8_t*>(P.scales) + s1 + k / 32));
      } else {
        const int gi = k / 16 + (t4 >> 1);
        c0 = e4m3_mult<BF16>(__ldg(static_cast<const uint8_t*>(P.scales) + s0 + gi));
        c1 = e4m3_mult<BF16>(__ldg(static_cast<const uint8_t*>(P.scales) + s1 + gi));
      }
      const uint32_t a00 = pair_of<FMT, BF16, 0>(w0, c0), a01 = pair_of<FMT, BF16, 1>(w0, c0);
      const uint32_t a02 = pair_of<FMT, BF16, 2>(w0, c0), a03 = pair_of<FMT, BF16, 3>(w0, c0);
      const uint32_t a10 = pair_of<FMT, BF16, 0>(w1, c1), a11 = pair_of<FMT, BF16, 1>(w1, c1);
      const uint32_t a12 = pair_of<FMT, BF16, 2>(w1, c1), a13 = pair_of<FMT, BF16, 3>(w1, c1);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (xok[nt]) v = __ldg(reinterpret_cast<const uint4*>(xrow[nt] + k));
        mma16816<BF16>(part[nt], a00, a10, a01, a11, __byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632));
        mma16816<BF16>(part[nt], a02, a12, a03, a13, __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
      }
      if constexpr (FMT != MOE_W_NVFP4) {
        if (FMT == MOE_W_MXFP4 || GB == 1 || (k / 32 + 1) % GB == 0 || k + 32 >= k1) {
          if constexpr (FMT == MOE_W_INT4) {
            f0 = scale_value(P.scales, s0 + k / (32 * GB), P.scale_type);
            f1 = scale_value(P.scales, s1 + k / (32 * GB), P.scale_type);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            acc[nt][0] = fmaf(part[nt][0], f0, acc[nt][0]);
            acc[nt][1] = fmaf(part[nt][1], f0, acc[nt][1]);
            acc[nt][2] = fmaf(part[nt][2], f1, acc[nt][2]);
            acc[nt][3] = fmaf(part[nt][3], f1, acc[nt][3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) part[nt][i] = 0.f;
          }
        }
      }
    }
    __syncwarp();
  }
  cp_wait<0>();
  if constexpr (FMT == MOE_W_NVFP4) {
    const float back = (BF16 ? kNvBackBf16 : kNvBackF16) * P.tensor_scale;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[nt][i] = part[nt][i] * back;
  }

  // sums of the warps: red[warp][NT * 4][32]
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[(warp * NT * 4 + nt * 4 + i) * 32 + lane] = acc[nt][i];
  __syncthreads();
  for (int nt = warp; nt < NT; nt += kWarps) {
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int w = 0; w < kWarps; ++w)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += red[(w * NT * 4 + nt * 4 + i) * 32 + lane];
    const int t = tok0 + nt * 8 + t4 * 2;
    if (P.swiglu) {
      const int n = tile * 8 + g;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (n < P.N / 2 && t + i < P.T) store_y(P, BF16, t + i, n, v[i] / (1.f + expf(-v[i])) * v[2 + i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = tile * kRows + g + (i >> 1) * 8;
        if (n < P.N && t + (i & 1) < P.T) store_y(P, BF16, t + (i & 1), n, v[i]);
      }
    }
  }
}

template <int FMT, int GB, bool BF16, int NT>
cudaError_t launch_nt(const LinearParams& P, cudaStream_t s) {
  constexpr size_t smem = static_cast<size_t>(kWarps) * kStages * kStageBytes;   // 54 KB
  static_assert(smem >= static_cast<size_t>(kWarps) * NT * 4 * 32 * 4, "the ring holds the warps' sums");
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  auto kern = linear_w4_kernel<FMT, GB, BF16, NT>;
  if (!done[dev & 63]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    done[dev & 63] = true;
  }
  const int per = P.swiglu ? 8 : kRows, rows = P.swiglu ? P.N / 2 : P.N;
  kern<<<dim3((rows + per - 1) / per, (P.T + 8 * NT - 1) / (8 * NT)), kThreads, smem, s>>>(P);
  return cudaGetLastError();
}

template <int FMT, int GB, bool BF16>
cudaError_t launch_type(const LinearParams& P, cudaStream_t s) {
  if (P.T <= 8) return launch_nt<FMT, GB, BF16, 1>(P, s);
  if (P.T <= 16) return launch_nt<FMT, GB, BF16, 2>(P, s);
  return launch_nt<FMT, GB, BF16, 4>(P, s);
}

template <bool BF16>
cudaError_t launch_linear(const LinearParams& P, int fmt, int group, cudaStream_t s) {
  if (fmt == MOE_W_MXFP4) return launch_type<MOE_W_MXFP4, 1, BF16>(P, s);
  if (fmt == MOE_W_NVFP4) return launch_type<MOE_W_NVFP4, 1, BF16>(P, s);
  if (group == 32) return launch_type<MOE_W_INT4, 1, BF16>(P, s);
  if (group == 64) return launch_type<MOE_W_INT4, 2, BF16>(P, s);
  return launch_type<MOE_W_INT4, 4, BF16>(P, s);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_linear_w4(moe_linear_shape s, const void* codes, const void* scales, const uint8_t* zeros,
                                    float tensor_scale, const void* x, int x_type, int64_t ldx, int T, void* y,
                                    int y_type, int64_t ldy, int flags, cudaStream_t stream) {
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
  const cudaError_t e = x_type == MOE_DT_BF16 ? launch_linear<true>(P, s.fmt, s.group, stream)
                                              : launch_linear<false>(P, s.fmt, s.group, stream);
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "linear_w4 launch: %s", cudaGetErrorString(e));
  return MOE_OK;
}
