// Dense 4-bit linear: y[t][n] = sum_k w[n][k] x[t][k], w from 4-bit codes and a
// scale per group of K.  The kernel, instantiated per format in linear_w4_*.cu.
//
// A CTA of 8 warps multiplies M rows of W by a tile of tokens with mma.sync
// (m16n8k16, fp32 accumulators); a warp has 16 * RT rows, 8 * NT tokens and a
// slice of K.  Codes and x arrive in stages of KS elements of K through a
// cp.async ring that all warps share; scales (and zeros) are fetched two stages
// ahead into registers, turned into what the product needs and put into shared
// memory one stage ahead.  One CTA barrier a stage.
//
// A thread turns 8 codes of a row (one 32-bit word) into four operand pairs of
// the x type, exactly:
//   INT4   code - zero             an integer of at most 4 bits
//   MXFP4  the E2M1 value          2 significant bits
//   NVFP4  E2M1 * E4M3 block scale 6 significant bits
// INT4 and MXFP4 scales multiply the fp32 sum of their group (or 32-element
// block), so every product is exact and only fp32 sums round.
//
// K order.  The MMA's k slots may hold any 16 elements as long as both operands
// agree.  A quad's four threads hold 8 consecutive k each, 32 in all: two MMAs.
// Masking the halves of a shifted word yields the pairs (k, k+4), ..., (k+3, k+7)
// and the words of x are permuted alike; where E2M1 converts to f16 by the byte,
// the pairs are (k, k+1), ... and x stays as it is.
//
// What bounds it: few tokens, the latency of a launch and of the one or two stages that
// a CTA then has, none of which is multiplied before it has landed whole
// (T = 1, N = 2048, K = 768: 2.8 us, of which the 0.8 MB take 0.13 at the copy rate;
// T = 1 with N = 4096, K = 4096 of MXFP4, 256 CTAs of two stages: 7.0 us, 1.3 TB/s;
// T = 8, N = 4096, K = 2048 of NVFP4, one stage: 4.9 us); many rows, instructions: 4 to 6 a pair of weights at two a
// clock for an SM (T = 4, N = 131072, K = 4096, INT4 by 128: 92 us, 3.0 TB/s).  K is
// split over warps rather than CTAs (their sums meet in shared memory, one launch);
// 8 warps of 16 rows, two CTAs an SM, gave the shortest chain.
//
// Rows in shared memory: the CTA's M rows in order, or with SwiGLU M/2 gate rows
// and then the M/2 up rows of the same outputs.  A 16-row MMA tile takes 8 of
// each, so that a thread's accumulators hold h and u of one output.
#pragma once

#include <atomic>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace moe {

struct LinearParams {
  const uint8_t* codes;
  const void* scales;
  const uint8_t* zeros;
  const void* x;
  void* y;
  int64_t ldx, ldy;
  int N, K, T, groups, scale_type, y_f32, swiglu, accumulate;
  float tensor_scale;
  // launch shape
  int wm_bits;             // warps along the rows (log2); the warps left over split K
  int stages, ring;        // stages in flight + 1; slots (no more than there are stages)
  int x_rows;              // token rows a stage holds
  int scale_vec;           // rows of scales (and zeros) are aligned for loads of several groups
};

// Whether the tcgen05 kernels multiply the groups' sums by the scales (see
// linear_w4_tc.cuh) rather than the weights.
inline bool scales_outside(const LinearParams& P, int fmt, bool bf16) {
  return bf16 ? fmt == MOE_W_INT4 && P.scale_type == MOE_DT_F32 && P.y_f32 : fmt != MOE_W_NVFP4;
}

// Launchers, one per format family (linear_w4_int4.cu, linear_w4_fp4.cu).
cudaError_t launch_linear_int4(const LinearParams& P, int group, bool bf16, const DeviceInfo& dev, cudaStream_t s);
cudaError_t launch_linear_fp4(const LinearParams& P, int fmt, bool bf16, const DeviceInfo& dev, cudaStream_t s);
// The same on the 5th-generation tensor cores (linear_w4_tc_*.cu).
cudaError_t launch_linear_tc_int4(const LinearParams& P, int group, bool bf16, const DeviceInfo& dev, int32_t* status,
                                  cudaStream_t s);
cudaError_t launch_linear_tc_fp4(const LinearParams& P, int fmt, bool bf16, const DeviceInfo& dev, int32_t* status,
                                 cudaStream_t s);

namespace w4 {

constexpr int kThreads = 256;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most n groups are in flight (n is the same for every thread).
__device__ __forceinline__ void cp_wait(int n) {
  switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
  }
}
constexpr int kMaxStages = 5;

template <typename V>
__device__ __forceinline__ V lds(const unsigned char* smem, uint32_t at) {
  return *reinterpret_cast<const V*>(smem + at);
}

// c = a b (+ c)
template <bool BF16, bool ZERO>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
#define MOE_MMA(TYPE)                                                                                               \
  if constexpr (ZERO)                                                                                               \
    asm("mma.sync.aligned.m16n8k16.row.col.f32." TYPE "." TYPE                                             \
                 ".f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"                                   \
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])                                                   \
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));                                 \
  else                                                                                                              \
    asm("mma.sync.aligned.m16n8k16.row.col.f32." TYPE "." TYPE                                             \
                 ".f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"                                       \
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])                                                   \
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  if constexpr (BF16) {
    MOE_MMA("bf16")
  } else {
    MOE_MMA("f16")
  }
#undef MOE_MMA
}

template <bool BF16>
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (BF16) asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (BF16) asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// (a & b) | c, with the constants in registers: one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// Pair I (0..3) of a word as two exact values of the x type.
//   INT4: `c` holds (M + zero, M + zero) with M = 128 (bf16) or 1024 (f16), where
//   the type's step is 1, and a code is OR-ed into M's low bits.
//   E2M1, f16: converted by the byte.
//   E2M1, bf16: sign and (exponent, mantissa) move to their places; the format's
//   subnormals are the type's, so the bits read as the value * 2^-126, which `c`
//   takes back (in part, where it multiplies with NVFP4's block scale: kNvBack).
template <int FMT, bool BF16, int I>
__device__ __forceinline__ uint32_t pair_of(uint32_t w, uint32_t c) {
  if constexpr (FMT == MOE_W_INT4) {
    return sub2<BF16>(and_or(w >> (4 * I), 0x000F000Fu, BF16 ? 0x43004300u : 0x64006400u), c);
  } else if constexpr (BF16) {
    const uint32_t sign = w << (12 - 4 * I);
    const uint32_t mag = (I < 2 ? w << (I < 2 ? 6 - 4 * I : 0) : w >> (I < 2 ? 0 : 4 * I - 6)) & 0x01C001C0u;
    return mul2<true>(and_or(sign, 0x80008000u, mag), c);
  } else {
    uint32_t h;
    asm("{ .reg .b8 b; cvt.u8.u32 b, %1; cvt.rn.f16x2.e2m1x2 %0, b; }" : "=r"(h) : "r"(w >> (8 * I)));
    return FMT == MOE_W_NVFP4 ? mul2<false>(h, c) : h;
  }
}
constexpr uint32_t kMxBack = 0x7E807E80u;     // 2^126 twice
// 2^119 and 2^7: a scale of up to 448 times 2^126 overflows.  (The sums are 2^-7 of
// their value until the end, so 7 bits are lost below fp32's normal range, no more.)
constexpr float kNvPart = 6.646139978924579e35f, kNvBack = 128.f;

// E8M0: 2^(b - 127); 0 is a subnormal of fp32, 255 is NaN.
__device__ __forceinline__ float e8m0_value(uint32_t b) {
  return __uint_as_float(b == 255 ? 0x7FC00000u : (b == 0 ? 0x00400000u : b << 23));
}

// E4M3 block scale as the multiplier `c` of pair_of (4 significant bits: exact).
template <bool BF16>
__device__ __forceinline__ uint32_t e4m3_mult(uint32_t b) {
  const __half h = __half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(b), __NV_E4M3));
  uint32_t u;
  if constexpr (BF16) u = __float_as_uint(__half2float(h) * kNvPart) >> 16;
  else u = __half_as_ushort(h);
  return u | (u << 16);
}

template <bool BF16>
__device__ __forceinline__ void store_y(const LinearParams& P, int t, int n, float v) {
  const int64_t at = static_cast<int64_t>(t) * P.ldy + n;
  if (P.y_f32) {
    float* y = static_cast<float*>(P.y) + at;
    *y = P.accumulate ? *y + v : v;
  } else if (BF16) {
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(P.y) + at;
    *y = __float2bfloat16_rn(P.accumulate ? __bfloat162float(*y) + v : v);
  } else {
    __half* y = static_cast<__half*>(P.y) + at;
    *y = __float2half_rn(P.accumulate ? __half2float(*y) + v : v);
  }
}

// GROUP: elements of K per scale; NT, RT: 8-token and 16-row tiles of a warp.
template <int FMT, int GROUP, bool BF16, int NT, int RT>
struct Geometry {
  static constexpr int KW = 256;                                        // K a warp takes from a stage
  static constexpr int STAGE_WEIGHTS = 8 * 16 * RT * KW;
  static constexpr int EPT = STAGE_WEIGHTS / GROUP / kThreads;          // scales a thread fetches per stage
  static constexpr int CPT = STAGE_WEIGHTS / 32 / kThreads;             // 16-byte chunks of codes a thread copies
  static constexpr int ENTRY = FMT == MOE_W_INT4 ? 8 : 4;               // bytes of a scale in shared memory
  // a 16-bit INT4 scale or a scale byte in global memory; EPT of them, EPT zeros
  using Elem = typename std::conditional<FMT == MOE_W_INT4, uint16_t, uint8_t>::type;
  static constexpr int VB = EPT * sizeof(Elem);
  template <int B>
  using Bytes = typename std::conditional<
      B == 1, uint8_t,
      typename std::conditional<
          B == 2, uint16_t,
          typename std::conditional<B == 4, uint32_t,
                                    typename std::conditional<B == 8, uint2, uint4>::type>::type>::type>::type;
  using Vec = Bytes<VB>;
  using ZVec = Bytes<EPT>;
  static_assert(VB <= 16, "one load");
  static_assert(CPT >= 2, "a thread copies rows of both parts");
  int wk, ks, m, gps, cpitch, xpitch, spitch, stage, sbuf, zero_at, s_at, bytes;
  // wk: warps along K; ks: K per stage; m: rows; gps: groups of a row per stage;
  // pitches: bytes of a row of codes (conflict-free 4-byte reads of 8 rows), of x
  // (16-byte reads of 2 rows) and of scales (8 rows apart, 16-byte writes)
  static constexpr int TOKENS = 8 * NT;
  __host__ __device__ explicit Geometry(const LinearParams& P) {
    wk = 8 >> P.wm_bits;
    ks = KW * wk;
    m = 16 * RT << P.wm_bits;
    gps = ks / GROUP;
    cpitch = ks / 2 + 16;
    xpitch = ks * 2 + 64;
    spitch = gps * ENTRY + 16;
    stage = m * cpitch + P.x_rows * xpitch;
    sbuf = (m * spitch + 15) / 16 * 16;
    zero_at = P.ring * stage;                 // one row of zeros for the tokens that are not there
    s_at = zero_at + xpitch;
    bytes = s_at + 2 * sbuf;
  }
};

template <int FMT, int GROUP, bool BF16, int NT, int RT>
__global__ void __launch_bounds__(kThreads, 2) linear_w4_kernel(const __grid_constant__ LinearParams P) {
  using G = Geometry<FMT, GROUP, BF16, NT, RT>;
  constexpr int KW = G::KW, KB = KW / 32, GB = GROUP >= 32 ? GROUP / 32 : 1;
  constexpr bool PERMUTE = FMT == MOE_W_INT4 || BF16;                // x pairs (k, k+4): see pair_of
  extern __shared__ __align__(16) unsigned char smem[];
  const G geo(P);
  const uint32_t sm = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const int wm = warp & ((1 << P.wm_bits) - 1), wk = warp >> P.wm_bits;
  const int tok0 = blockIdx.y * G::TOKENS;
  const int x_rows = min(P.x_rows, P.T - tok0);
  const int nst = (P.K + geo.ks - 1) / geo.ks;
  // Row r of shared memory is row first + r of W for r below `split`, else row
  // up + r - split (SwiGLU); rows from `valid` of each part on are not there.
  const int split = P.swiglu ? geo.m / 2 : geo.m, outs = P.swiglu ? P.N >> 1 : P.N;
  const int first = blockIdx.x * split, valid = min(split, outs - first);
  pdl_wait();
  pdl_trigger();

  // A thread's rows of a kind (codes, scales) are r0, r0 + step, ... ; n of them
  // in all.  The first half of them lies in the first part, the second half in
  // the second one (a single row lies where it does).
  auto row_of = [&](int r) { return r < split || !P.swiglu ? first + r : outs + first + r - split; };
  auto there = [&](int r) { return (r < split || !P.swiglu ? r : r - split) < valid; };

  // A stage's copies: thread -> 16-byte chunk `col` of every code_rows-th row (a
  // row of codes has a power of two <= 64 chunks, a row of x four times as many).
  const int cpr_bits = 31 - __clz(geo.ks / 32), col = tid & ((1 << cpr_bits) - 1);
  const int code_rows = kThreads >> cpr_bits, code_r = tid >> cpr_bits;
  const uint8_t* csrc[2];
  unsigned cok = 0;                                                  // which rows are there
#pragma unroll
  for (int i = 0; i < G::CPT; ++i) cok |= there(i * code_rows + code_r) << i;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    csrc[h] = P.codes + static_cast<size_t>(row_of(h * (G::CPT / 2) * code_rows + code_r)) * (P.K >> 1) + col * 16;
  const size_t cstep = static_cast<size_t>(code_rows) * (P.K >> 1);
  const int xpr_bits = cpr_bits + 2, xcol = tid & ((1 << xpr_bits) - 1);
  const int xrow_step = kThreads >> xpr_bits, xr0 = tid >> xpr_bits;
  const uint16_t* xsrc = static_cast<const uint16_t*>(P.x) + static_cast<int64_t>(tok0 + xr0) * P.ldx + xcol * 8;
  const int64_t xstep = xrow_step * P.ldx;
  const uint32_t cdst = sm + code_r * geo.cpitch + col * 16, cdstep = code_rows * geo.cpitch;
  const uint32_t xdst = sm + geo.m * geo.cpitch + xr0 * geo.xpitch + xcol * 16, xdstep = xrow_step * geo.xpitch;
  int slot_in = 0;                                                   // slot of the next stage to issue
  auto issue = [&](int st) {
    if (st < nst) {
      const int k0 = st * geo.ks;
      const uint32_t at = slot_in * geo.stage;
      // behind K zeros are written and nothing is read (from the row's start)
      const bool ok = k0 + col * 32 < P.K, xok = k0 + xcol * 8 < P.K;
      const int64_t off = ok ? k0 >> 1 : -col * 16;
#pragma unroll
      for (int i = 0; i < G::CPT; ++i)
        if (cok >> i & 1) cp_async16(cdst + at + i * cdstep, csrc[2 * i / G::CPT] + off + i % (G::CPT / 2) * cstep, ok);
      const uint16_t* xp = xsrc + (xok ? k0 : -xcol * 8);
      uint32_t xd = xdst + at;
      for (int r = xr0; r < x_rows; r += xrow_step, xp += xstep, xd += xdstep) cp_async16(xd, xp, xok);
      slot_in = slot_in + 1 == P.ring ? 0 : slot_in + 1;
    }
    cp_commit();
  };
  for (int i = 0; i < P.stages - 1; ++i) issue(i);

  // Scales of a stage: a thread takes EPT consecutive groups of one row, in one
  // load where rows are aligned for that (P.scale_vec), as raw values in registers.
  using E = typename G::Elem;
  const int tpr_bits = 31 - __clz(geo.gps / G::EPT);                 // threads of a row
  const int s_r = tid >> tpr_bits, sg = (tid & ((1 << tpr_bits) - 1)) * G::EPT;
  const bool s_ok = there(s_r);
  const size_t ssrc = static_cast<size_t>(row_of(s_r)) * P.groups + sg;
  uint32_t sraw[G::EPT], zraw[G::EPT];
  auto fetch = [&](int st) {
    const int j = st * geo.gps + sg;                                 // first group
    const size_t at = ssrc + st * geo.gps;
#pragma unroll
    for (int i = 0; i < G::EPT; ++i) {
      sraw[i] = 0;
      zraw[i] = 8;
    }
    if (!s_ok || j >= P.groups) return;
    if (P.scale_vec && j + G::EPT <= P.groups) {
      if (FMT == MOE_W_INT4 && P.scale_type == MOE_DT_F32) {
#pragma unroll
        for (int i = 0; i < G::EPT; ++i) sraw[i] = __ldg(static_cast<const uint32_t*>(P.scales) + at + i);
      } else {
        union { typename G::Vec v; E e[G::EPT]; } u;
        u.v = __ldg(reinterpret_cast<const typename G::Vec*>(static_cast<const E*>(P.scales) + at));
#pragma unroll
        for (int i = 0; i < G::EPT; ++i) sraw[i] = FMT == MOE_W_INT4 ? u.e[i] : 0x100u | u.e[i];   // 0x100: there is one
      }
      if (FMT == MOE_W_INT4 && P.zeros != nullptr) {
        union { typename G::ZVec v; uint8_t e[G::EPT]; } u;
        u.v = __ldg(reinterpret_cast<const typename G::ZVec*>(P.zeros + at));
#pragma unroll
        for (int i = 0; i < G::EPT; ++i) zraw[i] = u.e[i] & 15u;
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < G::EPT; ++i) {
      if (j + i >= P.groups) break;
      if constexpr (FMT == MOE_W_INT4) {
        sraw[i] = P.scale_type == MOE_DT_F32 ? __ldg(static_cast<const uint32_t*>(P.scales) + at + i)
                                             : __ldg(static_cast<const uint16_t*>(P.scales) + at + i);
        if (P.zeros != nullptr) zraw[i] = __ldg(P.zeros + at + i) & 15u;
      } else {
        sraw[i] = 0x100u | __ldg(static_cast<const uint8_t*>(P.scales) + at + i);
      }
    }
  };
  unsigned char* const sdst = smem + geo.s_at + s_r * geo.spitch + sg * G::ENTRY;
  auto put = [&](int st) {
    uint32_t v[G::EPT * G::ENTRY / 4];
#pragma unroll
    for (int i = 0; i < G::EPT; ++i) {
      if constexpr (FMT == MOE_W_INT4) {
        v[2 * i] = P.scale_type == MOE_DT_F32    ? sraw[i]
                   : P.scale_type == MOE_DT_BF16 ? sraw[i] << 16
                                                 : __float_as_uint(__half2float(__ushort_as_half(sraw[i])));
        v[2 * i + 1] = ((BF16 ? 0x4300u : 0x6400u) | zraw[i]) * 0x10001u;
      } else if constexpr (FMT == MOE_W_MXFP4) {
        v[i] = sraw[i] == 0 ? 0u : __float_as_uint(e8m0_value(sraw[i] & 255u));
      } else {
        v[i] = sraw[i] == 0 ? 0u : e4m3_mult<BF16>(sraw[i] & 255u);
      }
    }
    unsigned char* d = sdst + (st & 1) * geo.sbuf;
    if constexpr (G::EPT * G::ENTRY == 8) {
      *reinterpret_cast<uint2*>(d) = make_uint2(v[0], v[1]);
    } else {
#pragma unroll
      for (int i = 0; i < G::EPT * G::ENTRY / 4; i += 4)
        *reinterpret_cast<uint4*>(d + i * 4) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
  };
  fetch(0);
  for (int c = tid; c < geo.xpitch / 16; c += kThreads)
    *reinterpret_cast<uint4*>(smem + geo.zero_at + c * 16) = make_uint4(0, 0, 0, 0);
  put(0);
  if (nst > 1) fetch(1);

  float acc[RT][NT][4], part[RT][NT][4];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[rt][nt][i] = 0.f;

  // this thread's rows in shared memory: row + rt * rt_step + i * i_step, i = 0, 1
  const int rt_step = P.swiglu ? 8 : 16, i_step = P.swiglu ? split : 8, row = wm * RT * rt_step + g;
  const uint32_t code_at = row * geo.cpitch + wk * (KW / 2) + t4 * 4;
  const uint32_t scale_at = geo.s_at + row * geo.spitch +
                            (wk * (KW / GROUP) + (FMT == MOE_W_NVFP4 ? t4 >> 1 : 0)) * G::ENTRY;
  const uint32_t x_at = geo.m * geo.cpitch + g * geo.xpitch + wk * (KW * 2) + t4 * 16;
  int slot = 0;
  for (int st = 0; st < nst; ++st) {
    cp_wait(P.stages - 2);
    __syncthreads();
    if (st + 1 < nst) put(st + 1);
    if (st + 2 < nst) fetch(st + 2);
    issue(st + P.stages - 1);
    const uint32_t at = slot * geo.stage;
    slot = slot + 1 == P.ring ? 0 : slot + 1;
    if (st * geo.ks + wk * KW >= P.K) continue;                      // this warp's share lies behind K
    const uint32_t ca = at + code_at, sa = scale_at + (st & 1) * geo.sbuf;
    uint32_t xa[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      xa[nt] = nt * 8 + g < x_rows ? at + x_at + nt * 8 * geo.xpitch : geo.zero_at + t4 * 16;
    uint32_t c[2 * RT];
    float f[2 * RT];
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      uint32_t a[RT][2][4];
#pragma unroll
      for (int i = 0; i < 2 * RT; ++i) {
        const int dr = (i / 2) * rt_step + (i % 2) * i_step;
        const uint32_t so = sa + dr * geo.spitch;
        if constexpr (FMT == MOE_W_INT4) {
          if (b % GB == 0) {
            const uint2 v = lds<uint2>(smem, so + (b / GB) * 8);
            f[i] = __uint_as_float(v.x);
            c[i] = v.y;
          }
        } else if constexpr (FMT == MOE_W_MXFP4) {
          f[i] = lds<float>(smem, so + b * 4);
          c[i] = kMxBack;
        } else {
          c[i] = lds<uint32_t>(smem, so + b * 8);
        }
        const uint32_t w = lds<uint32_t>(smem, ca + dr * geo.cpitch + b * 16);
        a[i / 2][i % 2][0] = pair_of<FMT, BF16, 0>(w, c[i]);
        a[i / 2][i % 2][1] = pair_of<FMT, BF16, 1>(w, c[i]);
        a[i / 2][i % 2][2] = pair_of<FMT, BF16, 2>(w, c[i]);
        a[i / 2][i % 2][3] = pair_of<FMT, BF16, 3>(w, c[i]);
      }
      // INT4, MXFP4: the scale multiplies the group's sum.  NVFP4: the stage's sum is
      // added, so that no run of the tensor cores' truncating additions gets long.
      constexpr int RUN = FMT == MOE_W_NVFP4 ? KB : GB;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4 v = lds<uint4>(smem, xa[nt] + b * 64);
        uint32_t x0 = v.x, x1 = v.y, x2 = v.z, x3 = v.w;
        if constexpr (PERMUTE) {
          x0 = __byte_perm(v.x, v.z, 0x5410);
          x1 = __byte_perm(v.x, v.z, 0x7632);
          x2 = __byte_perm(v.y, v.w, 0x5410);
          x3 = __byte_perm(v.y, v.w, 0x7632);
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          float (&d)[4] = part[rt][nt];
          if (b % RUN == 0)
            mma16816<BF16, true>(d, a[rt][0][0], a[rt][1][0], a[rt][0][1], a[rt][1][1], x0, x1);
          else
            mma16816<BF16, false>(d, a[rt][0][0], a[rt][1][0], a[rt][0][1], a[rt][1][1], x0, x1);
          mma16816<BF16, false>(d, a[rt][0][2], a[rt][1][2], a[rt][0][3], a[rt][1][3], x2, x3);
          if ((b + 1) % RUN == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              acc[rt][nt][i] = FMT == MOE_W_NVFP4 ? acc[rt][nt][i] + d[i] : fmaf(d[i], f[2 * rt + i / 2], acc[rt][nt][i]);
          }
        }
      }
    }
  }
  if constexpr (FMT == MOE_W_NVFP4) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[rt][nt][i] *= BF16 ? kNvBack * P.tensor_scale : P.tensor_scale;
  }

  // the warps' sums over K, added in the order of the slices
  if (geo.wk > 1) {
    cp_wait(0);
    __syncthreads();
    float* red = reinterpret_cast<float*>(smem) + lane;
    const int wt = 8 / geo.wk, mine = warp & (wt - 1);               // warps of one slice
    if (wk > 0) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            red[((((wk - 1) * wt + mine) * RT + rt) * NT + nt) * 128 + i * 32] = acc[rt][nt][i];
    }
    __syncthreads();
    if (wk > 0) return;
    for (int w = 0; w < geo.wk - 1; ++w)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[rt][nt][i] += red[(((w * wt + mine) * RT + rt) * NT + nt) * 128 + i * 32];
  }
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int t = tok0 + nt * 8 + t4 * 2, r = row + rt * rt_step;
      const float (&v)[4] = acc[rt][nt];
      if (P.swiglu) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (r < valid && t + i < P.T) store_y<BF16>(P, t + i, first + r, v[i] / (1.f + expf(-v[i])) * v[2 + i]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (r + (i >> 1) * 8 < valid && t + (i & 1) < P.T) store_y<BF16>(P, t + (i & 1), first + r + (i >> 1) * 8, v[i]);
      }
    }
  }
}

constexpr int kSmemMax = 227 * 1024;

template <int FMT, int GROUP, bool BF16, int NT, int RT>
cudaError_t launch(LinearParams P, const DeviceInfo& dev, cudaStream_t s) {
  using G = Geometry<FMT, GROUP, BF16, NT, RT>;
  auto kern = linear_w4_kernel<FMT, GROUP, BF16, NT, RT>;
  static std::atomic<bool> done[64];
  if (!done[dev.id].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess) return e;
    done[dev.id].store(true, std::memory_order_release);
  }
  const int tiles = (P.N + 15) / 16;
  // Rows per CTA: the most that still give the SMs a CTA and a half each.  Fewer
  // rows mean more warps along K and a longer stage of x, so not so few that a
  // stage is longer than K or its x more than twice its codes.
  P.x_rows = P.T < G::TOKENS ? P.T : G::TOKENS;
  P.scale_vec = P.groups % G::EPT == 0 && aligned(P.scales, G::VB) && aligned(P.zeros, G::EPT);
  P.wm_bits = 3;
  while (P.wm_bits > 0 && (tiles / RT >> P.wm_bits) * 2 < dev.sm_count * 3) {
    LinearParams q = P;
    --q.wm_bits;
    q.ring = 2;
    const G geo(q);
    if (geo.ks / 2 >= P.K || P.x_rows * geo.ks * 4 > geo.m * geo.ks * 2 || geo.bytes > kSmemMax) break;
    P.wm_bits = q.wm_bits;
  }
  P.stages = 2;
  P.ring = 1;
  G geo(P);
  const int nst = (P.K + geo.ks - 1) / geo.ks;
  P.ring = nst < 2 ? nst : 2;
  const int per = P.swiglu ? geo.m / 2 : geo.m, outs = P.swiglu ? P.N / 2 : P.N;
  const dim3 grid((outs + per - 1) / per, (P.T + G::TOKENS - 1) / G::TOKENS);
  // As deep a ring as lets two CTAs share an SM, or one where one is all there is.
  const bool two = static_cast<int64_t>(grid.x) * grid.y > dev.sm_count;
  for (int n = 3; n <= kMaxStages && n <= nst + 1; ++n) {
    LinearParams q = P;
    q.stages = n;
    q.ring = nst < n ? nst : n;
    if (G(q).bytes > (two ? kSmemMax / 2 - 1024 : kSmemMax)) break;
    P = q;
  }
  geo = G(P);
  const int red = (geo.wk - 1) * (8 / geo.wk) * RT * NT * 512;       // the warps' sums use the same memory
  const int bytes = geo.bytes > red ? geo.bytes : red;
  const cudaError_t e = launch_pdl(kern, grid, dim3(kThreads), bytes, s, P);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Tokens per warp: NT tiles of 8 (above 32 tokens the grid's second dimension takes
// 32 each).  Up to 16 tokens a warp takes 32 rows (RT = 2) where that leaves every
// SM two CTAs, so that x is read from shared memory and permuted once for two row
// tiles: 20 % fewer instructions, though measured about even (T = 13, N = 128001,
// K = 4096, groups of 64: 155.6 against 155.4 us).
template <int FMT, int GROUP, bool BF16>
cudaError_t launch_tokens(const LinearParams& P, const DeviceInfo& dev, cudaStream_t s) {
  const bool wide = P.N >= 64 * dev.sm_count;
  if (P.T <= 8) return wide ? launch<FMT, GROUP, BF16, 1, 2>(P, dev, s) : launch<FMT, GROUP, BF16, 1, 1>(P, dev, s);
  if (P.T <= 16) return wide ? launch<FMT, GROUP, BF16, 2, 2>(P, dev, s) : launch<FMT, GROUP, BF16, 2, 1>(P, dev, s);
  return launch<FMT, GROUP, BF16, 4, 1>(P, dev, s);
}

}  // namespace w4
}  // namespace moe
