// The dense 4-bit linear on the 5th-generation tensor cores for up to 16 tokens
// and many rows, INT4 (groups of 64 or 128) and MXFP4.
//
// As linear_w4_tc.cuh, cut for a narrow product.  With 16 columns the MMAs take
// next to no time, and what counts is instructions per weight and hand-overs per
// stage: a stage holds 256 elements of K (16 KB of codes, rows of 128 bytes), a
// thread expands 128 codes of its row at once, and INT4 and MXFP4 scales multiply
// the groups' fp32 sums whatever the x type (POST), so that a weight costs one
// subtraction.  A stage's groups have an accumulator each and one hand-over
// together.  Adding up, a quarter of the warps takes a quarter of the groups (or
// half the tokens of one of two groups); the quarters' sums meet in shared memory
// at the end of a tile.
//
// Measured: T = 13, N = 128001, K = 4096, INT4 by 64, f16: 117 us, 2.4 TB/s, against
// 156 on the warp-level kernel.  Bound by the expanding instructions and the
// hand-overs of a stage (2080 cycles a 256 of K; its codes alone would take 800 at
// the copy rate).
//
// Warps 0-15: workers; quadrant (TMEM lanes) = warp % 4; warps 0-7 expand the even
// stages and 8-15 the odd ones, four warps a half of a stage's K.  Warp 16: TMA of
// the codes, 17: of the token rows.  Warps 18, 19: MMAs of the even and odd stages.
#pragma once

#include "linear_w4_tc.cuh"

namespace moe {
namespace w4t16 {

using namespace ::moe::tc;
using w4tc::kSet;
using w4tc::kThreads;
using w4tc::kWorkers;
using w4tc::TcParams;
using w4tc::TM;
using w4tc::wait_on;

constexpr int KS = 256, NT = 16;
constexpr int kCodeBytes = TM * KS / 2;
constexpr int kACols = KS / 2;                // TMEM columns of a set's A buffer
constexpr int kXAtom = NT * 128;              // 64 elements of the token rows

template <int FMT, int GROUP>
struct Cfg {
  static_assert(FMT == MOE_W_INT4 || FMT == MOE_W_MXFP4, "scales of groups");
  static constexpr int GPS = KS / GROUP;                               // groups of a stage: 2, 4, 8
  static constexpr int DCOLS = GPS * NT;                               // TMEM columns of its accumulators
  static constexpr int ND = (512 - 2 * kACols) / 2 / DCOLS < 2 ? 1 : 2;   // ... that a set has
  static constexpr int TOKENS = GPS == 2 ? 8 : 16;                     // tokens a thread adds up
  static constexpr int MINE = GPS <= 4 ? 1 : GPS / 4;                  // groups of a stage that it takes
  static constexpr int STAGE = kCodeBytes + 4 * kXAtom;
  static constexpr int S = 7;
  static constexpr int RED = 4 * TM * (TOKENS + 1) * 4;                // the quarters' sums
  static constexpr int N_BARS = 2 * S + 4 + 4 * ND + 2 + 2 + 1;
  static constexpr int BAR_BYTES = (N_BARS * 8 + 16 + 127) / 128 * 128;
  static constexpr int SMEM = 1024 + S * STAGE + RED + BAR_BYTES;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(2 * kACols + 2 * ND * DCOLS <= 512, "tensor memory");
};

template <int FMT, int GROUP, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    linear_w4_tc16_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                          const __grid_constant__ TcParams Q) {
  using C = Cfg<FMT, GROUP>;
  const LinearParams& P = Q.L;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* red = reinterpret_cast<float*>(smem + C::S * C::STAGE);       // [4][TM][TOKENS + 1]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::S * C::STAGE + C::RED);
  uint64_t* full = bars;                      // [S] a stage's codes and token rows landed
  uint64_t* empty = bars + C::S;              // [S] ... read by the workers and the MMAs
  uint64_t* afull = bars + 2 * C::S;          // [2] expanded weights written
  uint64_t* aempty = afull + 2;               // [2] ... and used
  uint64_t* dfull = aempty + 2;               // [2][ND] a stage's accumulators complete
  uint64_t* dempty = dfull + 2 * C::ND;       // [2][ND] ... and read
  uint64_t* drain = dempty + 2 * C::ND;       // [2]
  uint64_t* rfull = drain + 2;                // the quarters' sums written
  uint64_t* rempty = rfull + 1;               // ... and read
  uint64_t* stall = rempty + 1;               // never arrived on (testing aid)
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + C::N_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nst = (P.K + KS - 1) / KS;
  const int outs = P.swiglu ? P.N >> 1 : P.N, per = P.swiglu ? TM / 2 : TM;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::S; ++s) {
      mbar_init(&full[s], 2);
      mbar_init(&empty[s], kSet + 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&afull[i], kSet);
      mbar_init(&aempty[i], 1);
      mbar_init(&drain[i], 1);
    }
    for (int i = 0; i < 2 * C::ND; ++i) {
      mbar_init(&dfull[i], 1);
      mbar_init(&dempty[i], kWorkers);
    }
    mbar_init(rfull, kWorkers);
    mbar_init(rempty, kWorkers);
    mbar_init(stall, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWorkers + 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                 "n"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder, tmem_d = tmem + 2 * kACols;
  pdl_wait();
  pdl_trigger();

  if (warp == kWorkers || warp == kWorkers + 1) {
    // ------------------------------------------------------------ TMA
    const bool codes = warp == kWorkers;
    if (lane == 0) {
      const uint64_t pol = codes ? policy_evict_first() : policy_evict_last();
      int slot = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < Q.mt && ok; tile += gridDim.x) {
        const int m = tile * per;
        for (int s = 0; s < nst; ++s) {
          if (!wait_on(&empty[slot], phase ^ 1u, abort_flag, Q.wait_ns)) {
            ok = false;
            break;
          }
          uint8_t* at = smem + slot * C::STAGE;
          if (codes) {
            mbar_expect_tx(&full[slot], kCodeBytes);
            tma_load_2d(at, &tm_w, &full[slot], s * (KS / 2), m, pol);
            if (P.swiglu) tma_load_2d(at + kCodeBytes / 2, &tm_w, &full[slot], s * (KS / 2), outs + m, pol);
          } else {
            mbar_expect_tx(&full[slot], 4 * kXAtom);
#pragma unroll
            for (int a = 0; a < 4; ++a)
              tma_load_2d(at + kCodeBytes + a * kXAtom, &tm_x, &full[slot], s * KS + a * 64, 0, pol);
          }
          ++issued;
          if (++slot == C::S) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        report(Q.status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      // what was issued has landed before the CTA leaves (see linear_w4_tc.cuh)
      for (int i = issued < C::S ? issued : C::S; i > 0; --i) {
        if (--slot < 0) {
          slot = C::S - 1;
          phase ^= 1u;
        }
        mbar_drain(&full[slot], phase);
      }
    }
  } else if (warp >= kWorkers + 2) {
    // ------------------------------------------------------------ MMA
    const int set = warp - (kWorkers + 2);
    const uint32_t idesc = (1u << 4) | (BF16 ? (1u << 7) | (1u << 10) : 0u) | (static_cast<uint32_t>(NT >> 3) << 17) |
                           (static_cast<uint32_t>(TM >> 4) << 24);
    const uint64_t xdesc = desc_sw128(smem_u32(smem + kCodeBytes));
    const uint32_t a_tmem = tmem + set * kACols, d_set = tmem_d + set * C::ND * C::DCOLS;
    uint64_t* const df = dfull + set * C::ND;
    uint64_t* const de = dempty + set * C::ND;
    int d = 0, base = 0, slot = set;                                   // slot: of this set's next stage
    uint32_t dphase = 0, aphase = 0, phase = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t ph) {
      return __all_sync(kFull, wait_on(bar, ph, abort_flag, Q.wait_ns)) != 0;
    };
    for (int tile = blockIdx.x; tile < Q.mt && ok; tile += gridDim.x, base += nst) {
      const int own0 = (base + set) & 1;
      for (int s = own0; s < nst; s += 2) {
        ok = wait(&full[slot], phase) && wait(&afull[set], aphase) && wait(&de[d], dphase ^ 1u);
        if (!ok) break;
        aphase ^= 1u;
        tc_fence_after();
        const uint64_t xd = xdesc + (slot * C::STAGE >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < KS / 16; ++kk) {                       // K = 16: 8 columns of A, 32 bytes of x
            constexpr int MMAS = KS / 16 / C::GPS;                     // of a group
            tc_mma_f16_ts(d_set + d * C::DCOLS + kk / MMAS * NT, a_tmem + kk * 8,
                          xd + (((kk >> 2) * kXAtom) >> 4) + 2 * (kk & 3), idesc,
                          kk % MMAS > 0 ? 1u : 0u);
          }
          tc_commit(&df[d]);
          tc_commit(&aempty[set]);
          tc_commit(&empty[slot]);
        }
        __syncwarp();
        if (++d == C::ND) {
          d = 0;
          dphase ^= 1u;
        }
        if ((slot += 2) >= C::S) {
          slot -= C::S;
          phase ^= 1u;
        }
      }
    }
    if (!ok) {
      report(Q.status, MOE_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    if (elect_one()) tc_commit(&drain[set]);
    __syncwarp();
    mbar_drain(&drain[set], 0);
  } else {
    // ------------------------------------------------------------ workers
    const int quad = warp & 3, set = warp >> 3, half = (warp >> 2) & 1, quarter = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const int lrow = quad * 32 + lane;                                 // TMEM lane
    const int out_row = P.swiglu ? quad * 16 + (lane & 15) : lrow;     // output of the tile
    const int srow = P.swiglu && lane >= 16 ? TM / 2 + out_row : out_row;   // row of the stage
    constexpr int HC = 128 / GROUP;                                    // groups of half a stage
    constexpr int HK = 128 / HC;
    // first of this thread's groups of a stage (then every fourth) and of its tokens
    const int my_group = C::GPS == 2 ? quarter >> 1 : quarter;
    const int my_token = C::GPS == 2 ? (quarter & 1) * 8 : 0;
    int base = 0, d[2] = {0, 0}, slot = set;
    uint32_t dphase[2] = {0, 0}, aphase = 0, phase = 0, rphase = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t ph) {
      return __all_sync(kFull, wait_on(bar, ph, abort_flag, Q.wait_ns)) != 0;
    };
    auto arrive = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    if (Q.stall && blockIdx.x == 0) ok = wait(stall, 0);               // testing aid: runs out
    for (int tile = blockIdx.x; tile < Q.mt && ok; tile += gridDim.x, base += nst) {
      const int first = tile * per;
      const int wrow = min(first + out_row, outs - 1) + (P.swiglu && lane >= 16 ? outs : 0);
      const size_t sbase = static_cast<size_t>(wrow) * P.groups;
      // zeros of a stage's half ...
      auto fetch_c = [&](int s, uint32_t (&z)[HC]) {
#pragma unroll
        for (int i = 0; i < HC; ++i) {
          const int k = s * KS + half * 128 + i * HK;
          z[i] = 8u;
          if (FMT == MOE_W_INT4 && P.zeros != nullptr && k < P.K) z[i] = __ldg(P.zeros + sbase + k / GROUP) & 15u;
        }
      };
      // ... and the scales of this thread's groups of a stage
      auto fetch_s = [&](int s, uint32_t (&f)[C::MINE]) {
#pragma unroll
        for (int j = 0; j < C::MINE; ++j) {
          const int gi = s * C::GPS + my_group + 4 * j;
          f[j] = 0;
          if (gi >= P.groups) continue;
          if (FMT == MOE_W_MXFP4) f[j] = 0x100u | __ldg(static_cast<const uint8_t*>(P.scales) + sbase + gi);
          else if (P.scale_type == MOE_DT_F32) f[j] = __ldg(static_cast<const uint32_t*>(P.scales) + sbase + gi);
          else f[j] = __ldg(static_cast<const uint16_t*>(P.scales) + sbase + gi);
        }
      };
      auto scale_of = [&](uint32_t r) {
        if (FMT == MOE_W_MXFP4) return r == 0 ? 0.f : w4::e8m0_value(r & 255u);
        if (P.scale_type == MOE_DT_F32) return __uint_as_float(r);
        if (P.scale_type == MOE_DT_BF16) return __uint_as_float(r << 16);
        return __half2float(__ushort_as_half(static_cast<uint16_t>(r)));
      };
      float acc[C::TOKENS];
#pragma unroll
      for (int i = 0; i < C::TOKENS; ++i) acc[i] = 0.f;
      const int own0 = (base + set) & 1;                               // this set's first stage of the tile
      uint32_t zn[HC], f0[C::MINE], f1[C::MINE];                       // scales of the next two stages to add up
      fetch_c(own0, zn);
      fetch_s(0, f0);
      fetch_s(1, f1);
      // The accumulators of set st, this thread's groups and tokens, scaled, into acc.
      auto take = [&](int st, const float (&sc)[C::MINE]) {
        const int di = st * C::ND + d[st];
        if (!wait(&dfull[di], dphase[st])) return false;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < C::MINE; ++j) {
          float v[C::TOKENS];
          w4tc::tmem_load(tmem_d + lanes + di * C::DCOLS + (my_group + 4 * j) * NT + my_token, v);
          const float2 s2 = make_float2(sc[j], sc[j]);
#pragma unroll
          for (int i = 0; i < C::TOKENS; i += 2) {
            const float2 r = __ffma2_rn(make_float2(v[i], v[i + 1]), s2, make_float2(acc[i], acc[i + 1]));
            acc[i] = r.x;
            acc[i + 1] = r.y;
          }
        }
        tc_fence_before();
        arrive(&dempty[di]);
        if (++d[st] == C::ND) {
          d[st] = 0;
          dphase[st] ^= 1u;
        }
        return true;
      };
      auto add_up = [&](int s) {
        float f[C::MINE];
#pragma unroll
        for (int j = 0; j < C::MINE; ++j) {
          f[j] = scale_of(f0[j]);
          f0[j] = f1[j];
        }
        if (s + 2 < nst) fetch_s(s + 2, f1);
        return ((base + s) & 1) != 0 ? take(1, f) : take(0, f);
      };
      int next = 0;                                                    // the next stage to add up
      for (int s = own0; s < nst && ok; s += 2) {
        // stages up to s - 2 first: the MMAs of stage s - 2, whose A buffer is next,
        // may wait for accumulators
        for (; next < s - 1 && ok; ++next) ok = add_up(next);
        uint32_t c[HC];
#pragma unroll
        for (int i = 0; i < HC; ++i)
          c[i] = w4tc::pair_constant<FMT, BF16>(zn[i]);
        if (!ok || !wait(&full[slot], phase)) {
          ok = false;
          break;
        }
        const uint8_t* at = smem + slot * C::STAGE + srow * 128;
        uint4 q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          q[i] = *reinterpret_cast<const uint4*>(at + (((4 * half + i) ^ (srow & 7)) << 4));
        arrive(&empty[slot]);
        if ((slot += 2) >= C::S) {
          slot -= C::S;
          phase ^= 1u;
        }
        if (s + 2 < nst) fetch_c(s + 2, zn);
#pragma unroll
        for (int h = 0; h < 2; ++h) {                                  // 64 codes at a time
          const uint32_t w[8] = {q[2 * h].x, q[2 * h].y, q[2 * h].z, q[2 * h].w,
                                 q[2 * h + 1].x, q[2 * h + 1].y, q[2 * h + 1].z, q[2 * h + 1].w};
          uint32_t a[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t up = w[i] >> 4, ci = c[(h * 64 + i * 8) / HK];
            a[4 * i] = w4tc::natural_pair<FMT, BF16, 0>(w[i], up, ci);
            a[4 * i + 1] = w4tc::natural_pair<FMT, BF16, 1>(w[i], up, ci);
            a[4 * i + 2] = w4tc::natural_pair<FMT, BF16, 2>(w[i], up, ci);
            a[4 * i + 3] = w4tc::natural_pair<FMT, BF16, 3>(w[i], up, ci);
          }
          if (h == 0) {
            if (!wait(&aempty[set], aphase ^ 1u)) {
              ok = false;
              break;
            }
            aphase ^= 1u;
            tc_fence_after();
          }
          tmem_st32(tmem + lanes + set * kACols + half * 64 + h * 32, a);
        }
        if (!ok) break;
        tc_fence_before();
        arrive(&afull[set]);
      }
      for (; next < nst && ok; ++next) ok = add_up(next);
      // the quarters' sums, each thread's row and tokens, through shared memory
      if (!ok || !wait(rempty, rphase ^ 1u)) {
        ok = false;
        break;
      }
#pragma unroll
      for (int i = 0; i < C::TOKENS; ++i) red[(quarter * TM + lrow) * (C::TOKENS + 1) + i] = acc[i];
      arrive(rfull);
      if (!wait(rfull, rphase)) {
        ok = false;
        break;
      }
      rphase ^= 1u;
      // this thread's four tokens of its row
      float y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = quarter * 4 + i;
        if (C::GPS == 2) {
          const float* r = red + ((t >> 3) * TM + lrow) * (C::TOKENS + 1) + (t & 7);
          y[i] = r[0] + r[2 * TM * (C::TOKENS + 1)];
        } else {
          const float* r = red + lrow * (C::TOKENS + 1) + t;
          y[i] = r[0] + r[TM * (C::TOKENS + 1)] + r[2 * TM * (C::TOKENS + 1)] + r[3 * TM * (C::TOKENS + 1)];
        }
      }
      arrive(rempty);
      const int n = first + out_row;
      if (P.swiglu) {
        // lanes 0-15 hold h and 16-31 u of the same outputs: each half takes every other token
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float got = __shfl_xor_sync(kFull, lane < 16 ? y[i + 1] : y[i], 16);
          const float h = lane < 16 ? y[i] : got, u = lane < 16 ? got : y[i + 1];
          const int t = quarter * 4 + i + (lane >> 4);
          if (n < outs && t < P.T) w4::store_y<BF16>(P, t, n, h / (1.f + expf(-h)) * u);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n < outs && quarter * 4 + i < P.T) w4::store_y<BF16>(P, quarter * 4 + i, n, y[i]);
      }
    }
    if (!ok) {
      report(Q.status, MOE_ERR_TIMEOUT);
      *abort_flag = 1;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWorkers + 2)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512));
}

template <int FMT, int GROUP, bool BF16>
cudaError_t launch(const LinearParams& P, const DeviceInfo& dev, int32_t* status, cudaStream_t s) {
  using C = Cfg<FMT, GROUP>;
  auto kern = linear_w4_tc16_kernel<FMT, GROUP, BF16>;
  static std::atomic<bool> done[64];
  if (!done[dev.id].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    done[dev.id].store(true, std::memory_order_release);
  }
  TcParams Q{};
  Q.L = P;
  Q.wait_ns = wait_limit_ns();
  Q.stall = test_stall();
  Q.status = status;
  const int outs = P.swiglu ? P.N / 2 : P.N, per = P.swiglu ? TM / 2 : TM;
  Q.mt = (outs + per - 1) / per;
  Q.tt = 1;
  CUtensorMap tm_w, tm_x;
  const uint64_t wd[2] = {static_cast<uint64_t>(P.K) / 2, static_cast<uint64_t>(P.N)}, ws[1] = {wd[0]};
  const uint32_t wb[2] = {KS / 2, static_cast<uint32_t>(per)};
  const uint64_t xd[2] = {static_cast<uint64_t>(P.K), static_cast<uint64_t>(P.T)},
                 xs[1] = {static_cast<uint64_t>(P.ldx) * 2};
  const uint32_t xb[2] = {64, NT};
  if (encode_tiled_sw128(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, P.codes, wd, ws, wb) != CUDA_SUCCESS ||
      encode_tiled_sw128(&tm_x, BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, P.x, xd,
                         xs, xb) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const cudaError_t e = launch_pdl(kern, dim3(Q.mt < dev.sm_count ? Q.mt : dev.sm_count), dim3(kThreads), C::SMEM, s,
                                   tm_w, tm_x, Q);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace w4t16
}  // namespace moe
