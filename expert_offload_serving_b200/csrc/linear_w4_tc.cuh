// The dense 4-bit linear on the 5th-generation tensor cores.
//
// D[128 rows of W x NT tokens] += A[128 x 128 of K] x X^T a stage.  The codes
// (8 KB) and the token rows of a stage arrive by TMA; eight warps turn the codes
// into exact values of the x type (see linear_w4.cuh) in registers and write them
// to tensor memory, where they are the A operand of tcgen05.mma kind::f16 -- no
// trip of the expanded weights through shared memory, whose bandwidth two bytes a
// weight would use up.  TMEM lane = row of W, so a thread works on one row
// throughout: its zeros and scales are its own loads.
//
// Scales.  With bf16 x they go into the weights (PRE), and one fp32 accumulator
// runs through all of K: an NVFP4 weight has 6 significant bits and an MXFP4 one
// 2, exact in bf16; an INT4 weight (code - zero) * scale has up to 12 with a bf16
// scale and 15 with an fp16 one (two bf16 values itself), and becomes the exact sum
// of two bf16 values, two A planes and two MMAs.  An fp32 scale leaves up to 28
// bits: as two bf16 values the scale is within 2^-16, and two more roundings of the
// product by 2^-16 leave the weight within 2^-14.8 of itself.  A 16-bit y takes
// that, its own rounding is 2^-8; for an fp32 y these scales stay outside (T = 1000,
// N = K = 4096: 64.5 us with groups of 128, 127 of 64, 194 of 32, where they took 71,
// 76 and 82 inside; T = 24, N = 16384: 23.7, 30.5, 38.3 against 23.0, 23.9, 26.0).
// With f16 x, whose range does not hold every scale, and in that case INT4 and MXFP4
// scales multiply the group's fp32 sum (POST): the MMAs of a group write an
// accumulator of their own, one of ND in turn, and the warps read it back and add
// it, scaled, to sums in registers while the tensor core works on later groups.
// The hand-overs that takes cost more than the second plane: at T = 64, N = 16384,
// K = 4096 with groups of 128, POST took 25 us in bf16.
//
// Few tiles: a cluster of 2, 4 or 8 CTAs shares a tile, each with a part of K, and
// each adds up, out of the others' shared memory and in their order, the sums of a
// part of the tokens.
//
// Measured, bf16 y: T = 64, N = 16384, K = 4096, INT4 by 128: 23.3 us (369 TFLOP/s, 737
// with both planes; one set of eight warps took 44).  T = 1000, N = K = 4096 with SwiGLU,
// INT4 by 32: 67 us (498, 996 with both planes), by 128 60.5 us.  T = 64, N = 1024: 8.1
// us by clusters of 8.  A tile takes some 3 to 8 us beside its stages (first loads,
// draining, epilogue), a stage of 64 tokens 1200 cycles and one of 128 1350 to 1550,
// of which the two planes' MMAs are 512 and 1024 and the expanding instructions 640
// (two a clock for most of them).  What bounds it is the hand-overs' latency: without
// the second plane's MMAs T = 1000 took 14 % less, without the expanding arithmetic
// 12 %, without both 26 %, without the loads of scales no less.
//
// Two sets of eight warps take the stages in turn, each with its own A buffer,
// accumulators and MMA-issuing warp: the hand-overs of a stage (codes landed ->
// expanded -> multiplied -> added up) cost more time than its work, and the sets'
// run side by side.  Warps 0-15: workers; quadrant (TMEM lanes) = warp % 4.
// Expanding codes, warps 0-7 take the even stages and 8-15 the odd ones, four
// warps a half of the stage's K.  Adding up, all take every stage, each a quarter
// of the tokens.  Warp 16: TMA of the codes, 17: of the token rows.  Warps 18, 19:
// MMAs of the even and the odd stages.  Work is walked in the same order by all:
// output tiles dealt to the CTAs, stages of K within.  Every wait is bounded: on
// expiry the CTA records MOE_ERR_TIMEOUT, stops issuing, drains what it issued and
// frees its TMEM.
#pragma once

#include <atomic>
#include <type_traits>

#include "linear_w4.cuh"
#include "tc.cuh"

namespace moe {
namespace w4tc {

using namespace ::moe::tc;

constexpr int KS = 128;                       // K of a stage
constexpr int TM = 128;                       // rows of W of a tile
constexpr int kWorkers = 16, kSet = 8;      // warps that expand a stage
constexpr int kThreads = (kWorkers + 4) * 32;
constexpr int kCodeBytes = TM * KS / 2;
constexpr uint32_t kNegateA = 1u << 13;       // instruction descriptor: A counts negated
constexpr int kACols = KS / 2;                // TMEM columns of an A buffer (two 16-bit values a column)

struct TcParams {
  LinearParams L;
  uint64_t wait_ns;
  int stall, mt, tt;                          // tiles of rows, of tokens
  int ck_bits;                                // CTAs of a cluster that share a tile's K (log2)
  int32_t* status;
};

// Whether an x type has the scales outside the products of its own accord.
template <int FMT, bool BF16>
constexpr bool kPost = !BF16 && FMT != MOE_W_NVFP4;

// POST: the scale multiplies a group's sum.
template <int FMT, int GROUP, bool BF16, int NT, bool POST>
struct Cfg {
  static constexpr int PLANES = BF16 && FMT == MOE_W_INT4 && !POST ? 2 : 1;   // bf16 values of a weight
  static constexpr int AC = PLANES * kACols;                           // TMEM columns of a set's A buffer
  static constexpr int GPS = POST ? KS / GROUP : 1;                    // accumulators of a stage
  static constexpr int HC = FMT == MOE_W_NVFP4 ? 4 : GROUP == 32 ? 2 : 1;   // groups of half a stage
  static constexpr int ND = (512 - 2 * AC) / NT / 2 < 6 ? (512 - 2 * AC) / NT / 2 : 6;   // accumulators of a set
  static constexpr int XB = NT * 128;                                  // 64 elements of the token rows
  static constexpr int STAGE = kCodeBytes + 2 * XB;
  static constexpr int S = 220 * 1024 / STAGE < 12 ? 220 * 1024 / STAGE : 12;
  static constexpr int N_BARS = 2 * S + 4 + 4 * ND + 3;
  static constexpr int BAR_BYTES = (N_BARS * 8 + 16 + 127) / 128 * 128;
  static constexpr int SMEM = 1024 + S * STAGE + BAR_BYTES;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(kWorkers * 32 * NT <= S * STAGE, "the sums of a CTA fit the stages' memory");
  static_assert(STAGE % 1024 == 0 && S >= 3 && ND >= 1, "");
};

// Pair P (0..3) of a word in natural order: the codes 2P (low half) and 2P + 1.
// `up` is the word shifted right by a nibble.
template <int FMT, bool BF16, int P>
__device__ __forceinline__ uint32_t natural_pair(uint32_t w, uint32_t up, uint32_t c) {
  if constexpr (FMT == MOE_W_INT4) {
    // byte P of the word to the low half, of the shifted word to the high half
    // (the other two bytes are masked away)
    const uint32_t b = __byte_perm(w, up, P | (P << 4) | ((4 + P) << 8) | ((4 + P) << 12));
    return w4::sub2<BF16>(w4::and_or(b, 0x000F000Fu, BF16 ? 0x43004300u : 0x64006400u), c);
  } else {
    uint32_t h;
    asm("{ .reg .b8 b; cvt.u8.u32 b, %1; cvt.rn.f16x2.e2m1x2 %0, b; }" : "=r"(h) : "r"(w >> (8 * P)));
    // bf16: exponent and mantissa 3 places down read as the value * 2^-112
    if constexpr (BF16) return w4::mul2<true>(w4::and_or(h, 0x80008000u, (h >> 3) & 0x0FFF0FFFu), c);
    return FMT == MOE_W_NVFP4 ? w4::mul2<false>(h, c) : h;
  }
}

// The constant `c` of natural_pair from a zero point, or an E4M3 scale byte.
template <int FMT, bool BF16>
__device__ __forceinline__ uint32_t pair_constant(uint32_t raw) {
  if constexpr (FMT == MOE_W_INT4)
    return ((BF16 ? 0x4300u : 0x6400u) | raw) * 0x10001u;
  else if constexpr (FMT == MOE_W_MXFP4)
    return 0x77807780u;                                                // 2^112 twice
  const __half h = __half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(raw), __NV_E4M3));
  const uint32_t u = BF16 ? __float_as_uint(__half2float(h) * 5.192296858534828e33f) >> 16 : __half_as_ushort(h);
  return u | (u << 16);
}

// E8M0 as a bf16 pair, a quarter of it: 2^(b - 129), so that with 6 times it no
// value leaves bf16's range (small ones are subnormals, which hold them exactly).
// The sums are multiplied by 4.
__device__ __forceinline__ uint32_t e8m0_quarter(uint32_t b) {
  return (b == 255 ? 0x7FC0u : b < 3 ? 0x10u << b : (b - 2) << 7) * 0x10001u;
}

__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
  const __nv_bfloat162 r = __hfma2(reinterpret_cast<__nv_bfloat162&>(a), reinterpret_cast<__nv_bfloat162&>(b),
                                   reinterpret_cast<__nv_bfloat162&>(c));
  return reinterpret_cast<const uint32_t&>(r);
}
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t taddr, float (&v)[N]) {
  if constexpr (N == 8) tmem_ld8(taddr, v);
  else if constexpr (N == 16) tmem_ld16(taddr, v);
  else tmem_ld32(taddr, v);
}

// N consecutive elements of type E at index i of p (aligned to N of them) by one load,
// each masked and OR-ed.
template <typename E, int N>
__device__ __forceinline__ void load_groups(const void* p, size_t i, uint32_t (&v)[N], uint32_t keep, uint32_t mark) {
  constexpr int B = sizeof(E) * N;
  using V = typename std::conditional<
      B == 1, uint8_t,
      typename std::conditional<
          B == 2, uint16_t,
          typename std::conditional<B == 4, uint32_t, typename std::conditional<B == 8, uint2, uint4>::type>::type>::type>::type;
  static_assert(sizeof(V) == B, "one load");
  union {
    V v;
    E e[N];
  } u;
  u.v = __ldg(reinterpret_cast<const V*>(static_cast<const E*>(p) + i));
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = (u.e[j] & keep) | mark;
}

// A bounded wait for hand-overs that are due within a stage.  A look in vain is
// followed by a short sleep: waiting warps that look without pause took a third of
// the issue slots from those that work.  The clock is read only after 64 looks:
// reading it takes some 400 cycles, as long as a stage should.
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint64_t limit_ns) {
  for (int i = 0; i < 64; ++i) {
    if (mbar_try(bar, parity)) return true;
    __nanosleep(20);
  }
  return mbar_wait<false>(bar, parity, abort_flag, limit_ns);
}

// PRE: stages whose products run through one accumulator.  The tensor cores cut sums
// off instead of rounding them: K = 16384 in two planes through one accumulator is off
// by 7.7e-6 of the result's norm (2.4e-6 where a cluster shares it).  For an fp32 y
// the sums are added in registers after 8 stages (4.8e-7); a 16-bit y does not notice
// and they run on.
constexpr int kRun = 8;

// SHARED: a cluster of CTAs shares a tile's K.  RUNS: PRE sums are added in registers
// after each run.  (Instances of their own: the few more instructions of SHARED made
// the loops of the other one 12 % slower at NT = 64, and the sums that RUNS holds
// across them cost 8 % at NT = 32 and 64 and 14 % at 128.  T = 64, N = 16384, K = 4096,
// INT4 by 128: 23.3 us without, 25.4 with.)
template <int FMT, int GROUP, bool BF16, int NT, bool POST, bool SHARED, bool RUNS>
__global__ void __launch_bounds__(kThreads, 1)
    linear_w4_tc_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                        const __grid_constant__ TcParams Q) {
  using C = Cfg<FMT, GROUP, BF16, NT, POST>;
  const LinearParams& P = Q.L;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::S * C::STAGE);
  uint64_t* full = bars;                      // [S] a stage's codes and token rows landed
  uint64_t* empty = bars + C::S;              // [S] ... read by the workers and the MMAs
  uint64_t* afull = bars + 2 * C::S;          // [2] expanded weights written
  uint64_t* aempty = afull + 2;               // [2] ... and used
  uint64_t* dfull = aempty + 2;               // [2][ND] an accumulator complete
  uint64_t* dempty = dfull + 2 * C::ND;       // [2][ND] ... and read
  uint64_t* drain = dempty + 2 * C::ND;       // [2]
  uint64_t* stall = drain + 2;                // never arrived on (testing aid)
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + C::N_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // this CTA's stages of K: nst of them from s0 on (all, but for a shared tile)
  const int ck_bits = SHARED ? Q.ck_bits : 0, ck = 1 << ck_bits;
  const int rank = SHARED ? static_cast<int>(cluster_rank()) : 0;
  const int all = (P.K + KS - 1) / KS, s0 = all * rank >> ck_bits, nst = (all * (rank + 1) >> ck_bits) - s0;
  const int ntiles = Q.mt * Q.tt, tile0 = blockIdx.x >> ck_bits, tiles_step = gridDim.x >> ck_bits;
  constexpr int run = POST ? 1 : RUNS ? kRun : 1 << 30;
  int meetings = 0;                           // barriers over the cluster: two, on every path
  const int outs = P.swiglu ? P.N >> 1 : P.N, per = P.swiglu ? TM / 2 : TM;   // outputs: in all, of a tile

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::S; ++s) {
      mbar_init(&full[s], 2);
      mbar_init(&empty[s], kSet + 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&afull[i], kSet);
      mbar_init(&aempty[i], 1);
    }
    for (int i = 0; i < 2 * C::ND; ++i) {
      mbar_init(&dfull[i], 1);
      mbar_init(&dempty[i], kWorkers);
    }
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
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
  const uint32_t tmem = *tmem_holder, tmem_d = tmem + 2 * C::AC;
  pdl_wait();
  pdl_trigger();

  if (warp == kWorkers || warp == kWorkers + 1) {
    // ------------------------------------------------------------ TMA
    const bool codes = warp == kWorkers;
    if (lane == 0) {
      const uint64_t pol = codes && Q.tt == 1 ? policy_evict_first() : policy_evict_last();
      int slot = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = tile0; tile < ntiles && ok; tile += tiles_step) {
        const int m = tile / Q.tt * per, t = tile % Q.tt * NT;
        for (int s = 0; s < nst; ++s) {
          if (!wait_on(&empty[slot], phase ^ 1u, abort_flag, Q.wait_ns)) {
            ok = false;
            break;
          }
          uint8_t* at = smem + slot * C::STAGE;
          if (codes) {
            mbar_expect_tx(&full[slot], kCodeBytes);
            tma_load_2d(at, &tm_w, &full[slot], (s0 + s) * (KS / 2), m, pol);
            if (P.swiglu) tma_load_2d(at + kCodeBytes / 2, &tm_w, &full[slot], (s0 + s) * (KS / 2), outs + m, pol);
          } else {
            mbar_expect_tx(&full[slot], 2 * C::XB);
#pragma unroll
            for (int a = 0; a < 2; ++a)
              tma_load_2d(at + kCodeBytes + a * C::XB, &tm_x, &full[slot], (s0 + s) * KS + a * 64, t, pol);
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
      // What was issued has landed before the CTA leaves.  (Where the other kind of
      // a stage was never issued its barrier does not complete, and the bounded
      // wait has long outlasted the copy.)
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
    const uint32_t a_tmem = tmem + set * C::AC, d_set = tmem_d + set * C::ND * NT;
    uint64_t* const df = dfull + set * C::ND;
    uint64_t* const de = dempty + set * C::ND;
    int d = 0, base = 0, slot = set;                                   // slot: of this set's next stage
    uint32_t dphase = 0, aphase = 0, phase = 0;
    bool ok = true;
    // one verdict for the warp: its lanes take the same path
    auto wait = [&](uint64_t* bar, uint32_t ph) {
      return __all_sync(kFull, wait_on(bar, ph, abort_flag, Q.wait_ns)) != 0;
    };
    for (int tile = tile0; tile < ntiles && ok; tile += tiles_step, base += nst) {
      const int own0 = (base + set) & 1;
      for (int s = own0; s < nst && ok; s += 2) {
        ok = wait(&full[slot], phase) && wait(&afull[set], aphase);
        if (!ok) break;
        aphase ^= 1u;
        const uint64_t xd = xdesc + (slot * C::STAGE >> 4);
        // the set's first and last stage of a run (of one stage, in POST)
        const bool begin = POST || (s & (run - 1)) < 2, end = POST || (s & (run - 1)) >= run - 2 || s + 2 >= nst;
#pragma unroll
        for (int j = 0; j < C::GPS; ++j) {
          if (begin) {
            ok = wait(&de[d], dphase ^ 1u);
            if (!ok) break;
          }
          tc_fence_after();
          constexpr int MMAS = KS / 16 / C::GPS;
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < MMAS; ++i) {
              const int kk = j * MMAS + i;                             // K = 16: 8 columns of A, 32 bytes of x
              const uint64_t db = xd + (((kk >> 2) * C::XB) >> 4) + 2 * (kk & 3);
              tc_mma_f16_ts(d_set + d * NT, a_tmem + kk * 8, db, C::PLANES == 2 ? idesc | kNegateA : idesc,
                            i > 0 || !begin ? 1u : 0u);
              if (C::PLANES == 2) tc_mma_f16_ts(d_set + d * NT, a_tmem + kACols + kk * 8, db, idesc, 1u);
            }
            if (end) tc_commit(&df[d]);
            if (j == C::GPS - 1) {
              tc_commit(&aempty[set]);
              tc_commit(&empty[slot]);
            }
          }
          __syncwarp();
          if (end && ++d == C::ND) {
            d = 0;
            dphase ^= 1u;
          }
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
    // this thread's row: of the tile's outputs, and in the stage
    const int out_row = P.swiglu ? quad * 16 + (lane & 15) : quad * 32 + lane;
    const int srow = P.swiglu && lane >= 16 ? TM / 2 + out_row : out_row;
    // codes of the half stage: two 16-byte chunks of the row, swizzled over 64 bytes
    const uint32_t c0 = srow * 64 + (((2 * half) ^ ((srow >> 1) & 3)) << 4);
    const uint32_t c1 = srow * 64 + (((2 * half + 1) ^ ((srow >> 1) & 3)) << 4);
    constexpr int CN = NT / 4;                                         // tokens of this thread
    constexpr int HC = C::HC;
    constexpr int HK = 64 / HC;                                        // K of one
    int base = 0, d[2] = {0, 0}, slot = set;                           // base: stages of the tiles before this one
    uint32_t dphase[2] = {0, 0}, aphase = 0, phase = 0;                // slot: of this set's next stage
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t ph) {
      return __all_sync(kFull, wait_on(bar, ph, abort_flag, Q.wait_ns)) != 0;
    };
    auto arrive = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    if (Q.stall && blockIdx.x == 0) ok = wait(stall, 0);               // testing aid: runs out
    for (int tile = tile0; tile < ntiles && ok; tile += tiles_step, base += nst) {
      const int first = tile / Q.tt * per, tok0 = tile % Q.tt * NT;
      const int wrow = min(first + out_row, outs - 1) + (P.swiglu && lane >= 16 ? outs : 0);
      const size_t sbase = static_cast<size_t>(wrow) * P.groups;
      // Raw zeros and scales of a stage's half (0x10000 or more: there is one) ...  A
      // load touches a line per lane, whatever its width, and the lines are what it
      // costs: where rows are aligned for it (P.scale_vec), one takes all the groups.
      auto fetch_c = [&](int s, uint32_t (&z)[HC], uint32_t (&f)[HC]) {
        const int g0 = ((s0 + s) * KS + half * 64) / GROUP;
#pragma unroll
        for (int i = 0; i < HC; ++i) {
          z[i] = 8u;
          f[i] = 0;
        }
        const size_t at = sbase + g0;
        if (HC > 1 && P.scale_vec && g0 + HC <= P.groups) {
          if (FMT == MOE_W_INT4 && P.zeros != nullptr) load_groups<uint8_t, HC>(P.zeros, at, z, 15u, 0u);
          if (FMT != MOE_W_INT4) load_groups<uint8_t, HC>(P.scales, at, f, 255u, 0x10000u);
          else if (!POST && P.scale_type == MOE_DT_F32) load_groups<uint32_t, HC>(P.scales, at, f, ~0u, 0u);
          else if (!POST) load_groups<uint16_t, HC>(P.scales, at, f, 0xFFFFu, 0u);
          return;
        }
#pragma unroll
        for (int i = 0; i < HC; ++i) {
          if (g0 + i >= P.groups) continue;
          if (FMT == MOE_W_INT4 && P.zeros != nullptr) z[i] = __ldg(P.zeros + at + i) & 15u;
          if (FMT != MOE_W_INT4) f[i] = 0x10000u | __ldg(static_cast<const uint8_t*>(P.scales) + at + i);
          else if (!POST && P.scale_type == MOE_DT_F32) f[i] = __ldg(static_cast<const uint32_t*>(P.scales) + at + i);
          else if (!POST) f[i] = __ldg(static_cast<const uint16_t*>(P.scales) + at + i);
        }
      };
      // ... and the scales of a whole stage's groups (POST)
      auto fetch_s = [&](int s, uint32_t (&f)[C::GPS]) {
        const int g0 = (s0 + s) * C::GPS;
#pragma unroll
        for (int j = 0; j < C::GPS; ++j) f[j] = 0;
        if (!POST) return;
        const size_t at = sbase + g0;
        if (C::GPS > 1 && P.scale_vec && g0 + C::GPS <= P.groups) {
          if (FMT == MOE_W_MXFP4) load_groups<uint8_t, C::GPS>(P.scales, at, f, 255u, 0x10000u);
          else if (P.scale_type == MOE_DT_F32) load_groups<uint32_t, C::GPS>(P.scales, at, f, ~0u, 0u);
          else load_groups<uint16_t, C::GPS>(P.scales, at, f, 0xFFFFu, 0u);
          return;
        }
#pragma unroll
        for (int j = 0; j < C::GPS; ++j) {
          if (g0 + j >= P.groups) continue;
          if (FMT == MOE_W_MXFP4) f[j] = 0x10000u | __ldg(static_cast<const uint8_t*>(P.scales) + at + j);
          else if (P.scale_type == MOE_DT_F32) f[j] = __ldg(static_cast<const uint32_t*>(P.scales) + at + j);
          else f[j] = __ldg(static_cast<const uint16_t*>(P.scales) + at + j);
        }
      };
      auto scale_of = [&](uint32_t r) {
        if (FMT == MOE_W_MXFP4) return r == 0 ? 0.f : w4::e8m0_value(r & 255u);
        if (P.scale_type == MOE_DT_F32) return __uint_as_float(r);
        if (P.scale_type == MOE_DT_BF16) return __uint_as_float(r << 16);
        return __half2float(__ushort_as_half(static_cast<uint16_t>(r)));
      };
      float acc[CN];
#pragma unroll
      for (int i = 0; i < CN; ++i) acc[i] = 0.f;
      const int own0 = (base + set) & 1;                               // this set's first stage of the tile
      uint32_t zn[HC], sn[HC], fn[C::GPS];
      fetch_c(own0, zn, sn);
      fetch_s(0, fn);
      // An accumulator of a set, times sc, into acc.
      auto take = [&](int st, float sc) {
        uint64_t* const df = dfull + st * C::ND;
        if (!wait(&df[d[st]], dphase[st])) return false;
        tc_fence_after();
        float v[CN];
        tmem_load(tmem_d + lanes + (st * C::ND + d[st]) * NT + quarter * CN, v);
        tc_fence_before();
        arrive(&dempty[st * C::ND + d[st]]);
        if (++d[st] == C::ND) {
          d[st] = 0;
          dphase[st] ^= 1u;
        }
        const float2 s2 = make_float2(sc, sc);
#pragma unroll
        for (int i = 0; i < CN; i += 2) {
          const float2 r = __ffma2_rn(make_float2(v[i], v[i + 1]), s2, make_float2(acc[i], acc[i + 1]));
          acc[i] = r.x;
          acc[i + 1] = r.y;
        }
        return true;
      };
      // PRE: run r, the accumulators of the sets that have stages in it.
      const float pre_scale = FMT == MOE_W_NVFP4 ? P.tensor_scale : FMT == MOE_W_MXFP4 ? 4.f : 1.f;
      auto add_run = [&](int r) {
        const int n = min(run, nst - r * run);
        const bool odd = base & 1;                                     // set of the run's first stage (run is even)
        if ((n > 1 || !odd) && !take(0, pre_scale)) return false;
        return !(n > 1 || odd) || take(1, pre_scale);
      };
      // POST: the groups of stage s; the next stage's scales are on their way meanwhile.
      auto add_up = [&](int s) {
        float f[C::GPS];
#pragma unroll
        for (int j = 0; j < C::GPS; ++j) f[j] = scale_of(fn[j]);
        if (s + 1 < nst) fetch_s(s + 1, fn);
        const bool odd = (base + s) & 1;
#pragma unroll
        for (int j = 0; j < C::GPS; ++j)
          if (!(odd ? take(1, f[j]) : take(0, f[j]))) return false;
        return true;
      };
      int next = 0;                                                    // the next stage, or run, to add up
      for (int s = own0; s < nst && ok; s += 2) {
        // Stages up to s - 2 are added up before the wait for the buffer that stage
        // s - 2's MMAs read: these may in turn wait for accumulators (a stage can
        // have more groups than there are accumulators).
        if constexpr (POST || RUNS)
          for (; next * run + run < s && ok; ++next) ok = POST ? add_up(next) : add_run(next);
        uint32_t c[HC], s1[HC], s2[HC];
#pragma unroll
        for (int i = 0; i < HC; ++i) {
          s1[i] = s2[i] = 0;
          if (FMT == MOE_W_NVFP4) {
            c[i] = sn[i] == 0 ? 0u : pair_constant<FMT, BF16>(sn[i] & 255u);
          } else {
            c[i] = pair_constant<FMT, BF16>(zn[i]);
            if (!POST && FMT == MOE_W_MXFP4) s1[i] = sn[i] == 0 ? 0u : e8m0_quarter(sn[i] & 255u);
            if (!POST && FMT == MOE_W_INT4) {
              const float f = scale_of(sn[i]);
              const __nv_bfloat16 hi = __float2bfloat16_rn(f);
              s1[i] = __bfloat16_as_ushort(hi) * 0x10001u;
              s2[i] = __bfloat16_as_ushort(__float2bfloat16_rn(f - __bfloat162float(hi))) * 0x10001u;
            }
          }
        }
        if (!ok || !wait(&full[slot], phase)) {
          ok = false;
          break;
        }
        const uint8_t* at = smem + slot * C::STAGE;
        const uint4 q0 = *reinterpret_cast<const uint4*>(at + c0), q1 = *reinterpret_cast<const uint4*>(at + c1);
        arrive(&empty[slot]);
        if ((slot += 2) >= C::S) {
          slot -= C::S;
          phase ^= 1u;
        }
        if (s + 2 < nst) fetch_c(s + 2, zn, sn);
        const uint32_t w[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
        const uint32_t a_at = tmem + lanes + set * C::AC + half * 32;
        // four words (16 columns) at a time: registers
        auto expand = [&](int i0, auto third) {
          uint32_t a[16], lo[16];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = i0 + e, h = i * 8 / HK;
            const uint32_t up = w[i] >> 4;
            a[4 * e] = natural_pair<FMT, BF16, 0>(w[i], up, c[h]);
            a[4 * e + 1] = natural_pair<FMT, BF16, 1>(w[i], up, c[h]);
            a[4 * e + 2] = natural_pair<FMT, BF16, 2>(w[i], up, c[h]);
            a[4 * e + 3] = natural_pair<FMT, BF16, 3>(w[i], up, c[h]);
            if constexpr (!POST && FMT == MOE_W_MXFP4) {
#pragma unroll
              for (int p = 4 * e; p < 4 * e + 4; ++p) a[p] = w4::mul2<true>(a[p], s1[h]);
            }
            if constexpr (C::PLANES == 2) {
              // (code - zero) * scale = hi + lo: hi rounded, lo what is left, exact.  The
              // first plane holds -hi (the MMA negates it), which lo's one fused
              // multiply-add takes as it is.
#pragma unroll
              for (int p = 4 * e; p < 4 * e + 4; ++p) {
                const uint32_t v = a[p];
                a[p] = w4::mul2<true>(v, s1[h] ^ 0x80008000u);
                lo[p] = fma2(v, s1[h], a[p]);
                if constexpr (decltype(third)::value) lo[p] = fma2(v, s2[h], lo[p]);
              }
            }
          }
          if (i0 == 0) {
            ok = wait(&aempty[set], aphase ^ 1u);
            tc_fence_after();
          }
          tmem_st16(a_at + i0 * 4, a);
          if constexpr (C::PLANES == 2) tmem_st16(a_at + kACols + i0 * 4, lo);
        };
        if (C::PLANES == 2 && P.scale_type != MOE_DT_BF16) {
          expand(0, std::true_type());
          expand(4, std::true_type());
        } else {
          expand(0, std::false_type());
          expand(4, std::false_type());
        }
        tmem_st_wait();
        if (!ok) break;
        aphase ^= 1u;
        tc_fence_before();
        arrive(&afull[set]);
      }
      for (; next * run < nst && ok; ++next) ok = POST ? add_up(next) : add_run(next);
      if (!ok) break;
      // y[t][n] of tokens i and i + 1 of this thread: lanes hold consecutive n
      const int n = first + out_row;
      auto store_pair = [&](int i, float v0, float v1) {
        const int t = tok0 + quarter * CN + i;
        if (P.swiglu) {
          // lanes 0-15 hold h and 16-31 u of the same outputs: each half takes one token
          const float got = __shfl_xor_sync(kFull, lane < 16 ? v1 : v0, 16);
          const float h = lane < 16 ? v0 : got, u = lane < 16 ? got : v1;
          if (n < outs && t + (lane >> 4) < P.T) w4::store_y<BF16>(P, t + (lane >> 4), n, h / (1.f + expf(-h)) * u);
        } else {
          if (n < outs && t < P.T) w4::store_y<BF16>(P, t, n, v0);
          if (n < outs && t + 1 < P.T) w4::store_y<BF16>(P, t + 1, n, v1);
        }
      };
      if (!SHARED) {
#pragma unroll
        for (int i = 0; i < CN; i += 2) store_pair(i, acc[i], acc[i + 1]);
        continue;
      }
      // A shared tile: every CTA lays its sums out (the stages' memory is free, every
      // MMA has finished), and each adds up a part of the tokens.
      float* const red = reinterpret_cast<float*>(smem) + threadIdx.x;
#pragma unroll
      for (int i = 0; i < CN; ++i) red[i * kWorkers * 32] = acc[i];
      cluster_sync();
      ++meetings;
      const int share = CN >> ck_bits < 2 ? 2 : CN >> ck_bits;
      for (int i = rank * share; i < CN && i < (rank + 1) * share; i += 2) {
        float v0 = 0.f, v1 = 0.f;
        for (int r = 0; r < ck; ++r) {
          const uint32_t at = cluster_addr(red + i * kWorkers * 32, r);
          float a, b;
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(a) : "r"(at));
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(b) : "r"(at + kWorkers * 128));
          v0 += a;
          v1 += b;
        }
        store_pair(i, v0, v1);
      }
    }
    if (!ok) {
      report(Q.status, MOE_ERR_TIMEOUT);
      *abort_flag = 1;
    }
  }
  __syncwarp();
  if (SHARED)
    for (; meetings < 2; ++meetings) cluster_sync();                   // nobody leaves while its memory is read
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWorkers + 2)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512));
}

template <int FMT, int GROUP, bool BF16, int NT, bool POST, bool SHARED, bool RUNS>
cudaError_t launch_tiles(TcParams Q, const CUtensorMap& tm_w, const CUtensorMap& tm_x, int64_t tiles,
                         const DeviceInfo& dev, cudaStream_t s) {
  using C = Cfg<FMT, GROUP, BF16, NT, POST>;
  auto kern = linear_w4_tc_kernel<FMT, GROUP, BF16, NT, POST, SHARED, RUNS>;
  struct Device {
    std::atomic<bool> ready;
    int clusters[4];                          // that run side by side, of 1, 2, 4 and 8 CTAs
  };
  static Device devices[64];
  Device& d = devices[dev.id];
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  if (!d.ready.load(std::memory_order_acquire)) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    for (int b = 1; b <= 3 && SHARED; ++b) {
      cfg.gridDim = dim3(1u << b);
      at[0].val.clusterDim.x = 1u << b;
      e = cudaOccupancyMaxActiveClusters(&d.clusters[b], kern, &cfg);
      if (e != cudaSuccess) return e;
    }
    d.ready.store(true, std::memory_order_release);
  }
  // The most CTAs a tile that run side by side (the SMs of a GPC may not divide into
  // clusters: 16 tiles in clusters of 8 took two turns, 22 us, at T = 256, N = 1024,
  // K = 4096).
  if (SHARED)
    while (Q.ck_bits > 0 && tiles > d.clusters[Q.ck_bits]) --Q.ck_bits;
  cfg.gridDim = dim3(static_cast<unsigned>(SHARED                ? tiles << Q.ck_bits
                                           : tiles < dev.sm_count ? tiles
                                                                  : dev.sm_count));
  at[0].val.clusterDim.x = 1u << Q.ck_bits;
  cfg.attrs = SHARED ? at : at + 1;
  cfg.numAttrs = SHARED ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tm_w, tm_x, Q);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int FMT, int GROUP, bool BF16, int NT, bool POST>
cudaError_t launch(const LinearParams& P, const DeviceInfo& dev, int32_t* status, cudaStream_t s) {
  TcParams Q{};
  Q.L = P;
  Q.wait_ns = wait_limit_ns();
  Q.stall = test_stall();
  Q.status = status;
  using C = Cfg<FMT, GROUP, BF16, NT, POST>;
  constexpr int A = C::GPS > C::HC ? C::GPS : C::HC;                   // groups that are loaded at once
  const int e = FMT != MOE_W_INT4 ? 1 : P.scale_type == MOE_DT_F32 ? 4 : 2;
  Q.L.scale_vec = A > 1 && P.groups % A == 0 && aligned(P.scales, A * e) && aligned(P.zeros, A);
  const int outs = P.swiglu ? P.N / 2 : P.N, per = P.swiglu ? TM / 2 : TM;
  Q.mt = (outs + per - 1) / per;
  Q.tt = (P.T + NT - 1) / NT;
  CUtensorMap tm_w, tm_x;
  const uint64_t wd[2] = {static_cast<uint64_t>(P.K) / 2, static_cast<uint64_t>(P.N)}, ws[1] = {wd[0]};
  const uint32_t wb[2] = {KS / 2, static_cast<uint32_t>(per)};
  const uint64_t xd[2] = {static_cast<uint64_t>(P.K), static_cast<uint64_t>(P.T)},
                 xs[1] = {static_cast<uint64_t>(P.ldx) * 2};
  const uint32_t xb[2] = {64, NT};
  if (encode_tiled_sw64(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, P.codes, wd, ws, wb) != CUDA_SUCCESS ||
      encode_tiled_sw128(&tm_x, BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, P.x, xd,
                         xs, xb) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const int64_t tiles = static_cast<int64_t>(Q.mt) * Q.tt;
  // Tiles for less than half the SMs: clusters share them, as long as a CTA keeps
  // four stages.
  const int nst = (P.K + KS - 1) / KS;
  while (Q.ck_bits < 3 && tiles << (Q.ck_bits + 1) <= dev.sm_count && nst >> (Q.ck_bits + 1) >= 4) ++Q.ck_bits;
  if constexpr (!POST) {
    if (!P.y_f32)
      return Q.ck_bits > 0 ? launch_tiles<FMT, GROUP, BF16, NT, POST, true, false>(Q, tm_w, tm_x, tiles, dev, s)
                           : launch_tiles<FMT, GROUP, BF16, NT, POST, false, false>(Q, tm_w, tm_x, tiles, dev, s);
  }
  return Q.ck_bits > 0 ? launch_tiles<FMT, GROUP, BF16, NT, POST, true, true>(Q, tm_w, tm_x, tiles, dev, s)
                       : launch_tiles<FMT, GROUP, BF16, NT, POST, false, true>(Q, tm_w, tm_x, tiles, dev, s);
}

template <int FMT, int GROUP, bool BF16, bool POST = kPost<FMT, BF16>>
cudaError_t launch_tokens(const LinearParams& P, const DeviceInfo& dev, int32_t* status, cudaStream_t s) {
  if (P.T <= 32) return launch<FMT, GROUP, BF16, 32, POST>(P, dev, status, s);
  if (P.T <= 64) return launch<FMT, GROUP, BF16, 64, POST>(P, dev, status, s);
  return launch<FMT, GROUP, BF16, 128, POST>(P, dev, status, s);
}

}  // namespace w4tc
}  // namespace moe
