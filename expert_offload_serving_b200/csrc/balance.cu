// The balance loss with its per-expert counts, and the router's gradient.
//
// With f = counts and P = the mean softmax probability of a sequence,
//   loss[0] = 1/S' sum_s E/(k n_s) sum_e f_e P_e,   loss[1] = 1/n sum_t lse_t^2,
//   dlogits = dloss[0] coef_s p (f - <f, p>) + dloss[1] 2 coef_S lse p
//           + (on the chosen experts) gate (dgate - <gate, dgate>).
//
// Forward: one pass over the logits.  The tokens are cut into tiles, one CTA
// each; a warp holds a token's E logits in registers (lane l: experts l, l+32,
// ...) and adds its probabilities to running sums in registers.  A tile writes
// one partial per sequence that it touches, at row (tile + sequence): both grow
// along the tokens, so the rows are distinct and those of one sequence are
// consecutive.  A second kernel adds them up, one CTA per (sequence, 32
// experts), and its last CTA forms the loss.  Every sum has a fixed order; the
// atomics only count (integers) or hand out tickets.
//
// Few tokens of one sequence: one CTA does it all (5.3 us at T = 64, E = 128, k = 8);
// the latency of its steps bounds it.  T = 50000, E = 256, k = 6 in 29 sequences, a tenth
// masked: 22.7 us (2.1 TB/s) on inputs in turn, 20.7 on the same ones, some 13 in the
// first kernel, bound by instructions (a softmax and the sums of 8 values a lane), the
// rest the second one's chain of dependent loads.  Cut into 592 tiles 23.9 us, 296 25.9, 1184 24.2 (with the calls'
// gaps).
//
// Backward: one warp per token, nothing kept from the forward but counts and
// coef: the softmax is formed again from the logits, which costs no traffic
// (the row is read anyway): 4 E bytes in, 4 E out per token.  T = 50000, E = 256:
// 28.6 us on inputs in turn, 3.5 TB/s (25 on the same ones); instructions bound it (2.5
// a clock of an SM), HBM's share is 15.
// 4 tokens a warp; 2 took as long, 1 and 8 13 % longer.
#include <climits>
#include <cmath>
#include <type_traits>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxTiles = 592;      // 4 CTAs on each of 148 SMs
constexpr int kMaxS = 1 << 20;

struct BalanceLayout {
  int tile_tokens, tiles, eblocks;
  size_t rows, p, c, n, z, q, sn, sz, ticket, bytes;
};

BalanceLayout balance_layout(int T, int E, int S) {
  BalanceLayout L{};
  int C = (T + kMaxTiles - 1) / kMaxTiles;
  C = ((C < 1 ? 1 : C) + kWarps - 1) / kWarps * kWarps;
  L.tile_tokens = C;
  L.tiles = T > 0 ? (T + C - 1) / C : 1;
  L.eblocks = (E + 31) / 32;
  L.rows = static_cast<size_t>(L.tiles) + S;
  size_t at = 0;
  auto take = [&at](size_t bytes) {
    const size_t o = at;
    at += (bytes + 15) / 16 * 16;
    return o;
  };
  L.p = take(L.rows * E * 4);
  L.c = take(L.rows * E * 4);
  L.n = take(L.rows * 4);
  L.z = take(L.rows * 4);
  L.q = take(static_cast<size_t>(S) * L.eblocks * 8);
  L.sn = take(static_cast<size_t>(S) * 4);
  L.sz = take(static_cast<size_t>(S) * 8);
  L.ticket = take(4);
  L.bytes = at;
  return L;
}

struct BalanceWs {
  float* p;        // [rows][E] sums of probabilities
  int32_t* c;      // [rows][E] pairs
  int32_t* n;      // [rows] tokens
  float* z;        // [rows] sums of lse^2
  double* q;       // [S][eblocks] sums of counts * sum of probabilities
  int32_t* sn;     // [S]
  double* sz;      // [S]
  unsigned* ticket;
};

__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// Offset i, kept within [0, T] so that no bad value leads an access astray.
__device__ __forceinline__ int offset_at(const int32_t* off, int i, int T) {
  const int v = __ldg(off + i);
  return v < 0 ? 0 : (v > T ? T : v);
}

// The first sequence that ends after token t (S if none): the one that holds t, if
// any does.  A whole warp looks, at 32 offsets at a time.
__device__ __forceinline__ int sequence_of(const int32_t* off, int S, int T, int t, int lane) {
  int lo = 0, hi = S;                            // the answer lies in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const unsigned m = __ballot_sync(kFull, offset_at(off, min(lo + lane * step + step, hi), T) > t);
    if (m == 0) return hi;
    const int first = __ffs(m) - 1;
    hi = min(lo + first * step + step, hi) - 1;
    lo += first * step;
  }
  return hi;
}

// The expert of value j on a lane.  VEC: four consecutive experts a lane, in
// rounds of 128 (rows read and written 16 bytes at a time), else one in rounds
// of 32.
template <bool VEC>
__device__ __forceinline__ int expert_of(int j, int lane) {
  return VEC ? (j >> 2) * 128 + lane * 4 + (j & 3) : j * 32 + lane;
}

template <int VPL, bool VEC, typename V>
__device__ __forceinline__ void load_row(const V* __restrict__ row, int E, int lane, V none, V (&v)[VPL]) {
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < VPL; j += 4) {
      const int e = expert_of<true>(j, lane);
      const int4 x = e < E ? __ldg(reinterpret_cast<const int4*>(row + e)) : make_int4(0, 0, 0, 0);
      const V* xs = reinterpret_cast<const V*>(&x);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j + i] = e < E ? xs[i] : none;
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPL; ++j) v[j] = j * 32 + lane < E ? __ldg(row + j * 32 + lane) : none;
  }
}

// exp(l - top) through 2^x.  The rounded product is off by up to |x| 2^-24, so a
// value is off by |l - top| 2^-24 of itself: e^-16 (a value that adds 1e-7 to a
// sum) by 2^-20, and the large ones that make the sums by a few 2^-24.  (Values
// below 2^-126 are 0.)
__device__ __forceinline__ float exp_below(float l, float top) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"((l - top) * 1.4426950408889634f));
  return r;
}

// A row's maximum, 1 / sum of exp(l - max) and logsumexp; a row of nothing but
// -inf has inv = 0 and lse = 0 (and top 0, so that exp(l - top) is 0).
struct RowStat {
  float top, inv, lse;
};

// The softmax of a row held VPL values a lane: v becomes exp(l - max), the
// probabilities over inv.
template <int VPL>
__device__ __forceinline__ RowStat softmax_row(float (&v)[VPL]) {
  float top = v[0];
#pragma unroll
  for (int j = 1; j < VPL; ++j) top = fmaxf(top, v[j]);
  top = warp_max(top);
  const bool empty = top == -INFINITY;
  if (empty) top = 0.f;
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    v[j] = exp_below(v[j], top);
    sum += v[j];
  }
  sum = warp_sum(sum);
  RowStat r;
  r.top = top;
  r.inv = empty ? 0.f : __fdividef(1.f, sum);       // 1 <= sum <= E: within 2^-23 and 2^-21
  // log in full: a z-loss drives lse to 0, where __logf's 2^-21 would be all of it
  r.lse = empty ? 0.f : top + logf(sum);
  return r;
}

// What a warp gathers over its tokens of one sequence.
template <int VPL>
struct Gathered {
  float acc[VPL], z;
  int n;
};

// The tokens lo <= t < hi that count: probabilities into registers, pairs into the
// CTA's histogram.  A warp takes every `warps`-th group of G tokens, finds by a
// ballot which of them count, and works on two at a time (whose rows are in
// flight together; an odd last one stands in for its missing partner, at weight 0).
template <int VPL, bool VEC>
__device__ __forceinline__ Gathered<VPL> gather_tokens(const float* __restrict__ logits, int E,
                                                       const int32_t* __restrict__ idx, int k,
                                                       const uint8_t* __restrict__ mask, int lo, int hi, int warp,
                                                       int warps, int lane, int* hist, int32_t* status) {
  constexpr int R = VPL <= 8 ? 2 : 1;            // rows in flight: registers
  Gathered<VPL> r;
  r.z = 0.f;
  r.n = 0;
#pragma unroll
  for (int j = 0; j < VPL; ++j) r.acc[j] = 0.f;
  const int G = max(1, min(32, (hi - lo + warps - 1) / warps));
  for (int t0 = lo + warp * G; t0 < hi; t0 += warps * G) {
    const int mine = t0 + lane;
    unsigned m = __ballot_sync(kFull, lane < G && mine < hi && (mask == nullptr || __ldg(mask + mine) != 0));
    r.n += __popc(m);
    while (m != 0) {
      float v[R][VPL], w[R];
      int e[R], t = 0;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        w[i] = m != 0 ? 1.f : 0.f;
        if (m != 0) t = t0 + __ffs(m) - 1;
        m &= m - 1;
        load_row<VPL, VEC>(logits + static_cast<size_t>(t) * E, E, lane, -INFINITY, v[i]);
        e[i] = lane < k ? __ldg(idx + static_cast<size_t>(t) * k + lane) : 0;
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (lane < k && w[i] != 0.f) {
          if (e[i] >= 0 && e[i] < E) atomicAdd(&hist[e[i]], 1);
          else report(status, MOE_ERR_DEVICE);
        }
        const RowStat st = softmax_row<VPL>(v[i]);
        const float inv = w[i] * st.inv;
#pragma unroll
        for (int j = 0; j < VPL; ++j) r.acc[j] = fmaf(v[i][j], inv, r.acc[j]);
        r.z = fmaf(w[i] * st.lse, st.lse, r.z);
      }
    }
  }
  return r;
}

template <int VPL, bool VEC>
__global__ void __launch_bounds__(kThreads) balance_partial_kernel(
    const float* __restrict__ logits, int T, int E, const int32_t* __restrict__ idx, int k,
    const int32_t* __restrict__ seq, int S, const uint8_t* __restrict__ mask, int tile_tokens, BalanceWs ws,
    int32_t* status) {
  extern __shared__ float smem[];
  float* wsum = smem;                                        // [kWarps][E]
  int* hist = reinterpret_cast<int*>(smem + kWarps * E);     // [E]
  __shared__ float wz[kWarps];
  __shared__ int wn[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = threadIdx.x; e < E; e += kThreads) hist[e] = 0;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x == 0) *ws.ticket = 0;
  const int t0 = blockIdx.x * tile_tokens;
  const int t1 = min(T, t0 + tile_tokens);
  for (int s = seq == nullptr ? 0 : sequence_of(seq, S, T, t0, lane); s < S; ++s) {
    const int a = seq == nullptr ? 0 : offset_at(seq, s, T), b = seq == nullptr ? T : offset_at(seq, s + 1, T);
    if (a >= t1) break;
    const int lo = max(a, t0), hi = min(b, t1);
    if (lo >= hi) continue;
    __syncthreads();                                         // hist is clear, wsum may be written
    const Gathered<VPL> r =
        gather_tokens<VPL, VEC>(logits, E, idx, k, mask, lo, hi, warp, kWarps, lane, hist, status);
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (expert_of<VEC>(j, lane) < E) wsum[warp * E + expert_of<VEC>(j, lane)] = r.acc[j];
    if (lane == 0) {
      wz[warp] = r.z;
      wn[warp] = r.n;
    }
    __syncthreads();
    const size_t row = static_cast<size_t>(blockIdx.x) + s;
    for (int e = threadIdx.x; e < E; e += kThreads) {
      float p = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) p += wsum[w * E + e];
      ws.p[row * E + e] = p;
      ws.c[row * E + e] = hist[e];
      hist[e] = 0;
    }
    if (threadIdx.x == 0) {
      float zs = 0.f;
      int ns = 0;
      for (int w = 0; w < kWarps; ++w) {
        zs += wz[w];
        ns += wn[w];
      }
      ws.z[row] = zs;
      ws.n[row] = ns;
    }
  }
}

// Sum over the block in a fixed order; every thread gets it.
template <typename V>
__device__ V block_sum(V v, V* sh) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  V s = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) s += sh[w];
  return s;
}

// One CTA does it all where one sequence has few tokens: a second launch would cost
// more than the whole sum.  Device time in us, one CTA / two kernels:
//            T = 16      T = 48      T = 64      T = 96      T = 128     T = 160
//   E = 64   4.6 / 6.7   4.8 / 6.1   5.0 / 6.2   5.9 / 6.6   6.0 / 7.1   6.9 / 7.7
//   E = 256  5.2 / 7.3   5.5 / 7.3   5.8 / 7.4   7.1 / 7.6   7.2 / 7.6   8.4 / 8.0
//   E = 512  3.5 / 7.6   5.7 / 7.6   6.8 / 7.7   8.8 / 7.9    11 / 7.8    13 / 8.3
//   E = 1000 5.0 / 8.7   8.1 / 8.8   9.4 / 8.8    12 / 9.1    16 / 8.8    19 / 9.2
// Several sequences go to two kernels: one CTA that walked them took a chain each (64
// tokens, E = 128: in 2 sequences 10.6 against 8.6 us, in 16 67 against 12.4, in 128
// 479 against 17.7).
bool small_batch(int T, int E, int S) { return S == 1 && T <= (E <= 256 ? 128 : E <= 512 ? 64 : 48); }

template <int VPL, bool VEC>
__global__ void __launch_bounds__(VPL <= 8 ? 1024 : kThreads) balance_small_kernel(
    const float* __restrict__ logits, int T, int E, const int32_t* __restrict__ idx, int k,
    const int32_t* __restrict__ seq, const uint8_t* __restrict__ mask, float* __restrict__ loss,
    int32_t* __restrict__ counts, float* __restrict__ prob, float* __restrict__ coef, int32_t* status) {
  extern __shared__ float smem[];
  const int threads = blockDim.x, warps = threads >> 5;
  float* wsum = smem;                                        // [warps][E]
  int* hist = reinterpret_cast<int*>(smem + warps * E);      // [E]
  __shared__ float wz[32];
  __shared__ int wn[32];
  __shared__ double shd[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = threadIdx.x; e < E; e += threads) hist[e] = 0;
  pdl_wait();
  pdl_trigger();
  int a = 0, b = T;
  if (seq != nullptr) {
    a = offset_at(seq, 0, T);
    b = offset_at(seq, 1, T);
    if (threadIdx.x == 0 && (a > b || a != __ldg(seq) || b != __ldg(seq + 1))) report(status, MOE_ERR_DEVICE);
  }
  __syncthreads();                                           // hist is clear
  const Gathered<VPL> r = gather_tokens<VPL, VEC>(logits, E, idx, k, mask, a, b, warp, warps, lane, hist, status);
#pragma unroll
  for (int j = 0; j < VPL; ++j)
    if (expert_of<VEC>(j, lane) < E) wsum[warp * E + expert_of<VEC>(j, lane)] = r.acc[j];
  if (lane == 0) {
    wz[warp] = r.z;
    wn[warp] = r.n;
  }
  __syncthreads();
  double z = 0, q = 0;
  int n = 0;
  for (int w = 0; w < warps; ++w) {
    z += wz[w];
    n += wn[w];
  }
  for (int e = threadIdx.x; e < E; e += threads) {
    double p = 0;
    for (int w = 0; w < warps; ++w) p += wsum[w * E + e];
    const int c = hist[e];
    counts[e] = c;
    prob[e] = n > 0 ? static_cast<float>(p / n) : 0.f;
    q += p * c;
  }
  q = block_sum(q, shd);
  if (threadIdx.x != 0) return;
  const double factor = n > 0 ? E / (static_cast<double>(k) * n * n) : 0.0;
  coef[0] = static_cast<float>(factor);
  coef[1] = 1.f / static_cast<float>(n > 0 ? n : 1);
  loss[0] = static_cast<float>(q * factor);
  loss[1] = n > 0 ? static_cast<float>(z / n) : 0.f;
}

__global__ void __launch_bounds__(kThreads) balance_finish_kernel(
    int T, int E, int k, const int32_t* __restrict__ seq, int S, int tile_tokens, int eblocks, BalanceWs ws,
    float* __restrict__ loss, int32_t* __restrict__ counts, float* __restrict__ prob, float* __restrict__ coef,
    int32_t* status) {
  __shared__ double wp[kWarps][32];
  __shared__ int wc[kWarps][32];
  __shared__ double wall[kWarps][4];
  __shared__ bool last;
  const int s = blockIdx.x, eb = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = eb * 32 + lane;
  pdl_wait();
  pdl_trigger();
  int a = 0, b = T;
  if (seq != nullptr) {
    a = offset_at(seq, s, T);
    b = offset_at(seq, s + 1, T);
    if (threadIdx.x == 0 && eb == 0 && (a > b || a != __ldg(seq + s) || b != __ldg(seq + s + 1)))
      report(status, MOE_ERR_DEVICE);
  }
  // the rows of this sequence (none if it is empty)
  const size_t r0 = static_cast<size_t>(a / tile_tokens) + s;
  const int rows = a < b ? (b - 1) / tile_tokens - a / tile_tokens + 1 : 0;
  double p = 0, z = 0;
  int c = 0, n = 0;
  if (e < E)
#pragma unroll 4
    for (int r = warp; r < rows; r += kWarps) {
      p += ws.p[(r0 + r) * E + e];
      c += ws.c[(r0 + r) * E + e];
    }
  if (warp == 0)
    for (int r = lane; r < rows; r += 32) {
      n += ws.n[r0 + r];
      z += ws.z[r0 + r];
    }
  wp[warp][lane] = p;
  wc[warp][lane] = c;
  __syncthreads();
  if (warp == 0) {
    n = warp_sum(n);
    p = 0;
    c = 0;
    for (int w = 0; w < kWarps; ++w) {
      p += wp[w][lane];
      c += wc[w][lane];
    }
    if (e < E) {
      counts[static_cast<size_t>(s) * E + e] = c;
      prob[static_cast<size_t>(s) * E + e] = n > 0 ? static_cast<float>(p / n) : 0.f;
    }
    const double q = warp_sum(e < E ? p * c : 0.0);
    if (eb == 0) z = warp_sum(z);
    if (lane == 0) {
      ws.q[static_cast<size_t>(s) * eblocks + eb] = q;
      if (eb == 0) {
        ws.sn[s] = n;
        ws.sz[s] = z;
      }
      __threadfence();
      last = atomicAdd(ws.ticket, 1u) == static_cast<unsigned>(S) * eblocks - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  // The last CTA: every other one's sums are visible.  all[]: sequences with
  // tokens, tokens (whole numbers, exact in 64 bits), lse^2, balance terms.
  double all[4] = {0, 0, 0, 0};
  for (int i = threadIdx.x; i < S; i += kThreads) {
    const int ni = __ldcg(ws.sn + i);
    double q = 0;
    for (int j = 0; j < eblocks; ++j) q += __ldcg(ws.q + static_cast<size_t>(i) * eblocks + j);
    all[0] += ni > 0;
    all[1] += ni;
    all[2] += __ldcg(ws.sz + i);
    if (ni > 0) all[3] += q * E / (static_cast<double>(k) * ni * ni);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    all[i] = warp_sum(all[i]);
    if (lane == 0) wall[warp][i] = all[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    all[i] = 0;
    for (int w = 0; w < kWarps; ++w) all[i] += wall[w][i];
  }
  for (int i = threadIdx.x; i < S; i += kThreads) {
    const int ni = __ldcg(ws.sn + i);
    coef[i] = ni > 0 ? static_cast<float>(E / (static_cast<double>(k) * ni * ni * all[0])) : 0.f;
  }
  if (threadIdx.x == 0) {
    coef[S] = static_cast<float>(1.0 / (all[1] > 0 ? all[1] : 1.0));
    loss[0] = all[0] > 0 ? static_cast<float>(all[3] / all[0]) : 0.f;
    loss[1] = all[1] > 0 ? static_cast<float>(all[2] / all[1]) : 0.f;
  }
}

// `rows` consecutive tokens a warp.
template <int VPL, bool VEC>
__global__ void __launch_bounds__(kThreads) router_backward_kernel(
    const float* __restrict__ logits, int T, int E, const int32_t* __restrict__ idx, const float* __restrict__ gate,
    const float* __restrict__ dgate, int k, const int32_t* __restrict__ seq, int S, const uint8_t* __restrict__ mask,
    const int32_t* __restrict__ counts, const float* __restrict__ coef, const float* __restrict__ dloss,
    float* __restrict__ dlogits, int rows, int32_t* status) {
  const int lane = threadIdx.x & 31;
  const long long first = ((blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x) >> 5) * rows;
  pdl_wait();
  pdl_trigger();
  if (first >= T) return;
  const int end = static_cast<int>(min(first + rows, static_cast<long long>(T)));
  const bool with_loss = dloss != nullptr, with_gates = dgate != nullptr, on = lane < k;
  const float dl = with_loss ? __ldg(dloss) : 0.f, dz = with_loss ? 2.f * __ldg(dloss + 1) * __ldg(coef + S) : 0.f;
  int s = 0, seq_begin = 0, seq_end = 0;          // the sequence that ends first behind the token
  float cb0 = 0.f;
  if (seq == nullptr) {
    seq_end = T;
    if (with_loss) cb0 = dl * __ldg(coef);
  }
  const int t0 = static_cast<int>(first);
  const unsigned counted =
      mask == nullptr ? ~0u : __ballot_sync(kFull, t0 + lane < end && __ldg(mask + t0 + lane) != 0);   // rows <= 32
  for (int t = t0; t < end; ++t) {
    float* row = dlogits + static_cast<size_t>(t) * E;
    bool live = counted >> (t - t0) & 1u;
    if (t >= seq_end) {                           // seq != nullptr
      s = sequence_of(seq, S, T, t, lane);
      seq_begin = s < S ? offset_at(seq, s, T) : T;
      seq_end = s < S ? offset_at(seq, s + 1, T) : T;
      if (with_loss && s < S) cb0 = dl * __ldg(coef + s);
    }
    live = live && t >= seq_begin;
    if (!live) {
      for (int e = lane; e < E; e += 32) row[e] = 0.f;
      continue;
    }
    const float* lrow = logits + static_cast<size_t>(t) * E;
    const int32_t* crow = counts + static_cast<size_t>(s) * E;
    float d[VPL];
    // the pairs of the token, one a lane
    float g = 0.f, dg = 0.f;
    int e = -1;
    if (with_loss) load_row<VPL, VEC>(lrow, E, lane, -INFINITY, d);
    if (with_gates && on) {
      const size_t p = static_cast<size_t>(t) * k + lane;
      g = __ldg(gate + p);
      dg = __ldg(dgate + p);
      e = __ldg(idx + p);
      if (e < 0 || e >= E) {
        report(status, MOE_ERR_DEVICE);
        e = -1;
      }
    }
    RowStat st{0.f, 0.f, 0.f};
    float dot = 0.f, cz = 0.f;
    if (with_loss) {
      int32_t f[VPL];
      load_row<VPL, VEC>(crow, E, lane, 0, f);
      st = softmax_row<VPL>(d);
      cz = dz * st.lse;
#pragma unroll
      for (int j = 0; j < VPL; ++j) dot = fmaf(static_cast<float>(f[j]), d[j], dot);
      dot = warp_sum(dot) * st.inv;
      // p (cb (f - dot) + cz) with p = d inv
      const float cb = cb0 * st.inv, c0 = cz * st.inv - cb * dot;
#pragma unroll
      for (int j = 0; j < VPL; ++j) d[j] *= fmaf(cb, static_cast<float>(f[j]), c0);
    } else {
#pragma unroll
      for (int j = 0; j < VPL; ++j) d[j] = 0.f;
    }
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < VPL; j += 4)
        if (expert_of<true>(j, lane) < E)
          *reinterpret_cast<float4*>(row + expert_of<true>(j, lane)) = make_float4(d[j], d[j + 1], d[j + 2], d[j + 3]);
    } else {
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (j * 32 + lane < E) row[j * 32 + lane] = d[j];
    }
    if (!with_gates) continue;
    // The chosen experts' values again, by their pairs' lanes, with the gate term:
    // k values to form and store over those above instead of a search for each of
    // the k experts' owners.  An id that occurs twice is summed by its first lane.
    const float v = g * (dg - warp_sum(g * dg));
    const unsigned same = __match_any_sync(kFull, e);
    float sum = v;
    if (__any_sync(kFull, e >= 0 && __popc(same) > 1)) {
      sum = 0.f;
      for (int i = 0; i < k; ++i) {
        const float vi = __shfl_sync(kFull, v, i);
        if (same >> i & 1u) sum += vi;
      }
    }
    __syncwarp();
    if (e >= 0 && __ffs(same) - 1 == lane) {
      float x = 0.f;
      if (with_loss)
        x = exp_below(__ldg(lrow + e), st.top) * st.inv * fmaf(cb0, static_cast<float>(__ldg(crow + e)) - dot, cz);
      row[e] = x + sum;
    }
  }
}

moe_status check_sequences(int T, int E, int k, const int32_t* seq, int S) {
  MOE_REQUIRE(T >= 0, "T=%d < 0", T);
  MOE_REQUIRE(E >= 1 && E <= 1024, "E=%d outside [1, 1024]", E);
  MOE_REQUIRE(k >= 1 && k <= E && k <= 32, "k=%d outside [1, min(E, 32)]", k);
  MOE_REQUIRE(T <= (1 << 24) / k, "T*k too large");
  MOE_REQUIRE(S >= 1 && S <= kMaxS, "S=%d outside [1, %d]", S, kMaxS);
  MOE_REQUIRE(seq != nullptr || S == 1, "S=%d sequences need seq_offsets", S);
  MOE_REQUIRE(aligned(seq, 4), "misaligned seq_offsets");
  return MOE_OK;
}

// f(VPL, VEC): the number of experts a lane holds for E experts, and whether rows
// are moved 16 bytes at a time.
template <typename F>
cudaError_t with_row(int E, bool vec, F f) {
  const std::true_type yes;
  const std::false_type no;
  if (E <= 32) return f(std::integral_constant<int, 1>(), no);
  if (E <= 64) return f(std::integral_constant<int, 2>(), no);
  if (E <= 128) return vec ? f(std::integral_constant<int, 4>(), yes) : f(std::integral_constant<int, 4>(), no);
  if (E <= 256) return vec ? f(std::integral_constant<int, 8>(), yes) : f(std::integral_constant<int, 8>(), no);
  if (E <= 512) return vec ? f(std::integral_constant<int, 16>(), yes) : f(std::integral_constant<int, 16>(), no);
  return vec ? f(std::integral_constant<int, 32>(), yes) : f(std::integral_constant<int, 32>(), no);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_balance_loss_workspace_bytes(int T, int E, int S) {
  if (T < 0 || T > (1 << 24) || E < 1 || E > 1024 || S < 1 || S > kMaxS) return 0;
  return balance_layout(T, E, S).bytes;
}

extern "C" moe_status moe_balance_loss(const float* logits, int T, int E, const int32_t* idx, int k,
                                       const int32_t* seq_offsets, int S, const uint8_t* mask, float* loss,
                                       int32_t* counts, float* prob, float* coef, void* workspace, size_t ws_bytes,
                                       int32_t* dev_status, cudaStream_t stream) {
  clear_error();
  moe_status st = check_sequences(T, E, k, seq_offsets, S);
  if (st != MOE_OK) return st;
  MOE_REQUIRE(loss && counts && prob && coef && workspace && (T == 0 || (logits && idx)), "null pointer");
  MOE_REQUIRE(aligned(logits, 4) && aligned(idx, 4) && aligned(loss, 4) && aligned(counts, 4) && aligned(prob, 4) &&
                  aligned(coef, 4), "misaligned pointer");
  MOE_REQUIRE(aligned(workspace, 16), "workspace must be 16-byte aligned");
  const BalanceLayout L = balance_layout(T, E, S);
  if (ws_bytes < L.bytes)
    return fail(MOE_ERR_CAPACITY, "moe_balance_loss needs %zu bytes of workspace, got %zu", L.bytes, ws_bytes);
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != MOE_OK) return st;
  char* w = static_cast<char*>(workspace);
  BalanceWs ws;
  ws.p = reinterpret_cast<float*>(w + L.p);
  ws.c = reinterpret_cast<int32_t*>(w + L.c);
  ws.n = reinterpret_cast<int32_t*>(w + L.n);
  ws.z = reinterpret_cast<float*>(w + L.z);
  ws.q = reinterpret_cast<double*>(w + L.q);
  ws.sn = reinterpret_cast<int32_t*>(w + L.sn);
  ws.sz = reinterpret_cast<double*>(w + L.sz);
  ws.ticket = reinterpret_cast<unsigned*>(w + L.ticket);
  const bool vec = E % 4 == 0 && aligned(logits, 16);
  if (small_batch(T, E, S)) {
    const int warps = E <= 256 ? 32 : kWarps;   // registers: VPL <= 8 values a lane, or more
    const cudaError_t err = with_row(E, vec, [&](auto vpl, auto v) {
      return launch_pdl(balance_small_kernel<decltype(vpl)::value, decltype(v)::value>, dim3(1), dim3(warps * 32),
                        static_cast<size_t>(warps + 1) * E * 4, stream, logits, T, E, idx, k, seq_offsets, mask, loss,
                        counts, prob, coef, dev_status);
    });
    if (err != cudaSuccess) return fail(MOE_ERR_CUDA, "balance_small launch: %s", cudaGetErrorString(err));
    MOE_LAUNCH_CHECK("balance_small_kernel");
    return MOE_OK;
  }
  const size_t smem = static_cast<size_t>(kWarps + 1) * E * 4;     // <= 36 KB
  const cudaError_t err = with_row(E, vec, [&](auto vpl, auto v) {
    return launch_pdl(balance_partial_kernel<decltype(vpl)::value, decltype(v)::value>, dim3(L.tiles), dim3(kThreads),
                      smem, stream, logits, T, E, idx, k, seq_offsets, S, mask, L.tile_tokens, ws, dev_status);
  });
  if (err != cudaSuccess) return fail(MOE_ERR_CUDA, "balance_partial launch: %s", cudaGetErrorString(err));
  MOE_CUDA_TRY(launch_pdl(balance_finish_kernel, dim3(S, L.eblocks), dim3(kThreads), 0, stream, T, E, k, seq_offsets, S,
                          L.tile_tokens, L.eblocks, ws, loss, counts, prob, coef, dev_status));
  MOE_LAUNCH_CHECK("balance_finish_kernel");
  return MOE_OK;
}

extern "C" moe_status moe_router_backward(const float* logits, int T, int E, const int32_t* idx, const float* gate,
                                          const float* dgate, int k, const int32_t* seq_offsets, int S,
                                          const uint8_t* mask, const int32_t* counts, const float* coef,
                                          const float* dloss, float* dlogits, int32_t* dev_status,
                                          cudaStream_t stream) {
  clear_error();
  moe_status st = check_sequences(T, E, k, seq_offsets, S);
  if (st != MOE_OK || T == 0) return st;
  MOE_REQUIRE(dlogits != nullptr, "null dlogits");
  MOE_REQUIRE(dloss == nullptr || (logits && counts && coef), "dloss needs logits, counts and coef");
  MOE_REQUIRE(dgate == nullptr || (idx && gate), "dgate needs idx and gate");
  MOE_REQUIRE(aligned(logits, 4) && aligned(idx, 4) && aligned(gate, 4) && aligned(dgate, 4) && aligned(counts, 4) &&
                  aligned(coef, 4) && aligned(dloss, 4) && aligned(dlogits, 4), "misaligned pointer");
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != MOE_OK) return st;
  // One token a warp until every warp slot of the SMs (about 40 each) has had one,
  // then up to 4: what a warp reads once counts for more rows.
  int rows = T / (40 * dev.sm_count);
  rows = rows < 1 ? 1 : rows > 4 ? 4 : rows;
  const int blocks = (T + kWarps * rows - 1) / (kWarps * rows);
  const bool vec = E % 4 == 0 && aligned(logits, 16) && aligned(dlogits, 16) && aligned(counts, 16);
  const cudaError_t err = with_row(E, vec, [&](auto vpl, auto v) {
    return launch_pdl(router_backward_kernel<decltype(vpl)::value, decltype(v)::value>, dim3(blocks), dim3(kThreads), 0,
                      stream, logits, T, E, idx, gate, dgate, k, seq_offsets, S, mask, counts, coef, dloss, dlogits,
                      rows, dev_status);
  });
  if (err != cudaSuccess) return fail(MOE_ERR_CUDA, "router_backward launch: %s", cudaGetErrorString(err));
  return MOE_OK;
}
