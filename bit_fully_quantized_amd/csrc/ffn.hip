// The gated feed-forward block for gfx950 in bf16:
//
//   G = X Wg^T, U = X Wu^T, H = act(G) * U, Y = H Wd^T,
//   dH = dY Wd, dG = dH U act'(G), dU = dH act(G),
//   dX = dG Wg + dU Wu, dWg = dG^T X, dWu = dU^T X, dWd = dY^T H.
//
// Both projections are one tile product whose tiles hold as many rows of either weight
// (EL_PAIR), so a lane has a gate and its factor together and the activation and the
// product cost no pass of their own; G and U are written only for a backward pass.  There
// the product dH has an epilogue that reads G and U and writes dG and dU in the two
// layouts that the four products after it read, and H transposed; those four run in one
// launch.  Sums and the activation are fp32; H, dG and dU are rounded to bf16, the type of
// the operands, where a product takes them.  G and U are kept in 24 bits (fp32's sign,
// exponent and 15 bits): in bf16 their rounding would enter dX and dW as much as that of
// dG and dU does (3.0e-3 of dX's norm in all instead of 2.4e-3, 3.5e-3 of dWd's), and f16
// would not hold what bf16 activations reach.
#include <math.h>

#include <algorithm>
#include <array>
#include <cfloat>
#include <mutex>

#include "tj2_bf16.h"

namespace tj2 {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;

struct Act {
  float a, d;  // act(g), act'(g)
};
// v, or g's NaN, which a median with two numbers below drops
__device__ __forceinline__ float or_nan(float g, float v) { return g != g ? g : v; }
template <int ACT>
__device__ __forceinline__ Act activate(float g) {
  if constexpr (ACT == TJ2_SILU) {
    const float p = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * g));
    return {g * p, p * fmaf(g, 1.0f - p, 1.0f)};
  } else if constexpr (ACT == TJ2_GELU) {
    // g Phi(g).  The tail Phi(-|g|) is exp(-g^2 / 2), which the slope needs too, times a
    // function that varies slowly, t times a polynomial of degree 7 in t = 1 / (1 + 0.43 |g| /
    // sqrt 2): a fit to 1e-7 of itself, 7e-7 in fp32 for |g| < 4 (the library's erfc took most
    // of these kernels' time: 1235 x 528, 1552 features, backward kernel 25.0 us, and
    // 20.0 so).  From |g| = 14 on the exponential is 0 and the arguments are kept finite.
    const float c = __builtin_amdgcn_fmed3f(g, -14.0f, 14.0f), t = __builtin_amdgcn_rcpf(fmaf(0.304055929f, fabsf(c), 1.0f));
    const float e = __builtin_amdgcn_exp2f(-0.5f * kLog2e * c * c);
    float q = 0.0368549079f;
    q = fmaf(q, t, -0.155190811f);
    q = fmaf(q, t, 0.191860318f);
    q = fmaf(q, t, -0.0428701229f);
    q = fmaf(q, t, 0.123426266f);
    q = fmaf(q, t, 0.10247425f);
    q = fmaf(q, t, 0.122187942f);
    q = fmaf(q, t, 0.12125729f);
    q = q * t * e;
    const float p = g < 0.0f ? q : 1.0f - q;
    return {g * p, or_nan(g, fmaf(c * 0.39894228040143267794f, e, p))};
  } else {
    // (1 + tanh z) / 2 is the logistic function of 2 z; where it is 0 or 1, so is its
    // slope 0, and the polynomial is kept finite
    const float c = __builtin_amdgcn_fmed3f(g, -64.0f, 64.0f);
    const float k = 1.59576912160573071176f, z = k * fmaf(0.044715f * c * c, c, c);
    const float p = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * z));
    return {g * p, or_nan(g, fmaf(c * p * (1.0f - p), k * fmaf(0.134145f * c, c, 1.0f), p))};
  }
}

// G and U as the backward pass reads them: the upper 16 bits of fp32 of both, then the next
// 8 of both, rounded to the nearest (a NaN stays one: it is made a quiet one), in blocks of
// 64 tokens by 64 features, in them in the order in which a wave of the backward kernel
// holds them: 8 features of a lane (n + 16 g: tokens 4 n to 4 n + 3, features 16 g to 16 g +
// 15), lane after lane.  (Row by row, features of 64 tokens lie as far apart as a power of
// two and meet in one channel of the L2: 16384 x 1024, 4096 features, forward kernel 334 us,
// backward kernel 433.)
struct Saved {
  uint16_t *g, *u;
  uint8_t *gl, *ul;
  int64_t nf;  // chunks of 64 features
  __device__ __forceinline__ int64_t at(int64_t t, int64_t f) const {
    const int n = (int)(t >> 2) & 15, tn = (int)t & 3, g = (int)(f >> 4) & 3, half = (int)(f >> 3) & 1;
    return ((t >> 6) * nf + (f >> 6)) * 4096 + ((tn * 2 + half) * 64 + g * 16 + n) * 8 + (f & 7);
  }
};
__device__ __forceinline__ uint32_t round24(float v) {
  const uint32_t b = __float_as_uint(v);
  return v != v ? b | 0x00400000u : b + 0x80u;
}
template <int N>  // 2 or 8 neighbours
__device__ __forceinline__ void save24(uint16_t* hi, uint8_t* lo, const float* v) {
  uint32_t h[N / 2], l[(N + 3) / 4];
#pragma unroll
  for (int k = 0; k < N; k += 2) {
    const uint32_t a = round24(v[k]), b = round24(v[k + 1]);
    h[k / 2] = __builtin_amdgcn_perm(b, a, 0x07060302u);
    const uint32_t two = __builtin_amdgcn_perm(b, a, 0x0C0C0501u);
    l[k / 4] = k % 4 ? l[k / 4] | two << 16 : two;
  }
  if constexpr (N == 2) {
    *reinterpret_cast<uint32_t*>(hi) = h[0];
    *reinterpret_cast<uint16_t*>(lo) = (uint16_t)l[0];
  } else {
#pragma unroll
    for (int k = 0; k < N; k += 8) {
      *reinterpret_cast<uint4*>(hi + k) = uint4{h[k / 2], h[k / 2 + 1], h[k / 2 + 2], h[k / 2 + 3]};
      *reinterpret_cast<uint2*>(lo + k) = uint2{l[k / 4], l[k / 4 + 1]};
    }
  }
}
// value k (0..7) of 8 neighbours
__device__ __forceinline__ float value24(const uint4& hi, const uint2& lo, int k) {
  const uint32_t h = k < 2 ? hi.x : k < 4 ? hi.y : k < 6 ? hi.z : hi.w, l = k < 4 ? lo.x : lo.y;
  // bytes: 0, l[k % 4], h's half k % 2
  return __uint_as_float(__builtin_amdgcn_perm(h, l, (k & 1 ? 0x07060000u : 0x05040000u) | (uint32_t)(k & 3) << 8 | 0x0Cu));
}

__device__ __forceinline__ uint4 pack8(const float* v) {
  return uint4{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
}

// ---- both projections, the activation and the product ----------------------------------
// A tile holds the same rows of Wg and Wu, so gate and factor meet in a lane.  16384 x 1024,
// 4096 features: 288 us with G and U saved (275 GFLOP: 0.95 PFLOP/s), 200 without (1.37).  A
// tile of 256 x 256 takes 16 chunks at 1.6 us and then writes 262 KB (196 of them G and U),
// which no products cover: the stores are waited for with the next tile's loads, in order.
// Workgroups that start apart and tiles of 128 (two on a CU) did not cover it either.
struct GateArgs {
  TileOp P, Q;       // P: Wg and Wu [F, D], Q: X [T, D]
  uint32_t tiles_p, tiles_q;
  int32_t nch, nf;   // nf: chunks of 64 features of H
  uint16_t* h;       // [T, F], blocked
  Saved s;           // for the backward pass, or NULL
};

template <class T, int ACT>
__global__ __launch_bounds__(T::NT, T::WAVES) void ffn_gate_kernel(GateArgs p) {
  static_assert(T::kTM == 2 * T::PB, "a lane's first PB tiles are gates");
  __shared__ __attribute__((aligned(128))) typename T::Smem sm;
  const typename T::Items items(p.tiles_p, p.tiles_q, (uint32_t)p.nch, 1);
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
  constexpr int N = 4 * T::PB;  // neighbouring features of a lane
  T::run(p.P, p.Q, items, sm, [&](int64_t p0, int64_t q0, uint32_t, typename T::Acc& acc) __attribute__((always_inline)) {
    const int64_t f = p0 / 2 + (w / T::kWN) * 16 * T::PB + g * N, t0 = q0 + (w % T::kWN) * T::kTN * 16;
    if (f >= p.P.rows) return;  // (F is a multiple of 16: a lane's features are all there or none is)
#pragma unroll
    for (int tn = 0; tn < T::kTN; ++tn) {
      const int64_t t = t0 + T::q_row(tn, n);
      if (t >= p.Q.rows) continue;
      float v[N];
      if (p.s.g) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
          for (int k = 0; k < N; ++k) v[k] = acc[half * T::PB + k / 4][tn][k % 4];
#pragma unroll
          for (int k = 0; k < N; k += 8) {
            const int64_t at = p.s.at(t, f + k);
            save24<8>((half ? p.s.u : p.s.g) + at, (half ? p.s.ul : p.s.gl) + at, v + k);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = activate<ACT>(acc[k / 4][tn][k % 4]).a * acc[T::PB + k / 4][tn][k % 4];
      uint16_t* o = p.h + ((t >> 7) * p.nf + (f >> 6)) * 8192 + (t & 127) * 64 + (f & 63);
#pragma unroll
      for (int k = 0; k < N; k += 8) *reinterpret_cast<uint4*>(o + k) = pack8(v + k);
    }
  });
}

// The same for up to 32 tokens: one read of the weights, 8 rows of each a wave (lane n
// holds a gate's row where n & 2 is 0), so that a lane's four results are two gates and
// their factors.  Bound by that read's latency and, from 2048 wide on, its rate: 1 token of D
// 1024, F 4096 5.6 us (16.8 MB, 3.0 TB/s).  H is row-major; of up to 8 tokens in two bf16 parts (8 bits, and the next of
// what these leave), since their results have few of H's roundings to average over and the
// second part takes places of the output product's instruction that are idle (a second
// instruction for 9 to 32 tokens would cost 2 to 7 us of 11 to 45).
constexpr int kTwoParts = 8;
struct GateFewArgs {
  const uint16_t *x, *wg, *wu;
  int64_t ldx, ldw;
  int32_t T, D, F;
  uint16_t* h;  // [1 or 2][T][F]
  Saved s;
};
// LDS bytes of a token: whole chunks and 16 bytes, so that 16 tokens' pieces lie in different banks
__host__ __device__ constexpr int64_t few_pitch(int64_t D) { return (D * 2 + 127) / 128 * 128 + 16; }
template <int TN, int ACT>
__global__ __launch_bounds__(256, 2) void ffn_gate_few_kernel(GateFewArgs p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t xs[];  // [T][few_pitch(D)]
  constexpr int U = 8;  // chunks of 64 features in flight
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int px = (int)few_pitch(p.D), pieces = (p.D + 63) / 64 * 8;
  const uint32_t groups = (uint32_t)(p.F + 7) / 8, per = blockDim.x >> 6, waves = gridDim.x * per, chunks = (uint32_t)(p.D + 63) / 64;
  struct Batch {
    i32x4_t a[U][2];
  };
  const uint16_t* wrow = (n & 2 ? p.wu : p.wg) + (2 * (n >> 2) + (n & 1)) * p.ldw + g * 16;
  auto fetch = [&](Batch& f, uint32_t gr, uint32_t c0) __attribute__((always_inline)) {
    const uint16_t* w = wrow + (int64_t)gr * 8 * p.ldw;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = (int)(c0 + u) * 64 + h * 8;
        f.a[u][h] = i32x4_t{0, 0, 0, 0};
        // (F is a multiple of 16: a group's rows are all there)
        if (gr < groups && k + g * 16 < p.D) f.a[u][h] = *reinterpret_cast<const i32x4_t*>(w + k);
      }
  };
  const uint8_t* xl[TN];  // (columns past the last token repeat it and are not stored)
#pragma unroll
  for (int tn = 0; tn < TN; ++tn) xl[tn] = xs + min(tn * 16 + n, p.T - 1) * px + g * 32;
  float4_t acc[TN] = {};
  auto multiply = [&](const Batch& f, uint32_t c0) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c0 + u >= chunks) break;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int tn = 0; tn < TN; ++tn)
          acc[tn] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8_t, f.a[u][h]),
              *reinterpret_cast<const bf16x8_t*>(xl[tn] + (c0 + u) * 128 + h * 16), acc[tn], 0, 0, 0);
    }
  };
  uint32_t gr = blockIdx.x * per + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = 0;
  Batch f0, f1;
  fetch(f0, gr, 0);
  // the tokens, while the first weights are on their way
  for (int i = threadIdx.x; i < p.T * pieces; i += blockDim.x) {
    const int t = i / pieces, k = (i - t * pieces) * 8;
    uint4 v = {0u, 0u, 0u, 0u};
    if (k < p.D) v = *reinterpret_cast<const uint4*>(p.x + t * p.ldx + k);
    *reinterpret_cast<uint4*>(xs + t * px + k * 2) = v;
  }
  __syncthreads();
  if (gr >= groups) return;
  auto turn = [&](const Batch& now, Batch& next) __attribute__((always_inline)) -> bool {
    const bool last = c + U >= chunks;
    const uint32_t ng = last ? gr + waves : gr, nc = last ? 0 : c + U;
    fetch(next, ng, nc);
    multiply(now, c);
    if (last) {
      const int64_t f = (int64_t)gr * 8 + 2 * g;
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) {
        const int t = tn * 16 + n;
        if (t < p.T) {
          const float4_t v = acc[tn];
          const float h0 = activate<ACT>(v.x).a * v.z, h1 = activate<ACT>(v.y).a * v.w;
          const uint32_t hi = bf16_pair(h0, h1);
          uint16_t* o = p.h + (int64_t)t * p.F + f;
          *reinterpret_cast<uint32_t*>(o) = hi;
          const float r0 = h0 - __uint_as_float(hi << 16), r1 = h1 - __uint_as_float(hi & 0xFFFF0000u);
          // (of an infinity nothing is left)
          if (p.T <= kTwoParts) *reinterpret_cast<uint32_t*>(o + (int64_t)p.T * p.F) = bf16_pair(fabsf(r0) <= FLT_MAX ? r0 : 0.0f, fabsf(r1) <= FLT_MAX ? r1 : 0.0f);
          if (p.s.g) {
            const int64_t at = p.s.at(t, f);
            const float gv[2] = {v.x, v.y}, uv[2] = {v.z, v.w};
            save24<2>(p.s.g + at, p.s.gl + at, gv);
            save24<2>(p.s.u + at, p.s.ul + at, uv);
          }
        }
        acc[tn] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
      }
    }
    gr = ng;
    c = nc;
    return gr < groups;
  };
  while (turn(f0, f1) && turn(f1, f0)) {
  }
}

// Y = H Wd^T of up to 32 tokens: a workgroup takes 4 or 8 rows of Wd (fewer than the
// instruction's 16 so that more CUs read: 1 token of D 1024, F 4096 14.0 us with both
// kernels' waves on 64 to 128 CUs, 9.9 on all), its 16 waves the reduction in turn, joined in
// LDS.
struct DownFewArgs {
  const uint16_t *h, *wd;
  int64_t ldw;
  int32_t T, D, F, rows;
  void* y;
  int32_t bf16;
};
template <int TN>
__global__ __launch_bounds__(1024) void ffn_down_few_kernel(DownFewArgs p) {
  __shared__ float sh[16][16 * TN][17];
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int d0 = blockIdx.x * p.rows, steps = (p.F + 31) / 32;
  const int s0 = steps * wave / 16, s1 = steps * (wave + 1) / 16;
  const uint16_t* w = p.wd + (int64_t)(d0 + n) * p.ldw + g * 8;  // (D is a multiple of 16)
  // this lane's rows of H: tokens, and behind them from lane 8 on their second parts
  const bool two = p.T <= kTwoParts;
  const int rows = two ? 2 * p.T : p.T;
  int row[TN];
#pragma unroll
  for (int tn = 0; tn < TN; ++tn) row[tn] = !two ? tn * 16 + n : n % 8 < p.T && tn == 0 ? n / 8 * p.T + n % 8 : rows;
  float4_t acc[TN] = {};
  constexpr int U = 4;
  for (int s = s0; s < s1; s += U) {
    i32x4_t a[U], b[U][TN];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (s + u) * 32;
      const bool in = s + u < s1 && k + g * 8 < p.F;
      a[u] = i32x4_t{0, 0, 0, 0};
      if (in && n < p.rows) a[u] = *reinterpret_cast<const i32x4_t*>(w + k);
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) {
        b[u][tn] = i32x4_t{0, 0, 0, 0};
        if (in && row[tn] < rows) b[u][tn] = *reinterpret_cast<const i32x4_t*>(p.h + (int64_t)row[tn] * p.F + k + g * 8);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int tn = 0; tn < TN; ++tn)
        acc[tn] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a[u]), __builtin_bit_cast(bf16x8_t, b[u][tn]), acc[tn], 0, 0, 0);
  }
#pragma unroll
  for (int tn = 0; tn < TN; ++tn)
#pragma unroll
    for (int r = 0; r < 4; ++r) sh[wave][tn * 16 + n][4 * g + r] = acc[tn][r];
  __syncthreads();
  for (int i = threadIdx.x; i < 256 * TN; i += 1024) {
    const int t = i >> 4, d = i & 15;
    float v = sh[0][t][d];
#pragma unroll
    for (int k = 1; k < 16; ++k) v += sh[k][t][d];
    // (a sum that has left the range stays what it is: the second parts, 0 or of the other
    // sign, would make a NaN of an infinite weight's)
    if (two && t < 8 && fabsf(v) <= FLT_MAX) {
#pragma unroll
      for (int k = 0; k < 16; ++k) v += sh[k][t + 8][d];
    }
    if (t >= p.T || d >= p.rows) continue;
    const int64_t at = (int64_t)t * p.D + d0 + d;
    if (p.bf16) reinterpret_cast<uint16_t*>(p.y)[at] = (uint16_t)bf16_pair(v, 0.0f);
    else reinterpret_cast<float*>(p.y)[at] = v;
  }
}

// ---- dH and what follows from it ---------------------------------------------------------
// G and U are read and dG, dU (in both layouts that the products read) and H written by the
// lanes that hold dH.  16384 x 1024, 4096 features: 315 us for 1.07 GB (3.4 TB/s) and 137 GFLOP
// (which take 108): bound by memory, which a tile's products cover only in part (matrix units
// busy 20%).  A tile of 256 has no register to spare: 18 to 21 of a lane's wait in scratch (76
// to 88 bytes) while another part of the tile has its turn; the tiles of 64 need none.
struct DhArgs {
  TileOp P, Q;            // P: Wd^T [F, D], Q: dY [T, D]
  uint32_t tiles_p, tiles_q;
  int32_t nch, nf, nt;    // nf, nt: chunks of 64 features and of 64 tokens
  Saved s;                // G and U
  uint16_t* d;            // [T, dG | dU] blocked, nf chunks each, zero past the last feature; or NULL
  uint16_t *gt, *ut, *ht; // dG, dU, H transposed [F, T] blocked, zero past the last token; gt or ht NULL
};

template <class T, int ACT>
__global__ __launch_bounds__(T::NT, T::WAVES) void ffn_dh_kernel(DhArgs p) {
  static_assert(T::kTN == 4 && (T::PB == 2 || T::PB == 4), "64 tokens, and features 8 or 16 a lane");
  __shared__ __attribute__((aligned(128))) typename T::Smem sm;
  const typename T::Items items(p.tiles_p, p.tiles_q, (uint32_t)p.nch, 1);
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 15, g = lane >> 4;
  T::run(p.P, p.Q, items, sm, [&](int64_t p0, int64_t q0, uint32_t, typename T::Acc& acc) __attribute__((always_inline)) {
    const int64_t F = p.P.rows, pw = p0 + (w / T::kWN) * T::kTM * 16, qw = q0 + (w % T::kWN) * 64, t0 = qw + n * 4;
    const int ct = (int)(qw >> 6);
    static_assert(16 * T::kTM <= 128 && 128 % (16 * T::kTM) == 0, "a wave's features are of one block");
#pragma unroll
    for (int tb = 0; tb < T::kTM / T::PB; ++tb) {
      const int64_t f = pw + tb * 16 * T::PB + g * 4 * T::PB;  // this lane's 4 PB features
      const bool in = f < F;
      const int64_t turned = ((pw >> 7) * p.nt + ct) * 8192 + (f & 127) * 64 + n * 4;
#pragma unroll
      for (int half = 0; half < T::PB / 2; ++half) {
        uint4 gv[4], uv[4];
        uint2 gl[4], ul[4];
#pragma unroll
        for (int tn = 0; tn < 4; ++tn) {
          gv[tn] = uv[tn] = uint4{0u, 0u, 0u, 0u};
          gl[tn] = ul[tn] = uint2{0u, 0u};
          if (in && t0 + tn < p.Q.rows) {
            const int64_t at = p.s.at(t0 + tn, f + half * 8);
            gv[tn] = *reinterpret_cast<const uint4*>(p.s.g + at);
            uv[tn] = *reinterpret_cast<const uint4*>(p.s.u + at);
            gl[tn] = *reinterpret_cast<const uint2*>(p.s.gl + at);
            ul[tn] = *reinterpret_cast<const uint2*>(p.s.ul + at);
          }
        }
        static_for<2>([&](auto jc) __attribute__((always_inline)) {
          constexpr int j = decltype(jc)::value;
          const int tm = tb * T::PB + half * 2 + j;
          float dg[4][4], du[4][4], h[4][4];  // [token][feature]
#pragma unroll
          for (int tn = 0; tn < 4; ++tn) {
            const bool there = in && t0 + tn < p.Q.rows;  // (zeros times a NaN of the operands would not be zero)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float gr = value24(gv[tn], gl[tn], j * 4 + r), ur = value24(uv[tn], ul[tn], j * 4 + r);
              const Act a = activate<ACT>(gr);
              const float dh = there ? acc[tm][tn][r] : 0.0f;
              dg[tn][r] = dh * ur * a.d;
              du[tn][r] = dh * a.a;
              h[tn][r] = a.a * ur;
            }
            acc[tm][tn] = float4_t{__uint_as_float(bf16_pair(dg[tn][0], dg[tn][1])), __uint_as_float(bf16_pair(dg[tn][2], dg[tn][3])),
                                   __uint_as_float(bf16_pair(du[tn][0], du[tn][1])), __uint_as_float(bf16_pair(du[tn][2], du[tn][3]))};
          }
          // transposed: four neighbouring tokens of a feature, 128 bytes over 16 lanes
          if (in && ct < p.nt) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int64_t at = turned + (half * 8 + j * 4 + r) * 64;
              if (p.gt) {
                *reinterpret_cast<uint2*>(p.gt + at) = uint2{bf16_pair(dg[0][r], dg[1][r]), bf16_pair(dg[2][r], dg[3][r])};
                *reinterpret_cast<uint2*>(p.ut + at) = uint2{bf16_pair(du[0][r], du[1][r]), bf16_pair(du[2][r], du[3][r])};
              }
              if (p.ht) *reinterpret_cast<uint2*>(p.ht + at) = uint2{bf16_pair(h[0][r], h[1][r]), bf16_pair(h[2][r], h[3][r])};
            }
          }
        });
      }
      // as they are: 8 or 16 neighbouring features of a token
      const int cd = (int)(f >> 6);
      if (!p.d || cd >= p.nf) continue;
#pragma unroll
      for (int tn = 0; tn < 4; ++tn) {
        const int64_t t = t0 + tn;
        if (t >= p.Q.rows) continue;
        uint16_t* o = p.d + ((t >> 7) * 2 * p.nf + cd) * 8192 + (t & 127) * 64 + (f & 63);
#pragma unroll
        for (int half = 0; half < T::PB / 2; ++half) {
          const float4_t a = acc[tb * T::PB + half * 2][tn], b = acc[tb * T::PB + half * 2 + 1][tn];
          *reinterpret_cast<uint4*>(o + half * 8) = uint4{__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y)};
          *reinterpret_cast<uint4*>(o + (int64_t)p.nf * 8192 + half * 8) =
              uint4{__float_as_uint(a.z), __float_as_uint(a.w), __float_as_uint(b.z), __float_as_uint(b.w)};
        }
      }
    }
  });
}

// ---- products ----------------------------------------------------------------------------
// D[q, p] = sum_k Q[q, k] P[p, k], up to four in one launch, each with workgroups of its
// own; splits > 1: fp32 partial sums [z][q][p], joined by ffn_join_kernel.
// 16384 x 1024, 4096 features: Y 121 us (1.14 PFLOP/s), the four of the backward pass 540 to
// 600 us (687 GFLOP, 1.15 to 1.27: the clock falls under them; matrix units busy 59%).  Few
// tiles are bound by each chunk's way from memory: 300 x 1024 over 4096, 8 splits 12.0 us,
// and 3.9 for their sums.
constexpr int kJobs = 4;
struct FfnProduct {
  TileOp P, Q;
  uint32_t tiles_p, tiles_q;
  int32_t nch, splits;
  float* part;
  void* out;  // rows of P.rows elements
  int32_t bf16;
};
struct FfnProducts {
  FfnProduct x[kJobs];
  uint32_t first[kJobs];  // workgroup at which a job starts
  int32_t n;
};

template <class T>
__global__ __launch_bounds__(T::NT, T::WAVES) void ffn_product_kernel(FfnProducts jobs) {
  __shared__ __attribute__((aligned(128))) typename T::Smem sm;
  int job = 0;
  while (job + 1 < jobs.n && blockIdx.x >= jobs.first[job + 1]) ++job;
  const FfnProduct& p = jobs.x[job];
  const uint32_t end = job + 1 < jobs.n ? jobs.first[job + 1] : gridDim.x;
  const typename T::Items items(p.tiles_p, p.tiles_q, (uint32_t)p.nch, (uint32_t)p.splits, blockIdx.x - jobs.first[job], end - jobs.first[job]);
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
  T::run(p.P, p.Q, items, sm, [&](int64_t p0, int64_t q0, uint32_t z, typename T::Acc& acc) __attribute__((always_inline)) {
    constexpr int N = 4 * T::PB;  // neighbouring results of a lane
    const int64_t pw = p0 + (w / T::kWN) * T::kTM * 16 + g * N, qw = q0 + (w % T::kWN) * T::kTN * 16;
#pragma unroll
    for (int tn = 0; tn < T::kTN; ++tn) {
      const int64_t i = qw + T::q_row(tn, n);
      if (i >= p.Q.rows) continue;
#pragma unroll
      for (int tb = 0; tb < T::kTM / T::PB; ++tb) {
        const int64_t j = pw + tb * 4 * N;
        if (j >= p.P.rows) continue;  // (a multiple of 16)
        if (p.splits == 1 && p.bf16) {
          float v[N];
#pragma unroll
          for (int k = 0; k < N; ++k) v[k] = acc[tb * T::PB + k / 4][tn][k % 4];
          uint16_t* o = reinterpret_cast<uint16_t*>(p.out) + i * p.P.rows + j;
#pragma unroll
          for (int k = 0; k < N; k += 8) *reinterpret_cast<uint4*>(o + k) = pack8(v + k);
        } else {
          float* o = p.splits == 1 ? reinterpret_cast<float*>(p.out) : p.part + (size_t)z * (size_t)(p.Q.rows * p.P.rows);
#pragma unroll
          for (int k = 0; k < T::PB; ++k) *reinterpret_cast<float4_t*>(o + i * p.P.rows + j + 4 * k) = acc[tb * T::PB + k][tn];
        }
      }
    }
  });
}

// The sums of the splits' results in order, 4 a thread.  Memory: 16384 x 1024, 4096 features
// 12.4 us.
__global__ __launch_bounds__(256) void ffn_join_kernel(FfnProducts jobs) {
  int job = 0;
  while (job + 1 < jobs.n && blockIdx.x >= jobs.first[job + 1]) ++job;
  const FfnProduct& p = jobs.x[job];
  const int64_t n = p.Q.rows * p.P.rows, i = ((int64_t)(blockIdx.x - jobs.first[job]) * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  float4_t v = *reinterpret_cast<const float4_t*>(p.part + i);
#pragma unroll 4
  for (int z = 1; z < p.splits; ++z) v += *reinterpret_cast<const float4_t*>(p.part + (size_t)z * (size_t)n + i);
  if (p.bf16) *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + i) = uint2{bf16_pair(v.x, v.y), bf16_pair(v.z, v.w)};
  else *reinterpret_cast<float4_t*>(reinterpret_cast<float*>(p.out) + i) = v;
}

// Blocked copies and transposes, a workgroup per 64 x 64.  Memory: 16384 x 1024, 4096
// features 21 us before the forward's kernels, 44 before the backward's (134 MB, 3.7 TB/s of
// what reaches the L2).
constexpr int kBlocks = 5;
struct FfnBlocks {
  BlockArgs x[kBlocks];
  uint32_t first[kBlocks];
  int32_t n;
};
__global__ __launch_bounds__(256) void ffn_blocks_kernel(FfnBlocks jobs) {
  int job = 0;
  while (job + 1 < jobs.n && blockIdx.x >= jobs.first[job + 1]) ++job;
  const BlockArgs& p = jobs.x[job];
  const uint32_t b = blockIdx.x - jobs.first[job];
  block_tile(p, b % p.nr, b / p.nr);
}

using TileBig = Tile<EL_BF16, 2, 4, 8, 4>;   // 256 x 256
using TileMid = Tile<EL_BF16, 2, 2, 4, 4>;   // 128 x 128
using TileLow = Tile<EL_BF16, 2, 2, 2, 4>;   // 64 x 128
using PairBig = Tile<EL_PAIR, 2, 4, 8, 4>;   // 128 of either weight x 256
using PairMid = Tile<EL_PAIR, 2, 2, 4, 4>;   // 64 of either weight x 128
using PairLow = Tile<EL_PAIR, 2, 2, 4, 2>;   // 64 of either weight x 64

template <class T, class A>
uint32_t set_tiles(A& a) {
  a.tiles_p = (uint32_t)((a.P.rows + T::PROWS - 1) / T::PROWS);
  a.tiles_q = (uint32_t)((a.Q.rows + T::BN - 1) / T::BN);
  return a.tiles_p * a.tiles_q;
}
template <class F>
void with_activation(int act, F&& f) {
  if (act == TJ2_SILU) f(std::integral_constant<int, TJ2_SILU>{});
  else if (act == TJ2_GELU) f(std::integral_constant<int, TJ2_GELU>{});
  else f(std::integral_constant<int, TJ2_GELU_TANH>{});
}

// Tiles of 16 tokens of the few-token kernels, 0: none.  Forward here and in tiles, us:
// D 1024, F 4096: 1 token 9.9 and 20.5, 16 tokens 15.5 and 22.5 (32 24 and 23.5); D 2048, F
// 8192: 1 token 23.1 and 38.2, 16 tokens 38.2 and 40.6; D 512, F 2048: 17 tokens 10.9 and
// 17.2, 32 tokens 13.6 and 17.1; D 512, F 8192: 16 tokens 18.9 and 19.6, 17 tokens 22.2 and
// 19.5.
int few_tiles(int64_t T, int64_t D, int64_t F) {
  if (T <= 16 && D <= 2048) return 1;
  if (T <= 32 && D <= 512 && D * F <= (int64_t)1 << 21) return 2;
  return 0;
}
static_assert(16 * few_pitch(2048) <= 80 * 1024 && 32 * few_pitch(512) <= 80 * 1024, "two workgroups' tokens fit the LDS");

// Tile and splits of up to four products that run together: those of the least estimated
// time, the items (tiles times splits) being dealt out to the CUs' places, the longest
// first, as they become free.  What tiles and partial sums take (us on MI355X, operands in
// blocks, a chunk 64 elements) is of two kinds.  Several products: as timed, partial sums
// at 5 TB/s each way and a launch.  (Backward products of 16384 x 1024, 4096 features: 677 us
// with two splits for each of the weights' gradients and none for dX, whose 2.5 rounds of
// equal items take three; 544 as planned here.)  One product: fitted to 600 forward passes
// of 28 sizes under all tiles and splits, of which it picks one within 0.5% of the best in
// the mean (with the first kind's numbers 3.6%; those of the second cost backward passes
// 1.3%): 300 x 1024, 4096 features 30.8 -> 29.0 us, 600 40.0 -> 37.6, 64 x 2048, 8192 41.7 ->
// 38.7.  The tiles of 64 against none: backward of 2048 x 512, 2048 features 62.1 and 58.5.
enum class Tiles { Big, Mid, Low };
struct FfnPlan {
  Tiles tiles;
  int splits[kJobs];
};
struct FfnSize {
  int64_t p, q, k;
};
constexpr int kSplitChoices[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32};

// when the last place is free of n groups of count items of time t, the longest first
double deal(double places, const double* count, const double* t, int n) {
  struct Level {
    double at, places;
  };
  Level level[40] = {{0.0, places}};
  int levels = 1;
  for (int i = 0; i < n; ++i) {
    double left = count[i];
    // whole rounds at once
    const double whole = std::floor(left / places) - 1.0;
    if (whole > 0.0) {
      for (int l = 0; l < levels; ++l) level[l].at += whole * t[i];
      left -= whole * places;
    }
    while (left > 0.0 && levels < 39) {
      int least = 0;
      for (int l = 1; l < levels; ++l)
        if (level[l].at < level[least].at) least = l;
      const double take = std::min(left, level[least].places);
      left -= take;
      if (take == level[least].places) {
        level[least].at += t[i];
      } else {
        level[least].places -= take;
        level[levels++] = Level{level[least].at + t[i], take};
      }
    }
  }
  double last = 0.0;
  for (int l = 0; l < levels; ++l) last = std::max(last, level[l].at);
  return last;
}

// What a tile takes: P's and Q's rows, tiles of a CU, us a chunk alone on its CU and with
// the CU full, us for start and results.
struct TileCost {
  int64_t p, q, per_cu;
  double alone, full, fixed;
};
// of one product, and of several in a launch, by Tiles
constexpr TileCost kOne[3] = {{256, 256, 1, 0.75, 0.75, 4.5}, {128, 128, 2, 0.56, 0.73, 1.1}, {64, 128, 3, 0.44, 0.52, 0.0}},
                   kMany[3] = {{256, 256, 1, 1.6, 1.6, 5.0}, {128, 128, 2, 0.67, 0.97, 3.0}, {64, 128, 3, 0.5, 0.95, 3.0}};

// The plan's time, or `least` where it is seen to take no less before the items are dealt out.
double plan_time(const FfnPlan& plan, const FfnSize* x, int n, double least) {
  const TileCost c = (n == 1 ? kOne : kMany)[(int)plan.tiles];
  double count[kJobs], t[kJobs], items = 0.0, join = 0.0;
  for (int i = 0; i < n; ++i) {
    const int64_t nch = (x[i].k + 63) / 64;
    count[i] = (double)((x[i].p + c.p - 1) / c.p * ((x[i].q + c.q - 1) / c.q)) * plan.splits[i];
    t[i] = (double)((nch + plan.splits[i] - 1) / plan.splits[i]);
    items += count[i];
    if (plan.splits[i] > 1) join += (double)x[i].p * (double)x[i].q * plan.splits[i] * (n == 1 ? 2.3e-6 : 1.6e-6);
  }
  double deep = std::min((double)c.per_cu, std::ceil(items / kCus));  // tiles of a CU at once
  if (n > 1 && deep > 1.0) deep = (double)c.per_cu;
  const double chunk = deep == 1.0 ? c.alone : c.alone + (c.full - c.alone) * (deep - 1.0) / (double)(c.per_cu - 1);
  if (join > 0.0) join += n == 1 ? 0.8 : 3.0;
  double work = 0.0, longest = 0.0;
  for (int i = 0; i < n; ++i) {
    t[i] = t[i] * chunk + c.fixed;
    work += count[i] * t[i];
    longest = std::max(longest, t[i]);
  }
  // (a part in 10^9 for the rounding of the sums)
  if ((std::max(longest, work / (deep * kCus)) + join) * (1.0 - 1e-9) > least) return least;
  for (int i = 1; i < n; ++i)  // the longest first
    for (int k = i; k > 0 && t[k] > t[k - 1]; --k) {
      std::swap(t[k], t[k - 1]);
      std::swap(count[k], count[k - 1]);
    }
  return deal(deep * kCus, count, t, n) + join;
}

FfnPlan find_plan(const FfnSize* x, int n) {
  FfnPlan best = {};
  double least = 1e30;
  for (const Tiles tiles : {Tiles::Mid, Tiles::Big, Tiles::Low}) {
    FfnPlan c = {};
    c.tiles = tiles;
    // every choice for each product, equal ones (the gates' and factors' weights) alike
    auto choose = [&](auto&& self, int i) -> void {
      if (i == n) {
        if (const double t = plan_time(c, x, n, least); t < least) {
          least = t;
          best = c;
        }
        return;
      }
      for (int k = 0; k < i; ++k)
        if (x[k].p == x[i].p && x[k].q == x[i].q && x[k].k == x[i].k) {
          c.splits[i] = c.splits[k];
          return self(self, i + 1);
        }
      for (const int z : kSplitChoices) {
        if (z > 1 && (x[i].k + 63) / 64 < 4 * z) break;
        c.splits[i] = z;
        self(self, i + 1);
      }
    };
    choose(choose, 0);
  }
  return best;
}

// What has been found for the last sizes, for all threads (a backward pass runs on one of its
// own): 4 places for each of 256 remainders of the sizes, the oldest given up first.
template <int N, class V>
class Found {
 public:
  using Key = std::array<int64_t, N>;
  bool get(const Key& key, V* v) {
    std::lock_guard<std::mutex> lock(mu_);
    for (const Entry& e : set(key))
      if (e.used && e.key == key) {
        *v = e.v;
        return true;
      }
    return false;
  }
  void put(const Key& key, const V& v) {
    std::lock_guard<std::mutex> lock(mu_);
    Entry* s = set(key);
    std::copy_backward(s, s + kWays - 1, s + kWays);
    s[0] = Entry{key, v, true};
  }

 private:
  static constexpr int kWays = 4, kSets = 256;
  struct Entry {
    Key key;
    V v;
    bool used;
  };
  using Set = Entry[kWays];
  Set& set(const Key& key) {
    uint64_t h = 0;
    for (const int64_t k : key) h = (h ^ (uint64_t)k) * 0x9E3779B97F4A7C15u;
    return sets_[h >> 56];
  }
  std::mutex mu_;
  Set sets_[kSets] = {};
};

// A search takes up to 0.1 ms of the host.
FfnPlan ffn_plan(const FfnSize* x, int n) {
  static Found<1 + 3 * kJobs, FfnPlan> found;
  std::array<int64_t, 1 + 3 * kJobs> key = {n};
  for (int i = 0; i < n; ++i) {
    key[1 + 3 * i] = x[i].p;
    key[2 + 3 * i] = x[i].q;
    key[3 + 3 * i] = x[i].k;
  }
  FfnPlan plan;
  if (!found.get(key, &plan)) {
    plan = find_plan(x, n);
    found.put(key, plan);
  }
  return plan;
}
size_t part_bytes(const FfnPlan& plan, const FfnSize* x, int n) {
  size_t b = 0;
  for (int i = 0; i < n; ++i)
    if (plan.splits[i] > 1) b += up256((size_t)plan.splits[i] * (size_t)(x[i].p * x[i].q) * 4);
  return b;
}

template <class T>
void launch_products(FfnProducts& jobs, hipStream_t s) {
  uint32_t items[kJobs], total = 0, grid = 0;
  for (int i = 0; i < jobs.n; ++i) {
    items[i] = set_tiles<T>(jobs.x[i]) * (uint32_t)jobs.x[i].splits;
    total += items[i];
  }
  // few rounds: a workgroup an item, dealt out by the hardware; else each goes on itself
  const bool each = total <= 8 * kCus * T::PER_CU;
  for (int i = 0; i < jobs.n; ++i) {
    jobs.first[i] = grid;
    grid += each ? items[i] : T::grid(items[i]);
  }
  ffn_product_kernel<T><<<grid, T::NT, 0, s>>>(jobs);
}

// The products x under their plan, partial sums at `part`.
hipError_t run_products(FfnProduct* x, const FfnSize* size, int n, float* part, hipStream_t s) {
  const FfnPlan plan = ffn_plan(size, n);
  FfnProducts jobs = {}, joins = {};
  size_t at = 0;
  // those with the longest tiles first
  int order[kJobs] = {0, 1, 2, 3};
  std::sort(order, order + n, [&](int a, int b) {
    const int64_t ka = size[a].k / plan.splits[a], kb = size[b].k / plan.splits[b];
    return ka != kb ? ka > kb : a < b;
  });
  for (int i = 0; i < n; ++i) {
    x[i].nch = (int32_t)((size[i].k + 63) / 64);
    x[i].splits = plan.splits[i];
    if (x[i].splits > 1) {
      x[i].part = part + at / 4;
      at += up256((size_t)x[i].splits * (size_t)(size[i].p * size[i].q) * 4);
    }
  }
  for (int i = 0; i < n; ++i) jobs.x[i] = x[order[i]];
  jobs.n = n;
  if (plan.tiles == Tiles::Big) launch_products<TileBig>(jobs, s);
  else if (plan.tiles == Tiles::Low) launch_products<TileLow>(jobs, s);
  else launch_products<TileMid>(jobs, s);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  uint32_t grid = 0;
  for (int i = 0; i < n; ++i) {
    if (x[i].splits == 1) continue;
    joins.x[joins.n] = x[i];
    joins.first[joins.n++] = grid;
    grid += (uint32_t)((size[i].p * size[i].q / 4 + 255) / 256);
  }
  if (!grid) return hipSuccess;
  ffn_join_kernel<<<grid, 256, 0, s>>>(joins);
  return hipGetLastError();
}

hipError_t run_blocks(const BlockArgs* x, int n, hipStream_t s) {
  FfnBlocks b = {};
  uint32_t grid = 0;
  for (int i = 0; i < n; ++i) {
    b.x[i] = x[i];
    b.first[i] = grid;
    grid += x[i].nr * x[i].nc;
  }
  b.n = n;
  if (!grid) return hipSuccess;
  ffn_blocks_kernel<<<grid, 256, 0, s>>>(b);
  return hipGetLastError();
}

Saved saved_of(const FfnParams& f) {
  if (!f.gu) return Saved{};
  const int64_t n = up(f.T, 64) * up(f.F, 64);
  uint16_t* hi = reinterpret_cast<uint16_t*>(f.gu);
  uint8_t* lo = reinterpret_cast<uint8_t*>(hi + 2 * n);
  return Saved{hi, hi + n, lo, lo + n, up(f.F, 64) / 64};
}

// Of a product with an epilogue: 256 x 256 tiles or smaller ones.
bool big_tiles(int64_t p, int64_t q, int64_t k) {
  const double chunks = (double)((k + 63) / 64);
  return tile_time(true, tiles_of(p, q, 256), chunks, 9.0) < tile_time(false, tiles_of(p, q, 128), chunks, 9.0);
}

struct FfnFwdSpace {
  size_t h, x, g, u, d, part, bytes;
  bool blocked;
  int few;
  FfnFwdSpace(int64_t T, int64_t D, int64_t F) {
    size_t at = 0;
    auto take = [&](size_t n) { const size_t a = at; at += up256(n); return a; };
    few = few_tiles(T, D, F);
    blocked = T >= kBlockTokens;
    h = take(few ? (size_t)(T * F * (T <= kTwoParts ? 4 : 2)) : blocked_bytes(T, F));
    x = take(blocked ? blocked_bytes(T, D) : 0);
    g = take(blocked ? blocked_bytes(F, D) : 0);
    u = take(blocked ? blocked_bytes(F, D) : 0);
    d = take(blocked ? blocked_bytes(D, F) : 0);
    const FfnSize y = {D, T, F};
    part = take(few ? 0 : part_bytes(ffn_plan(&y, 1), &y, 1));
    bytes = at;
  }
};

struct FfnBwdSpace {
  size_t wd, w, x, dy, dyb, d, gt, ut, ht, part;  // (partial sums last: part_most bytes)
  bool blocked;
  FfnBwdSpace(int64_t T, int64_t D, int64_t F) {
    size_t at = 0;
    auto take = [&](size_t n) { const size_t a = at; at += up256(n); return a; };
    blocked = T >= kBlockTokens;
    wd = take(blocked_bytes(F, D));
    w = take(blocked_bytes(D, 2 * up(F, 64)));
    x = take(blocked_bytes(D, T));
    dy = take(blocked_bytes(D, T));
    dyb = take(blocked ? blocked_bytes(T, D) : 0);
    d = take(blocked_bytes(T, 2 * up(F, 64)));
    gt = take(blocked_bytes(F, T));
    ut = take(blocked_bytes(F, T));
    ht = take(blocked_bytes(F, T));
    part = at;
  }
  // whichever gradients are asked for
  static size_t part_most(int64_t T, int64_t D, int64_t F) {
    static Found<3, size_t> found;
    size_t most = 0;
    if (found.get({T, D, F}, &most)) return most;
    for (int want = 1; want < 8; ++want)
      for (const bool both : {true, false}) {
        FfnSize x4[kJobs];
        const int n = sizes(T, D, F, want & 1, want & 2, (want & 2) && both, want & 4, x4);
        if (both || (want & 2)) most = std::max(most, part_bytes(ffn_plan(x4, n), x4, n));
      }
    most = up256(most);
    found.put({T, D, F}, most);
    return most;
  }
  static int sizes(int64_t T, int64_t D, int64_t F, bool dx, bool dwg, bool dwu, bool dwd, FfnSize* x) {
    int n = 0;
    if (dx) x[n++] = FfnSize{D, T, 2 * up(F, 64)};
    if (dwg) x[n++] = FfnSize{D, F, T};
    if (dwu) x[n++] = FfnSize{D, F, T};
    if (dwd) x[n++] = FfnSize{F, D, T};
    return n;
  }
};

}  // namespace

#define TJ2_DO(call)                                     \
  do {                                                   \
    if (hipError_t e_ = (call); e_ != hipSuccess) return e_; \
  } while (0)

size_t ffn_saved_bytes(int64_t T, int64_t F) { return (size_t)(up(T, 64) * up(F, 64)) * 6; }

size_t ffn_fwd_workspace_bytes(int64_t T, int64_t D, int64_t F) { return FfnFwdSpace(T, D, F).bytes; }

hipError_t launch_ffn_fwd(const FfnParams& f, void* ws, hipStream_t s) {
  const FfnFwdSpace sp(f.T, f.D, f.F);
  uint8_t* w = reinterpret_cast<uint8_t*>(ws);
  uint16_t* h = reinterpret_cast<uint16_t*>(w + sp.h);
  if (sp.few) {
    const int32_t down_rows = f.D >= 8 * kCus ? 8 : 4;  // (D is at most 2048 here)
    const GateFewArgs a = {reinterpret_cast<const uint16_t*>(f.X), reinterpret_cast<const uint16_t*>(f.Wg), reinterpret_cast<const uint16_t*>(f.Wu),
                           f.ldx, f.ldw, (int32_t)f.T, (int32_t)f.D, (int32_t)f.F, h, saved_of(f)};
    const DownFewArgs d = {h, reinterpret_cast<const uint16_t*>(f.Wd), f.ldd, (int32_t)f.T, (int32_t)f.D, (int32_t)f.F, down_rows, f.Y, f.y_dtype == TJ2_BF16};
    // two waves a workgroup while those reach no more CUs
    const uint32_t groups = (uint32_t)((f.F + 7) / 8), per = groups <= 4 * kCus ? 2 : 4, rounds = (groups + 8 * kCus - 1) / (8 * kCus),
                   grid = (groups + rounds * per - 1) / (rounds * per);
    const size_t lds = (size_t)(f.T * few_pitch(f.D));
    auto run = [&](auto tn) {
      constexpr int TN = decltype(tn)::value;
      with_activation(f.act, [&](auto act) { ffn_gate_few_kernel<TN, act.value><<<grid, per * 64, lds, s>>>(a); });
      ffn_down_few_kernel<TN><<<(uint32_t)(f.D / down_rows), 1024, 0, s>>>(d);
    };
    if (sp.few == 1) run(std::integral_constant<int, 1>{});
    else run(std::integral_constant<int, 2>{});
    return hipGetLastError();
  }
  GateArgs a = {};
  TileOp wd;
  if (sp.blocked) {
    const BlockArgs b[4] = {block_args(f.X, f.T, f.D, f.ldx, w + sp.x, nullptr), block_args(f.Wg, f.F, f.D, f.ldw, w + sp.g, nullptr),
                            block_args(f.Wu, f.F, f.D, f.ldw, w + sp.u, nullptr), block_args(f.Wd, f.D, f.F, f.ldd, w + sp.d, nullptr)};
    TJ2_DO(run_blocks(b, 4, s));
    a.P = blocked_operand(w + sp.g, f.F, f.D);
    a.P.p2 = w + sp.u;
    a.Q = blocked_operand(w + sp.x, f.T, f.D);
    wd = blocked_operand(w + sp.d, f.D, f.F);
  } else {
    a.P = bf16_operand(f.Wg, f.F, f.D, f.ldw);
    a.P.p2 = reinterpret_cast<const uint8_t*>(f.Wu);
    a.Q = bf16_operand(f.X, f.T, f.D, f.ldx);
    wd = bf16_operand(f.Wd, f.D, f.F, f.ldd);
  }
  a.nch = (int32_t)(up(f.D, 64) / 64);
  a.nf = (int32_t)(up(f.F, 64) / 64);
  a.h = h;
  a.s = saved_of(f);
  // Low where the middle tiles would leave CUs idle or few with two (forward, us, middle and
  // low: 64 x 512, 2048 features 18.1 and 16.0 (16 middle tiles), 300 x 1024, 4096 33.4 and 32.1
  // (192), 600 x 1024, 4096 41.9 and 40.8 (320), 2048 x 512, 2048 41.4 and 42.6 (512)).
  const bool big = big_tiles(2 * f.F, f.T, f.D);
  with_activation(f.act, [&](auto act) {
    if (big) {
      const uint32_t items = set_tiles<PairBig>(a);
      ffn_gate_kernel<PairBig, act.value><<<PairBig::grid(items), PairBig::NT, 0, s>>>(a);
    } else if (const uint32_t items = set_tiles<PairMid>(a); items > kCus * 5 / 4) {
      ffn_gate_kernel<PairMid, act.value><<<PairMid::grid(items), PairMid::NT, 0, s>>>(a);
    } else {
      const uint32_t few = set_tiles<PairLow>(a);
      ffn_gate_kernel<PairLow, act.value><<<PairLow::grid(few), PairLow::NT, 0, s>>>(a);
    }
  });
  TJ2_DO(hipGetLastError());
  FfnProduct y = {};
  y.P = wd;
  y.Q = blocked_operand(h, f.T, f.F);
  y.out = f.Y;
  y.bf16 = f.y_dtype == TJ2_BF16;
  const FfnSize size = {f.D, f.T, f.F};
  return run_products(&y, &size, 1, reinterpret_cast<float*>(w + sp.part), s);
}

size_t ffn_bwd_workspace_bytes(int64_t T, int64_t D, int64_t F) {
  return FfnBwdSpace(T, D, F).part + FfnBwdSpace::part_most(T, D, F);
}

hipError_t launch_ffn_bwd(const FfnParams& f, const FfnGradParams& o, void* ws, hipStream_t s) {
  const FfnBwdSpace sp(f.T, f.D, f.F);
  uint8_t* w = reinterpret_cast<uint8_t*>(ws);
  const int64_t nf = up(f.F, 64) / 64;
  const bool dw = o.dWg || o.dWu;
  BlockArgs b[kBlocks];
  int n = 0;
  b[n++] = block_args(f.Wd, f.D, f.F, f.ldd, nullptr, w + sp.wd);
  if (o.dX) {
    b[n] = block_args(f.Wg, f.F, f.D, f.ldw, nullptr, w + sp.w);
    b[n++].pitch = (uint32_t)(2 * nf);
    b[n] = block_args(f.Wu, f.F, f.D, f.ldw, nullptr, w + sp.w + nf * 16384);
    b[n++].pitch = (uint32_t)(2 * nf);
  }
  if (dw) b[n++] = block_args(f.X, f.T, f.D, f.ldx, nullptr, w + sp.x);
  if (o.dWd || sp.blocked) b[n++] = block_args(o.dY, f.T, f.D, o.ldy, sp.blocked ? w + sp.dyb : nullptr, o.dWd ? w + sp.dy : nullptr);
  TJ2_DO(run_blocks(b, n, s));
  DhArgs a = {};
  a.P = blocked_operand(w + sp.wd, f.F, f.D);
  a.Q = sp.blocked ? blocked_operand(w + sp.dyb, f.T, f.D) : bf16_operand(o.dY, f.T, f.D, o.ldy);
  a.nch = (int32_t)(up(f.D, 64) / 64);
  a.nf = (int32_t)nf;
  a.nt = (int32_t)(up(f.T, 64) / 64);
  a.s = saved_of(f);
  a.d = o.dX ? reinterpret_cast<uint16_t*>(w + sp.d) : nullptr;
  a.gt = dw ? reinterpret_cast<uint16_t*>(w + sp.gt) : nullptr;
  a.ut = reinterpret_cast<uint16_t*>(w + sp.ut);
  a.ht = o.dWd ? reinterpret_cast<uint16_t*>(w + sp.ht) : nullptr;
  // Tiles of 64 features where big ones do not pay: the epilogue is long, and three of them
  // on a CU cover it in part (backward, us, with 128 x 128 and with 64 x 128: 1235 x 528, 1552
  // features 53.5 and 49.2, 2048 x 1024, 2048 87.6 and 84.3, 8192 x 256, 1024 72.5 and 72.6).
  const bool big = big_tiles(f.F, f.T, f.D);
  with_activation(f.act, [&](auto act) {
    if (big) {
      const uint32_t items = set_tiles<TileBig>(a);
      ffn_dh_kernel<TileBig, act.value><<<TileBig::grid(items), TileBig::NT, 0, s>>>(a);
    } else {
      const uint32_t items = set_tiles<TileLow>(a);
      ffn_dh_kernel<TileLow, act.value><<<TileLow::grid(items), TileLow::NT, 0, s>>>(a);
    }
  });
  TJ2_DO(hipGetLastError());
  FfnProduct x[kJobs] = {};
  FfnSize size[kJobs];
  const int jobs = FfnBwdSpace::sizes(f.T, f.D, f.F, o.dX, o.dWg, o.dWu, o.dWd, size);
  int k = 0;
  auto product = [&](TileOp Q, TileOp P, void* out, int dtype) {
    x[k].P = P;
    x[k].Q = Q;
    x[k].out = out;
    x[k++].bf16 = dtype == TJ2_BF16;
  };
  if (o.dX) product(blocked_operand(w + sp.d, f.T, 2 * nf * 64), blocked_operand(w + sp.w, f.D, 2 * nf * 64), o.dX, o.dx_dtype);
  if (o.dWg) product(blocked_operand(w + sp.gt, f.F, f.T), blocked_operand(w + sp.x, f.D, f.T), o.dWg, o.dw_dtype);
  if (o.dWu) product(blocked_operand(w + sp.ut, f.F, f.T), blocked_operand(w + sp.x, f.D, f.T), o.dWu, o.dw_dtype);
  if (o.dWd) product(blocked_operand(w + sp.dy, f.D, f.T), blocked_operand(w + sp.ht, f.F, f.T), o.dWd, o.dw_dtype);
  return run_products(x, size, jobs, reinterpret_cast<float*>(w + sp.part), s);
}

}  // namespace tj2
