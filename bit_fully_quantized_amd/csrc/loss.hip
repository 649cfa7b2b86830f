// Losses at the language-model head for gfx950.
//
// Cross entropy of logits z = X W^T (X [T, K], W [V, K], bf16) against one target
// per token, without the logits in memory:
//   loss_t = lse_t - z[t, y_t],  lse_t = log sum_v exp z[t, v]
//   dz[t, v] = w_t (exp(z[t, v] - lse_t) - [v = y_t]),  dX = dz W,  dW = dz^T X.
// The forward is one tile product whose epilogue reduces each token's logits of a
// tile to a running maximum and a sum of exponentials (a pair per 16 TM
// vocabulary entries); a second kernel joins the pairs.  The backward takes the
// vocabulary in pieces: the piece's logits again, dz of the piece in bf16 (row and
// transposed), then the two products it enters.
//
// Distillation from a teacher's top logits, on logits that are in memory (the head
// may be quantized): one workgroup a token, which keeps the row in registers, so
// logits are read once and the gradient is written once (rows that no registers hold
// are read three times: launch_distill_r).
#include <math.h>

#include <algorithm>

#include "tj2_skinny.h"

namespace tj2 {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// 2^((v - m) c): the difference first, which is exact for logits near m and 0 at it
// however large they are (a fused v c - m c is off by a half step of m c)
__device__ __forceinline__ float exp_scaled(float v, float m, float c) { return __builtin_amdgcn_exp2f((v - m) * c); }

// (r, s): s 2^r in total; r = -inf stands for nothing
__device__ __forceinline__ void join(float& r, float& s, float r2, float s2) {
  const float R = fmaxf(r, r2);
  const float b = R == -INFINITY ? 0.0f : R;
  s = s * __builtin_amdgcn_exp2f(r - b) + s2 * __builtin_amdgcn_exp2f(r2 - b);
  r = R;
}

constexpr float kNan = __builtin_nanf("");

struct CeArgs {
  TileOp P, Q;                 // P: W [V, K] (or a piece of it), Q: X [T, K]
  const int64_t* y;
  uint32_t tiles_p, tiles_q;
  int32_t nch;
  float2* part;                // forward: [parts][T]
  float* zt;                   // forward: [T], the target's logit
  // backward
  const float* lse;
  const float* c;              // [T] weights over their largest magnitude, 0 where ignored
  int64_t v0;                  // first vocabulary entry of the piece
  uint16_t* d;                 // dz of the piece [T, entries], blocked
  uint16_t* dt;                // and transposed [entries, T], blocked
  int32_t nd, nt;              // chunks of 64 entries and of 64 tokens in them, zero past the last one
};

// Logits of a tile reduced to one (r, s) per token and wave (16 TM entries), and the
// targets' logits: 16384 x 50304 over 1024 in 1.40 to 1.46 ms, 1.16 to 1.21 PFLOP/s with
// the epilogue (a library's product of that size, which stores its logits, 1.37 ms); the
// matrix units are busy 62% of cycles that power holds at 1.9 GHz.  What is rare is asked for once a wave: entries past the
// vocabulary's end, targets among the wave's entries, logits so large that a fused
// v c - r (one instruction instead of two; r the rounded m c, so nothing but the
// result is rounded) could overflow the exponential.
template <class T>
__global__ __launch_bounds__(T::NT, T::WAVES) void ce_fwd_kernel(CeArgs p) {
  __shared__ __attribute__((aligned(128))) typename T::Smem sm;
  const typename T::Items items(p.tiles_p, p.tiles_q, (uint32_t)p.nch, 1);
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 15, g = lane >> 4;
  T::run(p.P, p.Q, items, sm, [&](int64_t p0, int64_t q0, uint32_t, typename T::Acc& acc) __attribute__((always_inline)) {
    const int64_t pw = p0 + (w / T::kWN) * T::kTM * 16, qw = q0 + (w % T::kWN) * T::kTN * 16;
    const int there = (int)min(p.P.rows - pw, (int64_t)(16 * T::kTM));  // vocabulary entries of this wave
    const int mine = g * 4 * T::PB;                                     // this lane's first
    if (there < 16 * T::kTM) {
#pragma unroll
      for (int tm = 0; tm < T::kTM; ++tm)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (T::p_row(tm, 0, r) + mine >= there) {
#pragma unroll
            for (int tn = 0; tn < T::kTN; ++tn) acc[tm][tn][r] = -INFINITY;
          }
    }
    float2* part = p.part + pw / (16 * T::kTM) * p.Q.rows;
#pragma unroll
    for (int tn = 0; tn < T::kTN; ++tn) {
      const int64_t t = qw + T::q_row(tn, n);
      const bool in = t < p.Q.rows;
      const int64_t yw = in ? p.y[t] - pw : -1;
      const bool here = yw >= 0 && yw < there;
      if (__any(here)) {
        const int y = here ? (int)yw - mine : -1;
        float z = 0.0f;
        bool found = false;
#pragma unroll
        for (int tm = 0; tm < T::kTM; ++tm)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const bool is = T::p_row(tm, 0, r) == y;
            z = is ? acc[tm][tn][r] : z;
            found |= is;
            __builtin_amdgcn_sched_barrier(0);
          }
        if (found) p.zt[t] = z;
      }
      float m = -INFINITY;
#pragma unroll
      for (int tm = 0; tm < T::kTM; ++tm)
#pragma unroll
        for (int r = 0; r < 4; ++r) m = fmaxf(m, acc[tm][tn][r]);
      float r = m * kLog2e, s = 0.0f;
      const float b = m == -INFINITY ? 0.0f : r;
      if (__any(fabsf(m) > 0x1p24f && m != -INFINITY)) {
        const float mb = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int tm = 0; tm < T::kTM; ++tm)
#pragma unroll
          for (int k = 0; k < 4; ++k) s += exp_scaled(acc[tm][tn][k], mb, kLog2e);
      } else {
#pragma unroll
        for (int tm = 0; tm < T::kTM; ++tm)
#pragma unroll
          for (int k = 0; k < 4; ++k) s += __builtin_amdgcn_exp2f(fmaf(acc[tm][tn][k], kLog2e, -b));
      }
      join(r, s, __shfl_xor(r, 16), __shfl_xor(s, 16));
      join(r, s, __shfl_xor(r, 32), __shfl_xor(s, 32));
      if (g == 0 && in) part[t] = float2{r, s};
    }
  });
}

// The same for up to 64 tokens (scoring): one read of W, each lane's part of a token's
// sum kept over the wave's groups of 16 entries, one part a workgroup and token.  5 x
// 50304 over 1024 in 23 us, 4.5 TB/s of W.  Taken where the tokens fit the LDS: 16 over
// up to 2048 elements, 32 over 1024, 64 over 512.  Forward here and in tiles, join
// included, us: 5 tokens of 8000 x 1024 11.7 and 16.9, of 152000 x 1024 (W from memory)
// 56 and 70, 16 of 152000 x 2048 128 and 155, 64 of 152000 x 512 41.6 and 41.7; of W that
// the last cache holds from the call before, tiles catch up: 5 of 50304 x 1024 26.1 and
// 25.6, 32 of it 31.8 and 26.1, 64 of 50304 x 512 25.6 and 19.7.
template <class S, int TN>
__global__ __launch_bounds__(S::NT, 2) void ce_few_kernel(CeArgs p) {
  __shared__ typename S::Smem sm;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
  const int px = S::pitch(p.P.kb), whole = (p.P.kb + 127) / 128 * 8, T = (int)p.Q.rows;
  for (int i = threadIdx.x; i < S::TOKENS * whole; i += S::NT) {
    const int t = i / whole, c = (i - t * whole) * 16;
    uint4 v = {0u, 0u, 0u, 0u};
    if (t < T && c < p.P.kb) v = *reinterpret_cast<const uint4*>(p.Q.p + t * p.Q.ld + c);
    *reinterpret_cast<uint4*>(sm.x + t * px + c) = v;
  }
  __syncthreads();
  float r[TN], s[TN];
  int64_t y[TN];
#pragma unroll
  for (int tn = 0; tn < TN; ++tn) {
    r[tn] = -INFINITY;
    s[tn] = 0.0f;
    y[tn] = tn * 16 + n < T ? p.y[tn * 16 + n] : -1;
  }
  S::run(p.P, sm, [&](uint32_t group, const typename S::Acc& acc) __attribute__((always_inline)) {
    const int64_t v0 = (int64_t)group * 16 + g * 4;
#pragma unroll
    for (int tn = 0; tn < TN; ++tn) {
      float m = -INFINITY;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (v0 + k == y[tn]) p.zt[tn * 16 + n] = acc[tn][k];
        if (v0 + k < p.P.rows) m = fmaxf(m, acc[tn][k]);
      }
      if (v0 < p.P.rows) {
        float e = 0.0f;
        // four logits of -inf (masked entries) add nothing; their difference to m would be NaN
        const float mb = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (v0 + k < p.P.rows) e += exp_scaled(acc[tn][k], mb, kLog2e);
        join(r[tn], s[tn], m * kLog2e, e);
      }
    }
  });
  __syncthreads();  // the tokens in LDS are done with
  float2* sh = reinterpret_cast<float2*>(sm.x);
#pragma unroll
  for (int tn = 0; tn < TN; ++tn) {
    join(r[tn], s[tn], __shfl_xor(r[tn], 16), __shfl_xor(s[tn], 16));
    join(r[tn], s[tn], __shfl_xor(r[tn], 32), __shfl_xor(s[tn], 32));
    if (g == 0) sh[w * S::TOKENS + tn * 16 + n] = float2{r[tn], s[tn]};
  }
  __syncthreads();
  if (threadIdx.x < T) {
    float R = -INFINITY, e = 0.0f;
#pragma unroll
    for (int k = 0; k < S::WAVES; ++k) join(R, e, sh[k * S::TOKENS + threadIdx.x].x, sh[k * S::TOKENS + threadIdx.x].y);
    p.part[(int64_t)blockIdx.x * T + threadIdx.x] = float2{R, e};
  }
}

// Token by token: the parts of its sum joined (S shares of them at a time),
// the loss from the target's logit; a target outside the vocabulary gives NaN.
// 16384 tokens of 393 parts in 11 us, 4.7 TB/s; few tokens take a launch's 4.
template <int L, int S>
__global__ __launch_bounds__(L * S) void ce_join_kernel(const float2* part, int parts, const float* zt, const int64_t* y,
                                                       int64_t T, int64_t V, int64_t ignore, float* loss, float* lse) {
  __shared__ float2 sh[S][L];
  const int l = threadIdx.x % L, q = threadIdx.x / L;
  const int64_t t = (int64_t)blockIdx.x * L + l;
  float r = -INFINITY, s = 0.0f;
  if (t < T) {
    const int a = (int)((int64_t)parts * q / S), b = (int)((int64_t)parts * (q + 1) / S);
    const float2* at = part + (int64_t)a * T + t;
#pragma unroll 8
    for (int i = a; i < b; ++i, at += T) {
      const float2 v = *at;
      join(r, s, v.x, v.y);
    }
  }
  sh[q][l] = float2{r, s};
#pragma unroll
  for (int o = S / 2; o; o /= 2) {
    __syncthreads();
    if (q < o) {
      join(r, s, sh[q + o][l].x, sh[q + o][l].y);
      sh[q][l] = float2{r, s};
    }
  }
  if (q || t >= T) return;
  const float e = (r + __builtin_amdgcn_logf(s)) * kLn2;
  lse[t] = e;
  if (loss) {
    const int64_t k = y[t];
    loss[t] = k == ignore ? 0.0f : (uint64_t)k < (uint64_t)V ? e - zt[t] : kNan;
  }
}

// dz of a tile in bf16, both ways: 16384 x 8192 over 1024 in 290 us (16384 in 570 to 600),
// of which the product takes some 80% and the 4 bytes a logit the rest.
// bf16, the type of X and W, because the two products run on bf16 instructions: dz in two
// bf16 terms would double their work.  Each entry is off by half a step, 2^-8
// of itself, at most: the gradients of 16384 x 50304 in bf16 are then 2.0e-3 of their norm
// from the exact ones, and 1.7e-3 with dz in fp32.  Gradients asked for in fp32 have this
// dz too.
// The exponential is clamped to [0, 1], which costs nothing (an output modifier) and holds
// where the fused v c - r overflows; it turns a NaN into 0, so a token whose lse is NaN, or
// -inf (all its logits are), gets a NaN weight instead.
template <class T>
__global__ __launch_bounds__(T::NT, T::WAVES) void ce_dz_kernel(CeArgs p) {
  static_assert(T::kTN == 4 && T::PB == 4, "64 tokens, and entries 16 a lane");
  __shared__ __attribute__((aligned(128))) typename T::Smem sm;
  const typename T::Items items(p.tiles_p, p.tiles_q, (uint32_t)p.nch, 1);
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 15, g = lane >> 4;
  T::run(p.P, p.Q, items, sm, [&](int64_t p0, int64_t q0, uint32_t, typename T::Acc& acc) __attribute__((always_inline)) {
    const int64_t pw = p0 + (w / T::kWN) * T::kTM * 16, qw = q0 + (w % T::kWN) * 64, t0 = qw + n * 4;
    const int there = (int)min(p.P.rows - pw, (int64_t)(16 * T::kTM));
    const int mine = g * 16;
    float c[4], b[4];
    int y[4];
    bool any = false;
#pragma unroll
    for (int tn = 0; tn < 4; ++tn) {
      const bool in = t0 + tn < p.Q.rows;
      const float l = in ? p.lse[t0 + tn] : 0.0f;
      c[tn] = in ? p.c[t0 + tn] : 0.0f;
      if (!(l > -INFINITY) && c[tn] != 0.0f) c[tn] = kNan;  // NaN, or no entry of the token is left
      b[tn] = l * kLog2e;
      const int64_t yw = in ? p.y[t0 + tn] - p.v0 - pw : -1;
      const bool here = yw >= 0 && yw < there;
      y[tn] = here ? (int)yw - mine : -1;
      any |= here;
    }
#pragma unroll
    for (int tm = 0; tm < T::kTM; ++tm)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int tn = 0; tn < 4; ++tn)
          acc[tm][tn][r] = c[tn] * __builtin_amdgcn_fmed3f(__builtin_amdgcn_exp2f(fmaf(acc[tm][tn][r], kLog2e, -b[tn])), 0.0f, 1.0f);
    if (__any(any)) {
#pragma unroll
      for (int tm = 0; tm < T::kTM; ++tm) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int tn = 0; tn < 4; ++tn)
            acc[tm][tn][r] = T::p_row(tm, 0, r) == y[tn] ? acc[tm][tn][r] - c[tn] : acc[tm][tn][r];
        // (in this order: the compiler would first form all conditions, in more
        // registers than there are)
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (there < 16 * T::kTM) {
#pragma unroll
      for (int tm = 0; tm < T::kTM; ++tm)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (T::p_row(tm, 0, r) + mine >= there) {
#pragma unroll
            for (int tn = 0; tn < 4; ++tn) acc[tm][tn][r] = 0.0f;
          }
    }
    // transposed: four neighbouring tokens of an entry, 128 bytes over 16 lanes
    const int ct = (int)(qw >> 6);
    if (ct < p.nt) {
      uint16_t* dt = p.dt + ((pw >> 7) * p.nt + ct) * 8192 + ((pw & 127) + mine) * 64 + n * 4;
      static_assert(16 * T::kTM <= 128 && 128 % (16 * T::kTM) == 0, "a wave's entries are of one block");
#pragma unroll
      for (int tm = 0; tm < T::kTM; ++tm)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (T::p_row(tm, 0, r) + mine < there)
            *reinterpret_cast<uint2*>(dt + T::p_row(tm, 0, r) * 64) =
                uint2{bf16_pair(acc[tm][0][r], acc[tm][1][r]), bf16_pair(acc[tm][2][r], acc[tm][3][r])};
    }
    // as it is: 16 neighbouring entries of a token
#pragma unroll
    for (int tn = 0; tn < 4; ++tn) {
      const int64_t t = t0 + tn;
      if (t >= p.Q.rows) continue;
#pragma unroll
      for (int tb = 0; tb < T::kTM / 4; ++tb) {
        const int cd = (int)(pw >> 6) + tb;
        if (cd >= p.nd) continue;
        uint16_t* o = p.d + ((t >> 7) * p.nd + cd) * 8192 + (t & 127) * 64 + mine;
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          const float4_t a = acc[tb * 4 + k][tn], e = acc[tb * 4 + k + 1][tn];
          *reinterpret_cast<uint4*>(o + 4 * k) =
              uint4{bf16_pair(a.x, a.y), bf16_pair(a.z, a.w), bf16_pair(e.x, e.y), bf16_pair(e.z, e.w)};
        }
      }
    }
  });
}

// What the tile products read, in one launch: the first workgroup the tokens' weights,
// then a workgroup per 64 x 64 elements of X and of W.  Small backward passes are as
// long as their launches: 700 x 9000 over 96 took 49 us with a launch for each of
// these, each product and each join, and takes 35.
//
// Weights: c = w / max |w| (0 where the target is ignored) and that maximum: equal
// weights become 1, so that the bf16 of (softmax - 1) near a target is as exact as can
// be.
struct WeightArgs {
  const float* w;
  const int64_t* y;
  int64_t T, V, ignore;
  float *c, *top;
};
__device__ __forceinline__ void ce_weights(const WeightArgs& p) {
  __shared__ float sh[4];
  float m = 0.0f;
  // 16 tokens a thread at once, so that their loads are in flight together
  constexpr int N = 16;
  int64_t y[N];
  float w[N];
  auto load = [&](int64_t t0) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t t = min(t0 + i * 256 + threadIdx.x, p.T - 1);
      y[i] = p.y[t];
      w[i] = p.w[t];
    }
  };
  for (int64_t t0 = 0; t0 < p.T; t0 += N * 256) {
    load(t0);
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, y[i] != p.ignore ? fabsf(w[i]) : 0.0f);
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = m;
  __syncthreads();
  m = fmaxf(fmaxf(sh[0], sh[1]), fmaxf(sh[2], sh[3]));
  if (m == 0.0f) m = 1.0f;
  for (int64_t t0 = 0; t0 < p.T; t0 += N * 256) {
    if (p.T > N * 256) load(t0);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t t = t0 + i * 256 + threadIdx.x;
      if (t < p.T) p.c[t] = y[i] == p.ignore ? 0.0f : (uint64_t)y[i] < (uint64_t)p.V ? w[i] / m : kNan;
    }
  }
  if (threadIdx.x == 0) *p.top = m;
}

// A bf16 matrix [rows, cols] (cols a multiple of 16) into blocked operands: `copy`
// [rows, cols] and `turned` [cols, rows], zero up to whole chunks; either may be
// NULL.  64 x 64 through LDS.  Rows of ignored tokens (y, if not NULL) become zero:
// their dz is, but an infinity or NaN in them times zero would not be.
struct BlockArgs {
  const uint16_t* in;
  int64_t rows, cols, ld;
  uint16_t *copy, *turned;
  uint32_t nr, nc;  // chunks of rows and of columns
  const int64_t* y;
  int64_t ignore;
};
__device__ __forceinline__ void block_tile(const BlockArgs& p, uint32_t br, uint32_t bc) {
  __shared__ uint16_t tile[64][66];
  const int64_t r0 = (int64_t)br * 64, c0 = (int64_t)bc * 64;
  const int t = threadIdx.x;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = i * 32 + (t >> 3), c = (t & 7) * 8;
    uint4 v = {0u, 0u, 0u, 0u};
    if (r0 + r < p.rows && c0 + c < p.cols && !(p.y && p.y[r0 + r] == p.ignore)) v = *reinterpret_cast<const uint4*>(p.in + (r0 + r) * p.ld + c0 + c);
    if (p.copy && r0 + r < p.rows)
      *reinterpret_cast<uint4*>(p.copy + ((r0 >> 7) * p.nc + bc) * 8192 + ((r0 & 127) + r) * 64 + c) = v;
    uint32_t* s = reinterpret_cast<uint32_t*>(&tile[r][c]);
    s[0] = v.x; s[1] = v.y; s[2] = v.z; s[3] = v.w;
  }
  if (!p.turned) return;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = i * 32 + (t >> 3), r = (t & 7) * 8;
    if (c0 + c >= p.cols) continue;
    uint32_t v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = tile[r + 2 * k][c] | ((uint32_t)tile[r + 2 * k + 1][c] << 16);
    *reinterpret_cast<uint4*>(p.turned + ((c0 >> 7) * p.nr + br) * 8192 + ((c0 & 127) + c) * 64 + r) = uint4{v[0], v[1], v[2], v[3]};
  }
}

// weights: whether the first workgroup takes them
__global__ __launch_bounds__(256) void ce_prepare_kernel(WeightArgs w, int weights, Pair<BlockArgs> jobs) {
  uint32_t b = blockIdx.x;
  if (weights) {
    if (b == 0) return ce_weights(w);
    --b;
  }
  const int job = b < jobs.first ? 0 : 1;
  const BlockArgs& p = jobs.x[job];
  if (job) b -= jobs.first;
  block_tile(p, b % p.nr, b / p.nr);
}

// D[q, p] = sum_k Q[q, k] P[p, k] in bf16 operands:
//   splits > 1: fp32 partial sums [z][q][p];
//   else: fp32 sums kept in `sum` over the pieces (first: set, else added to).
struct ProductArgs {
  TileOp P, Q;
  uint32_t tiles_p, tiles_q;
  int32_t nch, splits, first;
  float* sum;      // splits > 1: partial
  void* out;       // final result (no sum kept): scaled by *scale
  const float* scale;
  int64_t ldo;
  int32_t bf16;
};

// One product or both of a piece: both of 16384 x 8192 over 1024 in 490 us, 1.12 PFLOP/s
// with the sums of dX read and written; 16384 x 1024 over 16384 alone in 430 to 500 us, 1.10
// to 1.28 PFLOP/s, the faster the cooler the GPU starts (2.0 GHz at first, 1.75 after some).
template <class T>
__global__ __launch_bounds__(T::NT, T::WAVES) void ce_product_kernel(Pair<ProductArgs> jobs) {
  __shared__ __attribute__((aligned(128))) typename T::Smem sm;
  const Share mine(jobs.first);
  const ProductArgs& p = jobs.x[mine.job];
  const typename T::Items items(p.tiles_p, p.tiles_q, (uint32_t)p.nch, (uint32_t)p.splits, mine.block, mine.blocks);
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
  T::run(p.P, p.Q, items, sm, [&](int64_t p0, int64_t q0, uint32_t z, typename T::Acc& acc) __attribute__((always_inline)) {
    const int64_t pw = p0 + (w / T::kWN) * T::kTM * 16 + g * 4 * T::PB, qw = q0 + (w % T::kWN) * T::kTN * 16 + n * T::kTN;
    const float scale = p.out ? *p.scale : 1.0f;
    float* sum = p.sum ? p.sum + (size_t)z * (size_t)p.Q.rows * (size_t)p.P.rows : nullptr;
#pragma unroll
    for (int tn = 0; tn < T::kTN; ++tn) {
      if (qw + tn >= p.Q.rows) continue;
#pragma unroll
      for (int tb = 0; tb < T::kTM / T::PB; ++tb) {
        const int64_t j = pw + tb * 16 * T::PB;
        // P has a multiple of 16 rows and a lane 4 PB = 16 of them
        if (j >= p.P.rows) continue;
        if (p.out) {
          float v[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = acc[tb * T::PB + k / 4][tn][k % 4] * scale;
          if (p.bf16) {
            uint16_t* o = reinterpret_cast<uint16_t*>(p.out) + (qw + tn) * p.ldo + j;
#pragma unroll
            for (int k = 0; k < 16; k += 8)
              *reinterpret_cast<uint4*>(o + k) = uint4{bf16_pair(v[k], v[k + 1]), bf16_pair(v[k + 2], v[k + 3]),
                                                      bf16_pair(v[k + 4], v[k + 5]), bf16_pair(v[k + 6], v[k + 7])};
          } else {
            float* o = reinterpret_cast<float*>(p.out) + (qw + tn) * p.ldo + j;
#pragma unroll
            for (int k = 0; k < 16; k += 4) *reinterpret_cast<float4*>(o + k) = float4{v[k], v[k + 1], v[k + 2], v[k + 3]};
          }
        } else {
          float4_t* o = reinterpret_cast<float4_t*>(sum + (qw + tn) * p.P.rows + j);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float4_t v = acc[tb * T::PB + k][tn];
            if (!p.first) v += o[k];
            o[k] = v;
          }
        }
      }
    }
  });
}

// dX of up to 64 tokens from W as it lies, one read of it: no turned copy.  A wave takes
// 64 columns of W (4 n to 4 n + 3 a lane, whole lines over 16 lanes) and 32 rows a step,
// eight a lane, whose halves it pairs into four operand tiles (tile c: columns 4 i + c),
// so that a lane's results are 16 neighbours of a token.  The waves of a workgroup take
// its rows in turn and join in LDS; workgroups split the rows, joined by ce_sum_kernel.
// Bound by the read of W: 16 x 50304 over 1024 in 19.7 us, 5.2 TB/s.
struct DxFewArgs {
  const uint16_t* W;
  int64_t ldw, T, K, V;
  const uint16_t* d;  // dz, blocked (T <= 64: rows of 64 entries in blocks of 128 rows)
  float* part;        // [splits][T][K]
  uint32_t blocks;    // of 64 columns
  int32_t steps, splits;
};
template <int TN>
__global__ __launch_bounds__(256, TN == 4 ? 2 : 4) void ce_dx_few_kernel(DxFewArgs p) {
  __shared__ __attribute__((aligned(16))) float sh[16 * TN][64 + 4];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
  const uint32_t kb = blockIdx.x % p.blocks, z = blockIdx.x / p.blocks;
  const int64_t k = (int64_t)kb * 64 + 4 * n;
  const bool in = k < p.K;
  const int s0 = (int)((int64_t)p.steps * z / p.splits), s1 = (int)((int64_t)p.steps * (z + 1) / p.splits);
  struct Step {
    uint2 w[8];
    i32x4_t d[TN];
  };
  auto fetch = [&](Step& f, int s) __attribute__((always_inline)) {
    const int64_t v = (int64_t)s * 32 + 8 * g;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f.w[j] = uint2{0u, 0u};
      if (in && s < s1 && v + j < p.V) f.w[j] = *reinterpret_cast<const uint2*>(p.W + (v + j) * p.ldw + k);
    }
    if (s < s1) {
#pragma unroll
      for (int tn = 0; tn < TN; ++tn)
        f.d[tn] = *reinterpret_cast<const i32x4_t*>(p.d + (v >> 6) * 8192 + (tn * 16 + n) * 64 + (v & 63));
    }
  };
  float4_t acc[4][TN] = {};
  auto multiply = [&](const Step& f) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      i32x4_t a;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = c < 2 ? f.w[2 * j].x : f.w[2 * j].y, hi = c < 2 ? f.w[2 * j + 1].x : f.w[2 * j + 1].y;
        a[j] = (int)__builtin_amdgcn_perm(hi, lo, c & 1 ? 0x07060302u : 0x05040100u);
      }
#pragma unroll
      for (int tn = 0; tn < TN; ++tn)
        acc[c][tn] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, f.d[tn]),
                                                             acc[c][tn], 0, 0, 0);
    }
  };
  Step f0, f1;
  fetch(f0, s0 + w);
  for (int s = s0 + w; s < s1; s += 8) {
    fetch(f1, s + 4);
    multiply(f0);
    fetch(f0, s + 8);
    if (s + 4 < s1) multiply(f1);
  }
  // the waves' sums, in their order; a lane's column 16 g + 4 r + c of token 16 tn + n
  for (int q = 0; q < 4; ++q) {
    if (w == q) {
#pragma unroll
      for (int tn = 0; tn < TN; ++tn)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float4_t* o = reinterpret_cast<float4_t*>(&sh[tn * 16 + n][16 * g + 4 * r]);
          float4_t v = {acc[0][tn][r], acc[1][tn][r], acc[2][tn][r], acc[3][tn][r]};
          if (q) v += *o;
          *o = v;
        }
    }
    __syncthreads();
  }
  float* out = p.part + (size_t)z * (size_t)(p.T * p.K);
  for (int i = threadIdx.x; i < 16 * TN * 16; i += 256) {
    const int64_t t = i >> 4, col = (int64_t)kb * 64 + (i & 15) * 4;
    if (t < p.T && col < p.K) *reinterpret_cast<float4_t*>(out + t * p.K + col) = *reinterpret_cast<const float4_t*>(&sh[t][(i & 15) * 4]);
  }
}

// out = scale * (sum of `parts` fp32 slices), in order; 4 a thread (n a multiple of 16).
// One result or two.  Bound by memory: 16384 x 1024 fp32 to bf16 in 15 us.
struct SumArgs {
  const float* sum;
  int parts, bf16;
  int64_t n;
  const float* scale;
  void* out;
};
__global__ __launch_bounds__(256) void ce_sum_kernel(Pair<SumArgs> jobs) {
  const Share mine(jobs.first);
  const SumArgs& p = jobs.x[mine.job];
  const int64_t i = ((int64_t)mine.block * 256 + threadIdx.x) * 4, n = p.n;
  if (i >= n) return;
  float4_t v = *reinterpret_cast<const float4_t*>(p.sum + i);
#pragma unroll 8
  for (int z = 1; z < p.parts; ++z) v += *reinterpret_cast<const float4_t*>(p.sum + (size_t)z * (size_t)n + i);
  const float s = *p.scale;
  v *= s;
  if (p.bf16) *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + i) = uint2{bf16_pair(v.x, v.y), bf16_pair(v.z, v.w)};
  else *reinterpret_cast<float4_t*>(reinterpret_cast<float*>(p.out) + i) = v;
}

// sum slice 0 (kept over the pieces) += the piece's slices, in order; bound by memory as
// ce_sum_kernel
__global__ __launch_bounds__(256) void ce_fold_kernel(float* kept, const float* part, int parts, int64_t n, int first) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  float4_t v = *reinterpret_cast<const float4_t*>(part + i);
#pragma unroll 8
  for (int z = 1; z < parts; ++z) v += *reinterpret_cast<const float4_t*>(part + (size_t)z * (size_t)n + i);
  if (!first) v += *reinterpret_cast<const float4_t*>(kept + i);
  *reinterpret_cast<float4_t*>(kept + i) = v;
}

using TileBig = Tile<EL_BF16, 2, 4, 8, 4>;  // 256 x 256
using TileMid = Tile<EL_BF16, 2, 2, 4, 4>;  // 128 x 128

int64_t tiles_of(int64_t p, int64_t q, int64_t b) { return (p + b - 1) / b * ((q + b - 1) / b); }

// Estimated time (us on MI355X) of `items` tiles over `chunks` chunks of 64 elements:
// a tile of 256 takes 1.9 a chunk and `fixed` for its start and results, one of 128
// 1.1 alone on its CU and 1.5 beside another, and half of `fixed`.
double tile_time(bool big, int64_t items, double chunks, double fixed) {
  if (big) return (double)((items + kCus - 1) / kCus) * (chunks * 1.9 + fixed);
  const int64_t full = items / (2 * kCus), rest = items % (2 * kCus);
  return (double)full * (chunks * 1.5 + fixed / 2) + (rest ? chunks * (rest > kCus ? 1.5 : 1.1) + fixed / 2 : 0.0);
}
// 256 x 256 tiles for the logits of V entries and T tokens, else 128 x 128 (forward of
// 1235 x 32003 over 528: 65.4 and 76.9 us; 777 x 5000 over 1024: 31.6 and 24.6).
bool ce_big(int64_t V, int64_t T, int64_t K) {
  const double chunks = (double)((K + 63) / 64);
  return tile_time(true, tiles_of(V, T, 256), chunks, 9.0) < tile_time(false, tiles_of(V, T, 128), chunks, 9.0);
}
// Splits of a product of p by q results over k in tiles of one size, and its time (the
// whole backward of 1235 x 32003 over 528: 192 us with unsplit products, 174 with 8 to
// 16 splits).
struct ProductPlan {
  bool big;
  int splits;
  double time;
};
ProductPlan product_plan(int64_t p, int64_t q, int64_t k, bool big) {
  ProductPlan best = {big, 1, 1e30};
  const int64_t nch = (k + 63) / 64;
  for (int z = 1; z <= 32 && z * 8 <= std::max<int64_t>(nch, 8); z *= 2) {
    double t = tile_time(big, tiles_of(p, q, big ? 256 : 128) * z, (double)((nch + z - 1) / z), 6.0);
    if (z > 1) t += 3.0 + (double)p * (double)q * 8.0 * z / 6e6;
    if (t < best.time) best = ProductPlan{big, z, t};
  }
  return best;
}
// Of a piece's products, dX (x) and dW (w; either may not be asked for).  Two of one
// tile run in one launch, where the second fills what the first leaves idle: about 10
// us (backward of 200 x 50304 over 1024: 193 us with a tile of 128 for dX and 256 for
// dW, 180 with 128 and 169 with 256 for both; of 500 x 8000 over 304 39.5 with 128 for
// both, 53.7 with 256).
struct CePlans {
  ProductPlan x[2], w[2];  // of tiles of 128 and 256
  CePlans(int64_t T, int64_t K, int64_t vn)
      : x{product_plan(K, T, vn, false), product_plan(K, T, vn, true)},
        w{product_plan(K, vn, T, false), product_plan(K, vn, T, true)} {}
  // the tiles, as indexes of x and w, and the time of those asked for
  double pick(bool dx, bool dw, int& ix, int& iw) const {
    double least = 1e30;
    for (int i = 0; i < 4; ++i) {
      const double t = (dx ? x[i & 1].time : 0.0) + (dw ? w[i >> 1].time : 0.0) - (dx && dw && (i & 1) == i >> 1 ? 10.0 : 0.0);
      if (t < least) {
        least = t;
        ix = i & 1;
        iw = i >> 1;
      }
    }
    return least;
  }
};

template <class T>
void launch_fwd_tile(CeArgs a, hipStream_t s) {
  a.tiles_p = (uint32_t)((a.P.rows + T::BM - 1) / T::BM);
  a.tiles_q = (uint32_t)((a.Q.rows + T::BN - 1) / T::BN);
  ce_fwd_kernel<T><<<T::grid((uint64_t)a.tiles_p * a.tiles_q), T::NT, 0, s>>>(a);
}
// 1 to 4 tiles of 16 tokens, where their operand fits the LDS of ce_few_kernel
template <int TN>
bool launch_few(const CeArgs& a, uint32_t grid, hipStream_t s) {
  using Few = Skinny<EL_BF16, TN, 66 * 1024>;
  if (a.Q.rows > Few::TOKENS || !Few::fits(a.Q.rows, a.P.kb)) return false;
  ce_few_kernel<Few, TN><<<grid, Few::NT, 0, s>>>(a);
  return true;
}
uint32_t few_grid(int64_t V) { return Skinny<EL_BF16, 1, 66 * 1024>::grid(V); }
bool few_fits(int64_t T, int64_t K) {
  return Skinny<EL_BF16, 1, 66 * 1024>::fits(T, K * 2) || Skinny<EL_BF16, 2, 66 * 1024>::fits(T, K * 2) ||
         Skinny<EL_BF16, 4, 66 * 1024>::fits(T, K * 2);
}

template <class T>
void launch_dz_tile(CeArgs a, hipStream_t s) {
  a.tiles_p = (uint32_t)((a.P.rows + T::BM - 1) / T::BM);
  a.tiles_q = (uint32_t)((a.Q.rows + T::BN - 1) / T::BN);
  ce_dz_kernel<T><<<T::grid((uint64_t)a.tiles_p * a.tiles_q), T::NT, 0, s>>>(a);
}
template <class T>
uint32_t product_tiles(ProductArgs& x) {
  x.tiles_p = (uint32_t)((x.P.rows + T::BM - 1) / T::BM);
  x.tiles_q = (uint32_t)((x.Q.rows + T::BN - 1) / T::BN);
  return T::grid((uint64_t)x.tiles_p * x.tiles_q * (uint32_t)x.splits);
}
// Up to two products of one tile in one launch.
template <class T>
void launch_products(ProductArgs* x, int n, hipStream_t s) {
  const uint32_t first = product_tiles<T>(x[0]), others = n > 1 ? product_tiles<T>(x[1]) : 0;
  ce_product_kernel<T><<<first + others, T::NT, 0, s>>>(Pair<ProductArgs>{{x[0], x[n - 1]}, first});
}
void launch_sums(const SumArgs* x, int n, hipStream_t s) {
  auto grid = [](const SumArgs& a) { return (uint32_t)((a.n / 4 + 255) / 256); };
  const uint32_t first = grid(x[0]);
  ce_sum_kernel<<<first + (n > 1 ? grid(x[1]) : 0), 256, 0, s>>>(Pair<SumArgs>{{x[0], x[n - 1]}, first});
}

TileOp bf16_operand(const void* p, int64_t rows, int64_t cols, int64_t ld) {
  TileOp o = {};
  o.p = reinterpret_cast<const uint8_t*>(p);
  o.rows = rows;
  o.ld = ld * 2;
  o.cs = 128;
  o.bs = 128 * o.ld;
  o.kb = (int32_t)(cols * 2);
  return o;
}

// A workspace operand in blocks of 128 rows by 64 columns.
TileOp blocked_operand(const void* p, int64_t rows, int64_t cols) {
  TileOp o = {};
  o.p = reinterpret_cast<const uint8_t*>(p);
  o.rows = rows;
  o.ld = 128;
  o.cs = 128 * 128;
  o.bs = (cols + 63) / 64 * o.cs;
  o.kb = (int32_t)(cols * 2);
  return o;
}

int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }
size_t blocked_bytes(int64_t rows, int64_t cols) { return (size_t)(up(rows, 128) * up(cols, 64) * 2); }

// Tokens from which the operands of the logits are copied into blocks first.
constexpr int64_t kBlockTokens = 2048;

struct CeFwdSpace {
  size_t part, zt, xb, wb, bytes;
  int64_t parts;
  bool few, big, blocked;
};
CeFwdSpace ce_fwd_space(int64_t T, int64_t K, int64_t V) {
  CeFwdSpace s;
  size_t at = 0;
  auto take = [&](size_t n) { const size_t a = at; at += up256(n); return a; };
  s.blocked = T >= kBlockTokens;
  s.few = few_fits(T, K);
  s.big = ce_big(V, T, K);
  const int64_t per = s.big ? 16 * TileBig::kTM : 16 * TileMid::kTM;  // entries of a part
  s.parts = s.few ? few_grid(V) : (V + per - 1) / per;
  s.part = take((size_t)(s.few ? s.parts : up(V, 256) / per) * (size_t)T * 8);
  s.zt = take((size_t)T * 4);
  s.xb = take(s.blocked ? blocked_bytes(T, K) : 0);
  s.wb = take(s.blocked ? blocked_bytes(V, K) : 0);
  s.bytes = at;
  return s;
}

// Whether dX is taken from W as it lies: few tokens, and a W of 2^22 elements, whose
// turned copy costs more than the launch that this adds (backward with the copy and
// without: 16 x 50304 over 1024 124 and 79 us, 40 tokens 125 and 88, 30 x 8000 over 704 41
// and 37; 50 x 20000 over 128 33 and 36, 20 x 1000 over 64 20 and 23; 100 x 50304 over
// 1024, with sums that no longer fit the registers, 138 and 171).
bool dx_few(int64_t T, int64_t K, int64_t V) { return T <= 64 && K * V >= (int64_t)1 << 22; }
// Workgroups over the rows of W: as many as run at once, of 16 steps of 32 rows at least
int dx_few_splits(int64_t K, int64_t V) {
  const int64_t steps = (V + 31) / 32, blocks = (K + 63) / 64;
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(32, steps / 16), 4 * kCus / blocks));
}

// Partial sums of a piece's split products, whichever gradients are asked for.
size_t split_bytes(const CePlans& plans, int64_t T, int64_t K, int64_t vn, bool few) {
  size_t part = 0;
  for (int want = 1; want < 4; ++want) {
    int ix = 0, iw = 0;
    plans.pick((want & 1) && !few, want & 2, ix, iw);
    const int zx = few || !(want & 1) ? 1 : plans.x[ix].splits, zw = want & 2 ? plans.w[iw].splits : 1;
    part = std::max(part, (zx > 1 ? (size_t)zx * (size_t)(T * K * 4) : 0) + (zw > 1 ? (size_t)zw * (size_t)(vn * K * 4) : 0));
  }
  return part;
}

// Vocabulary entries of a piece of the backward (a multiple of 256).  What the workspace
// holds of a piece - dz twice, 4 bytes a logit, copies of its rows of W and the split
// products' sums - takes at most half of what bf16 logits of all entries would, though 384
// MiB may always be used and never more than 1 GiB, and 1024 entries are taken in any case.
// Each piece costs launches, a read and write of dX's sums and rounds of tiles that it
// leaves partly idle, so of the sizes from the largest to its half the one of the least
// estimated time is taken.  Backward with this rule, and with pieces of 2^28 logits
// whatever they take: 16384 x 50304 over 1024 5.01 ms in 772 MB, 4.78 in 1313; 5000 x
// 50304 1.75 ms in 395 MB, 1.72 in 1602; 4096 x 50304 1.32 ms in 436 MB, 1.31 in 1134;
// 9000 x 20000 over 512 0.87 ms in 407 MB, 0.72 in 958; 1024 x 131072 over 4096 3.47 ms in
// 294 MB, 3.20 in 1703; 1235 x 32003 over 528 is one piece in both.
int64_t ce_piece(int64_t T, int64_t K, int64_t V) {
  const int64_t all = (V + 255) / 256;
  if (T <= 64) return all * 256;  // dX of few tokens takes W at once; dz takes 384 bytes an entry
  const int64_t entry = 2 * (up(T, 128) + up(T, 64) + up(K, 128) + (T >= kBlockTokens ? up(K, 64) : 0));
  const int64_t room = std::clamp<int64_t>(T * V, (int64_t)3 << 27, (int64_t)1 << 30);
  const int64_t most = std::min(all, std::max<int64_t>(room / (256 * entry), 4));
  struct Cost {
    double time;
    size_t split;
  };
  auto cost = [&](int64_t vn) {
    const double chunks = (double)((K + 63) / 64);
    const CePlans plans(T, K, vn);
    int ix = 0, iw = 0;
    return Cost{std::min(tile_time(true, tiles_of(vn, T, 256), chunks, 9.0), tile_time(false, tiles_of(vn, T, 128), chunks, 9.0)) +
                    plans.pick(true, true, ix, iw) + 20.0 + (double)(T * K) * 8.0 / 5e6,
                split_bytes(plans, T, K, vn, false)};
  };
  int64_t best = 4;
  double least = 1e30;
  for (int64_t n = most; n >= std::max<int64_t>((most + 1) / 2, 4); n -= std::max<int64_t>(1, most / 32)) {
    const int64_t whole = V / (n * 256), rest = V - whole * n * 256;
    const Cost a = cost(std::min(n * 256, V)), b = rest && whole ? cost(rest) : Cost{0.0, 0};
    if ((size_t)(n * 256 * entry) + std::max(a.split, b.split) > (size_t)room) continue;
    if (n == all) return n * 256;
    if (const double time = (double)std::max<int64_t>(whole, 1) * a.time + b.time; time < least) {
      least = time;
      best = n;
    }
  }
  return std::min(best, all) * 256;
}

struct CeBwdSpace {
  size_t c, top, xb, xt, wb, wt, d, dt, dx, part, bytes;
  int64_t piece;
  bool blocked, few;
};
CeBwdSpace ce_bwd_space(int64_t T, int64_t K, int64_t V) {
  CeBwdSpace s;
  s.few = dx_few(T, K, V);
  s.piece = ce_piece(T, K, V);
  s.blocked = T >= kBlockTokens;
  size_t at = 0;
  auto take = [&](size_t n) { const size_t a = at; at += up256(n); return a; };
  s.c = take((size_t)T * 4);
  s.top = take(4);
  s.xb = take(s.blocked ? blocked_bytes(T, K) : 0);
  s.xt = take(blocked_bytes(K, T));
  s.wb = take(s.blocked ? blocked_bytes(s.piece, K) : 0);
  s.wt = take(s.few ? 0 : blocked_bytes(K, s.piece));
  s.d = take(blocked_bytes(T, s.piece));
  s.dt = take(blocked_bytes(s.piece, T));
  s.dx = take(s.piece < V ? (size_t)(T * K * 4) : 0);
  // partial sums of split products, of a whole piece and of the last one
  size_t part = 0;
  for (const int64_t vn : {std::min(s.piece, V), V % s.piece})
    if (vn) part = std::max(part, split_bytes(CePlans(T, K, vn), T, K, vn, s.few));
  if (s.few) part += (size_t)dx_few_splits(K, V) * (size_t)(T * K * 4);
  s.part = take(part);
  s.bytes = at;
  return s;
}

BlockArgs block_args(const void* in, int64_t rows, int64_t cols, int64_t ld, void* copy, void* turned) {
  return BlockArgs{reinterpret_cast<const uint16_t*>(in), rows,
                   cols, ld, reinterpret_cast<uint16_t*>(copy),
                   reinterpret_cast<uint16_t*>(turned), (uint32_t)((rows + 63) / 64), (uint32_t)((cols + 63) / 64), nullptr, 0};
}
// w, x: NULL for none
void launch_prepare(const WeightArgs* w, const BlockArgs* x, const BlockArgs& v, hipStream_t s) {
  const WeightArgs no_weights = {};
  const BlockArgs none = {};
  const uint32_t grid = (w ? 1 : 0) + (x ? x->nr * x->nc : 0) + v.nr * v.nc;
  ce_prepare_kernel<<<grid, 256, 0, s>>>(w ? *w : no_weights, w != nullptr, Pair<BlockArgs>{{x ? *x : none, v}, x ? x->nr * x->nc : 0});
}

}  // namespace

size_t ce_fwd_workspace_bytes(int64_t T, int64_t K, int64_t V) { return ce_fwd_space(T, K, V).bytes; }

#define TJ2_STEP()                                                      \
  do {                                                                  \
    if (hipError_t e_ = hipGetLastError(); e_ != hipSuccess) return e_; \
  } while (0)

hipError_t launch_ce_fwd(const CeParams& c, void* ws, hipStream_t s) {
  const CeFwdSpace sp = ce_fwd_space(c.T, c.K, c.V);
  uint8_t* w = reinterpret_cast<uint8_t*>(ws);
  CeArgs a = {};
  if (sp.blocked) {
    const BlockArgs x = block_args(c.X, c.T, c.K, c.ldx, w + sp.xb, nullptr);
    launch_prepare(nullptr, &x, block_args(c.W, c.V, c.K, c.ldw, w + sp.wb, nullptr), s);
    TJ2_STEP();
    a.P = blocked_operand(w + sp.wb, c.V, c.K);
    a.Q = blocked_operand(w + sp.xb, c.T, c.K);
  } else {
    a.P = bf16_operand(c.W, c.V, c.K, c.ldw);
    a.Q = bf16_operand(c.X, c.T, c.K, c.ldx);
  }
  a.y = c.y;
  a.nch = (int32_t)(up(c.K, 64) / 64);
  a.part = reinterpret_cast<float2*>(w + sp.part);
  a.zt = reinterpret_cast<float*>(w + sp.zt);
  if (sp.few) {
    const uint32_t grid = few_grid(c.V);
    if (!launch_few<1>(a, grid, s) && !launch_few<2>(a, grid, s)) launch_few<4>(a, grid, s);
  } else if (sp.big) {
    launch_fwd_tile<TileBig>(a, s);
  } else {
    launch_fwd_tile<TileMid>(a, s);
  }
  TJ2_STEP();
  // few tokens and many parts: many threads a token
  if (c.T <= 2048 && sp.parts > 64) ce_join_kernel<16, 64><<<(uint32_t)((c.T + 15) / 16), 1024, 0, s>>>(a.part, (int)sp.parts, a.zt, c.y, c.T, c.V, c.ignore, c.loss, c.lse);
  else ce_join_kernel<64, 4><<<(uint32_t)((c.T + 63) / 64), 256, 0, s>>>(a.part, (int)sp.parts, a.zt, c.y, c.T, c.V, c.ignore, c.loss, c.lse);
  return hipGetLastError();
}

size_t ce_bwd_workspace_bytes(int64_t T, int64_t K, int64_t V) { return ce_bwd_space(T, K, V).bytes; }

hipError_t launch_ce_bwd(const CeParams& c, void* ws, hipStream_t s) {
  const CeBwdSpace sp = ce_bwd_space(c.T, c.K, c.V);
  uint8_t* w = reinterpret_cast<uint8_t*>(ws);
  float* top = reinterpret_cast<float*>(w + sp.top);
  float *dx = reinterpret_cast<float*>(w + sp.dx), *part = reinterpret_cast<float*>(w + sp.part);
  const WeightArgs weights = {c.dloss, c.y, c.T, c.V, c.ignore, reinterpret_cast<float*>(w + sp.c), top};
  BlockArgs xb = block_args(c.X, c.T, c.K, c.ldx, sp.blocked ? w + sp.xb : nullptr, w + sp.xt);
  xb.y = c.y;
  xb.ignore = c.ignore;
  const bool one = sp.piece >= c.V;
  for (int64_t v0 = 0; v0 < c.V; v0 += sp.piece) {
    const int64_t vn = std::min(sp.piece, c.V - v0);
    const uint16_t* W = reinterpret_cast<const uint16_t*>(c.W) + v0 * c.ldw;
    launch_prepare(v0 ? nullptr : &weights, v0 ? nullptr : &xb,
                   sp.few ? BlockArgs{} : block_args(W, vn, c.K, c.ldw, sp.blocked ? w + sp.wb : nullptr, w + sp.wt), s);
    TJ2_STEP();
    CeArgs a = {};
    a.P = sp.blocked ? blocked_operand(w + sp.wb, vn, c.K) : bf16_operand(W, vn, c.K, c.ldw);
    a.Q = sp.blocked ? blocked_operand(w + sp.xb, c.T, c.K) : bf16_operand(c.X, c.T, c.K, c.ldx);
    a.y = c.y;
    a.nch = (int32_t)(up(c.K, 64) / 64);
    a.lse = c.lse;
    a.c = reinterpret_cast<float*>(w + sp.c);
    a.v0 = v0;
    a.d = reinterpret_cast<uint16_t*>(w + sp.d);
    a.dt = reinterpret_cast<uint16_t*>(w + sp.dt);
    a.nd = (int32_t)(up(vn, 64) / 64);
    a.nt = (int32_t)(up(c.T, 64) / 64);
    if (ce_big(vn, c.T, c.K)) launch_dz_tile<TileBig>(a, s);
    else launch_dz_tile<TileMid>(a, s);
    TJ2_STEP();
    // dX += dz W and dW = dz^T X of the piece; split products leave partial sums
    const CePlans plans(c.T, c.K, vn);
    int ix = 0, iw = 0;
    plans.pick(c.dX && !sp.few, c.dW, ix, iw);
    ProductArgs x[2];
    bool big[2];
    int n = 0;
    SumArgs sums[2];
    int joins = 0;
    float* at = part;
    const int64_t nx = c.T * c.K, nw = vn * c.K;
    const bool last = v0 + vn == c.V;
    bool fold = false;
    if (c.dX && sp.few) {
      DxFewArgs x = {};
      x.W = W;
      x.ldw = c.ldw;
      x.T = c.T;
      x.K = c.K;
      x.V = vn;
      x.d = a.d;
      x.part = at;
      x.blocks = (uint32_t)((c.K + 63) / 64);
      x.steps = (int32_t)((vn + 31) / 32);
      x.splits = dx_few_splits(c.K, vn);
      const uint32_t grid = x.blocks * (uint32_t)x.splits;
      if (c.T <= 16) ce_dx_few_kernel<1><<<grid, 256, 0, s>>>(x);
      else if (c.T <= 32) ce_dx_few_kernel<2><<<grid, 256, 0, s>>>(x);
      else ce_dx_few_kernel<4><<<grid, 256, 0, s>>>(x);
      TJ2_STEP();
      sums[joins++] = SumArgs{at, x.splits, c.dx_dtype == TJ2_BF16, nx, top, c.dX};
      at += (size_t)x.splits * (size_t)nx;
    } else if (c.dX) {
      const ProductPlan& plan = plans.x[ix];
      ProductArgs& q = x[n];
      q = {};
      q.P = blocked_operand(w + sp.wt, c.K, up(vn, 64));
      q.Q = blocked_operand(w + sp.d, c.T, up(vn, 64));
      q.nch = a.nd;
      q.splits = plan.splits;
      q.scale = top;
      q.bf16 = c.dx_dtype == TJ2_BF16;
      q.ldo = c.K;
      q.first = q.splits > 1 || v0 == 0;
      if (q.splits > 1) {
        q.sum = at;
        at += (size_t)q.splits * (size_t)nx;
      } else if (one) {
        q.out = c.dX;
      } else {
        q.sum = dx;
      }
      fold = q.splits > 1 && !one;
      if (q.splits > 1 && one) sums[joins++] = SumArgs{part, q.splits, q.bf16, nx, top, c.dX};
      if (!one && last) sums[joins++] = SumArgs{dx, 1, q.bf16, nx, top, c.dX};
      big[n++] = plan.big;
    }
    if (c.dW) {
      const ProductPlan& plan = plans.w[iw];
      ProductArgs& q = x[n];
      q = {};
      q.P = blocked_operand(w + sp.xt, c.K, up(c.T, 64));
      q.Q = blocked_operand(w + sp.dt, vn, up(c.T, 64));
      q.nch = a.nt;
      q.splits = plan.splits;
      q.scale = top;
      q.bf16 = c.dw_dtype == TJ2_BF16;
      q.ldo = c.K;
      q.first = 1;
      uint8_t* out = reinterpret_cast<uint8_t*>(c.dW) + (size_t)(v0 * c.K) * (q.bf16 ? 2 : 4);
      if (q.splits > 1) {
        q.sum = at;
        sums[joins++] = SumArgs{at, q.splits, q.bf16, nw, top, out};
      } else {
        q.out = out;
      }
      big[n++] = plan.big;
    }
    // in one launch where they take the same tile
    for (int i = 0; i < n;) {
      const int k = i + 1 < n && big[i] == big[i + 1] ? 2 : 1;
      if (big[i]) launch_products<TileBig>(x + i, k, s);
      else launch_products<TileMid>(x + i, k, s);
      TJ2_STEP();
      i += k;
    }
    if (fold) {
      ce_fold_kernel<<<(uint32_t)((nx / 4 + 255) / 256), 256, 0, s>>>(dx, part, x[0].splits, nx, v0 == 0);
      TJ2_STEP();
    }
    if (joins) launch_sums(sums, joins, s);
    TJ2_STEP();
  }
  return hipSuccess;
}
#undef TJ2_STEP

// ---- distillation -------------------------------------------------------------------
namespace {

constexpr int kDistillMaxK = 512;

template <class T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<uint16_t>(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t from_f32<uint16_t>(float v) { return (uint16_t)bf16_pair(v, 0.0f); }

// 16 bytes as floats and back
template <class T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(const uint4& q, float (&v)[4]) {
    v[0] = __uint_as_float(q.x); v[1] = __uint_as_float(q.y); v[2] = __uint_as_float(q.z); v[3] = __uint_as_float(q.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&v)[4]) {
    return uint4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
  }
};
template <>
struct Vec<uint16_t> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(const uint4& q, float (&v)[8]) {
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&v)[8]) {
    return uint4{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
  }
};

struct MaxOp {
  // NaN is kept: a row with one has a NaN loss
  __device__ __forceinline__ float operator()(float a, float b) const { return a > b || a != a ? a : b; }
};
struct SumOp {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};

// 16 bytes that pass through once: without the caches' keeping them
__device__ __forceinline__ uint4 stream_load(const uint4* p) {
  return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p)));
}
__device__ __forceinline__ void stream_store(uint4* p, const uint4& v) {
  __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, v), reinterpret_cast<u32x4_t*>(p));
}

// K values of every thread reduced over the workgroup (sh: its own LDS per call).
template <int WAVES, int K, class F>
__device__ __forceinline__ void block_reduce(float (&v)[K], float (*sh)[K], F f) {
#pragma unroll
  for (int o = 32; o; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = f(v[k], __shfl_xor(v[k], o));
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) sh[threadIdx.x >> 6][k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    v[k] = sh[threadIdx.x % WAVES][k];
#pragma unroll
    for (int o = WAVES / 2; o; o >>= 1) v[k] = f(v[k], __shfl_xor(v[k], o));
  }
}

struct DistillArgs {
  const void* z;
  void* dz;
  int64_t ldz, ldd;
  const int32_t* ids;
  const void* u;
  const int64_t* y;      // optional
  const float* w;        // row weights of the gradient
  float* loss;           // optional
  int64_t T, V, ignore;
  int32_t k;
  float tau, alpha;
};

// One token.  R > 0: the row's 16-byte vectors in registers, R a thread (logits
// are read once); R = 0: the row is read again for each of the three passes.
// Elements before the first and after the last aligned vector are one per thread;
// HARD: the hard target's term is there too (a second sum of exponentials at
// temperature 1).  Bound by memory: 16384 x 50304 bf16 with 64 entries in 635 us, 5.2
// TB/s, a large copy's rate.
template <class T, int R, bool HARD, int kThreads>
__global__ __launch_bounds__(kThreads, R <= 8 ? 8 : R <= 13 ? 6 : 4) void distill_kernel(DistillArgs p) {
  constexpr int N = Vec<T>::N, WAVES = kThreads / 64;
  constexpr int RR = R > 0 ? R : 1;
  __shared__ float sh_max[WAVES][2], sh_sum[WAVES][4];
  __shared__ __attribute__((aligned(16))) int32_t id[kDistillMaxK];
  __shared__ float pr[kDistillMaxK];
  // what the few entries' threads keep meanwhile: in registers it would be spilled
  __shared__ float keep_u[kDistillMaxK], keep_z[kDistillMaxK], keep_edge[16], keep_target;
  __shared__ uint8_t keep_flags[kDistillMaxK];  // 1: the first place that lists its entry, 2: not the only one
  __shared__ int32_t named;  // the hard target is among the teacher's entries
  const int t = threadIdx.x;
  const int64_t row = blockIdx.x;
  const T* z = reinterpret_cast<const T*>(p.z) + row * p.ldz;
  T* dz = p.dz ? reinterpret_cast<T*>(p.dz) + row * p.ldd : nullptr;
  const int V = (int)p.V;  // at most 2^30
  const int64_t y = p.y ? p.y[row] : 0;
  const bool on = !p.y || y != p.ignore;
  const float w = p.w ? p.w[row] : 1.0f;

  // aligned middle [head, head + N * nv)
  const int head = min((int)(((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) / sizeof(T)), V);
  const int nv = (V - head) / N;
  const int tail = V - head - nv * N;
  const uint4* zv = reinterpret_cast<const uint4*>(z + head);
  const bool edge = t < head + tail;
  const int ei = t < head ? t : V - tail + (t - head);
  // the gradient's vectors: the same places, if its row is aligned alike
  const bool vec_out = dz && (((reinterpret_cast<uintptr_t>(dz) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0);

  if (!on) {  // no loss and no gradient
    if (t == 0 && p.loss) p.loss[row] = 0.0f;
    if (dz) {
      if (vec_out)
        for (int i = t; i < nv; i += kThreads) reinterpret_cast<uint4*>(dz + head)[i] = uint4{0u, 0u, 0u, 0u};
      else
        for (int i = t; i < nv * N; i += kThreads) dz[head + i] = from_f32<T>(0.0f);
      if (edge) dz[ei] = from_f32<T>(0.0f);
    }
    return;
  }

  uint4 q[RR];
  auto vec = [&](int r, int i) __attribute__((always_inline)) -> uint4 {
    if constexpr (R > 0) return q[r];
    return zv[i];
  };
  // f(r, i) for each of this thread's vectors i
  auto each = [&](auto&& f) __attribute__((always_inline)) {
    if constexpr (R > 0) {
      // the places are worked out again in each pass: kept from the loads to the stores
      // they would be spilled (16384 rows of 50304 bf16: 0.3 GB beside the 3.3 GB of
      // logits, 623 to 690 us by where the buffers lie, 635 without)
      int at = t;
      asm volatile("" : "+v"(at));
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int i = at + r * kThreads;
        if (i < nv) f(r, i);
        // one vector at a time: interleaved, their temporaries would take the
        // registers that let another row share the CU
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      for (int i = t; i < nv; i += kThreads) f(0, i);
    }
  };
  if constexpr (R > 0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = t + r * kThreads;
      if (i < nv) q[r] = stream_load(zv + i);
    }
  }
  const float ze = edge ? to_f32<T>(z[ei]) : 0.0f;
  if (edge) keep_edge[t] = ze;
  // read before anything is written: dz may be z
  if (HARD && t == 0) {
    keep_target = (uint64_t)y < (uint64_t)V ? to_f32<T>(z[y]) : kNan;
    named = 0;
  }

  // the teacher's probabilities: softmax of its kept logits over tau
  const bool has_k = t < p.k;
  float u = -INFINITY;
  if (t < ((p.k + 3) & ~3)) {
    int32_t my = -1;
    if (has_k) {
      my = p.ids[row * p.k + t];
      float zm = 0.0f;
      if (my >= 0 && my < V) {
        u = to_f32<T>(reinterpret_cast<const T*>(p.u)[row * p.k + t]) / p.tau;
        zm = to_f32<T>(z[my]);
      }
      keep_u[t] = u;
      keep_z[t] = zm;
    }
    id[t] = my;
  }
  __syncthreads();
  // an entry that is listed twice is written once, by its first place
  if (has_k) {
    const int32_t my = id[t];
    bool first = my >= 0 && my < V, again = false;
    if (first) {
      for (int j = 0; j < p.k; j += 4) {
        const int4 o = *reinterpret_cast<const int4*>(id + j);
        const int same = (o.x == my) | (o.y == my) << 1 | (o.z == my) << 2 | (o.w == my) << 3;
        if (j <= t) {
          const int before = t - j < 4 ? same & ((1 << (t - j)) - 1) : same;
          first &= before == 0;
        }
        again |= (t - j >= 0 && t - j < 4 ? same & ~(1 << (t - j)) : same) != 0;
      }
      if (HARD && my == y) named = 1;
    }
    keep_flags[t] = (uint8_t)(first | again << 1);
  }
  float m = edge ? ze : -INFINITY;
  each([&](int r, int i) __attribute__((always_inline)) {
    float v[N];
    Vec<T>::get(vec(r, i), v);
#pragma unroll
    for (int k = 0; k < N; ++k) m = MaxOp{}(m, v[k]);
  });
  float top[2] = {m, u};
  block_reduce<WAVES>(top, sh_max, MaxOp{});
  m = top[0];
  const float mu = top[1];
  const bool some = mu != -INFINITY && p.alpha > 0.0f;  // the teacher kept something of this row, and it counts
  const float ctau = kLog2e / p.tau;
  // sums: exp(z / tau), exp(z), the teacher's exp(u), and sum of those times
  // (u - mu) - (z - m) / tau, of which the divergence is made
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (edge) {
    sum[0] = exp_scaled(ze, m, ctau);
    if constexpr (HARD) sum[1] = exp_scaled(ze, m, kLog2e);
  }
  each([&](int r, int i) __attribute__((always_inline)) {
    float v[N];
    Vec<T>::get(vec(r, i), v);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      sum[0] += exp_scaled(v[k], m, ctau);
      if constexpr (HARD) sum[1] += exp_scaled(v[k], m, kLog2e);
    }
  });
  if (has_k) {
    const int32_t my = id[t];
    const float ku = keep_u[t];
    float eu = 0.0f;
    if (my >= 0 && some) {
      eu = __builtin_amdgcn_exp2f((ku - mu) * kLog2e);
      if (eu > 0.0f || eu != eu) sum[3] = eu * ((ku - mu) - (keep_z[t] - m) / p.tau);
    }
    sum[2] = eu;
    pr[t] = eu;
    if (my >= V) sum[3] = kNan;  // an id outside the vocabulary makes the row NaN, also where no teacher's term is taken
  }
  block_reduce<WAVES>(sum, sh_sum, SumOp{});
  const float st = sum[0], s1 = sum[1], su = sum[2];
  // sum p (log p - log q) = sum p ((u - mu) - (z - m) / tau) - log su + log st
  const float kl = some ? sum[3] / su + (__builtin_amdgcn_logf(st) - __builtin_amdgcn_logf(su)) * kLn2 : sum[3];
  float loss = p.alpha > 0.0f ? p.alpha * p.tau * p.tau * kl : kl;  // (0 or NaN)
  if constexpr (HARD) loss += (1.0f - p.alpha) * (m + __builtin_amdgcn_logf(s1) * kLn2 - keep_target);
  if (t == 0 && p.loss) p.loss[row] = loss;
  if (!dz) return;

  // dz = w (alpha tau (q_tau - p) + (1 - alpha)(q_1 - [target])): the softmax
  // parts everywhere, then the few entries with a teacher's or target's part
  const float bad = loss != loss ? kNan : 0.0f;
  const float at = some ? p.alpha * p.tau * w : 0.0f, gt = at / st + bad;
  const float a1 = (1.0f - p.alpha) * w, g1 = HARD ? a1 / s1 : 0.0f;
  auto grad = [&](float v) __attribute__((always_inline)) {
    float g = gt * exp_scaled(v, m, ctau);
    if constexpr (HARD) g = fmaf(g1, exp_scaled(v, m, kLog2e), g);
    return g;
  };
  each([&](int r, int i) __attribute__((always_inline)) {
    float v[N];
    Vec<T>::get(vec(r, i), v);
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = grad(v[k]);
    if (vec_out) {
      stream_store(reinterpret_cast<uint4*>(dz + head) + i, Vec<T>::put(v));
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) dz[head + i * N + k] = from_f32<T>(v[k]);
    }
  });
  if (edge) dz[ei] = from_f32<T>(grad(keep_edge[t]));
  // the row is written before its few other entries are: by waves of their own, so the
  // stores themselves are waited for
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (has_k && (keep_flags[t] & 1)) {
    const int32_t my = id[t];
    float mass = some ? pr[t] / su : 0.0f;
    if (keep_flags[t] & 2)
      for (int j = t + 1; j < p.k; ++j)
        if (id[j] == my) mass += some ? pr[j] / su : 0.0f;
    float g = grad(keep_z[t]) - at * mass;
    if (HARD && my == y) g -= a1;
    dz[my] = from_f32<T>(g);
  }
  if constexpr (HARD) {
    if (t == 0 && (uint64_t)y < (uint64_t)V && !named) dz[y] = from_f32<T>(grad(keep_target) - a1);
  }
}

// Few rows: 1024 threads each, so that one row takes less time; many: 512, of which
// three rows fit a CU at R = 13 and cover each other's loads and stores.  Up to 106496
// bf16 or 53248 fp32 entries a row stays in registers; beyond (R = 0) it is read for each
// of the three passes.  Loss and gradient of 16384 bf16 rows: 106496 entries 1335 us (floor
// 1326), 128256 2376 (1597), 151936 3360 (1891); of 8192 fp32 rows: 53248 650 (663), 60001
// 1121 (747); of 37 bf16 rows: 106496 19, 128256 24.  Short rows leave threads idle: 16384
// of 1000 entries 121 us (12).
template <class T, bool HARD>
void launch_distill_r(const DistillArgs& a, hipStream_t s) {
  const bool few = a.T < 512;
  const int64_t nv = a.V / Vec<T>::N, r = (nv + (few ? 1023 : 511)) / (few ? 1024 : 512);
  const uint32_t grid = (uint32_t)a.T;
  if (few) {
    if (r <= 4) distill_kernel<T, 4, HARD, 1024><<<grid, 1024, 0, s>>>(a);
    else if (r <= 8) distill_kernel<T, 8, HARD, 1024><<<grid, 1024, 0, s>>>(a);
    else if (r <= 13) distill_kernel<T, 13, HARD, 1024><<<grid, 1024, 0, s>>>(a);
    else distill_kernel<T, 0, HARD, 1024><<<grid, 1024, 0, s>>>(a);
  } else {
    if (r <= 4) distill_kernel<T, 4, HARD, 512><<<grid, 512, 0, s>>>(a);
    else if (r <= 8) distill_kernel<T, 8, HARD, 512><<<grid, 512, 0, s>>>(a);
    else if (r <= 13) distill_kernel<T, 13, HARD, 512><<<grid, 512, 0, s>>>(a);
    else if (r <= 26) distill_kernel<T, 26, HARD, 512><<<grid, 512, 0, s>>>(a);
    else distill_kernel<T, 0, HARD, 512><<<grid, 512, 0, s>>>(a);
  }
}

}  // namespace

int distill_max_k() { return kDistillMaxK; }

hipError_t launch_distill(const DistillParams& d, hipStream_t s) {
  DistillArgs a = {};
  a.z = d.z;
  a.dz = d.dz;
  a.ldz = d.ldz;
  a.ldd = d.ldd;
  a.ids = d.ids;
  a.u = d.u;
  a.y = d.y;
  a.w = d.w;
  a.loss = d.loss;
  a.T = d.T;
  a.V = d.V;
  a.ignore = d.ignore;
  a.k = d.k;
  a.tau = d.tau;
  a.alpha = d.alpha;
  const bool hard = d.alpha != 1.0f;
  if (d.dtype == TJ2_BF16) {
    if (hard) launch_distill_r<uint16_t, true>(a, s);
    else launch_distill_r<uint16_t, false>(a, s);
  } else {
    if (hard) launch_distill_r<float, true>(a, s);
    else launch_distill_r<float, false>(a, s);
  }
  return hipGetLastError();
}

}  // namespace tj2
