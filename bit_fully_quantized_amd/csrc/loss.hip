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
// logits are read once and the gradient is written once.
#include <math.h>

#include <algorithm>

#include "tj2_tile.h"

namespace tj2 {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// 2^((v - m) c): the difference first, which is exact for logits near m and 0 at it
// however large they are (a fused v c - m c is off by a half step of m c)
__device__ __forceinline__ float exp_scaled(float v, float m, float c) { return __builtin_amdgcn_exp2f((v - m) * c); }

// (m, s) of sum exp: s exp(m) in total; m = -inf stands for nothing
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float M = fmaxf(m, m2);
  const float b = M == -INFINITY ? 0.0f : M;
  s = s * __builtin_amdgcn_exp2f((m - b) * kLog2e) + s2 * __builtin_amdgcn_exp2f((m2 - b) * kLog2e);
  m = M;
}

struct CeArgs {
  TileOp P, Q;                 // P: W [V, K] (or a piece of it), Q: X [T, K]
  const int64_t* y;
  int64_t V, ignore;
  uint32_t tiles_p, tiles_q;
  int32_t nch;
  float2* part;                // forward: [parts][T]
  float* zt;                   // forward: [T], the target's logit
  // backward
  const float* lse;
  const float* c;              // [T] weights over their largest magnitude, 0 where ignored
  int64_t v0;                  // first vocabulary entry of the piece
  uint16_t* d;                 // dz of the piece [T][ldd]
  uint16_t* dt;                // and transposed [piece rows][ldt]
  int64_t ldd, ldt;
};

template <class T>
__global__ __launch_bounds__(T::NT, 1) void ce_fwd_kernel(CeArgs p) {
  __shared__ __attribute__((aligned(128))) typename T::Smem sm;
  uint32_t tp, tq;
  tile_of(blockIdx.x, gridDim.x, p.tiles_q, p.tiles_p, tq, tp);
  const int64_t p0 = (int64_t)tp * T::BM, q0 = (int64_t)tq * T::BN;
  typename T::Acc acc = {};
  T::run(p.P, p0, p.Q, q0, 0, p.nch, sm, acc);

  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
  const int wm = w / T::kWN;
  const int64_t pw = p0 + wm * T::kTM * 16, qw = q0 + (w % T::kWN) * T::kTN * 16;
  const int there = (int)min(p.P.rows - pw, (int64_t)(16 * T::kTM));  // vocabulary entries of this wave
  const int left = there - g * 4 * T::PB;
#pragma unroll
  for (int tn = 0; tn < T::kTN; ++tn) {
    const int64_t t = qw + T::q_row(tn, n);
    const bool in = t < p.Q.rows;
    // the target's place among the wave's entries, -1: not among them
    const int64_t yw = in ? p.y[t] - pw : -1;
    const int y = yw >= 0 && yw < there ? (int)yw - g * 4 * T::PB : -1;
    float m = -INFINITY;
#pragma unroll
    for (int tm = 0; tm < T::kTM; ++tm)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int v = T::p_row(tm, 0, r);
        if (v >= left) acc[tm][tn][r] = -INFINITY;
        else if (v == y) p.zt[t] = acc[tm][tn][r];
        m = fmaxf(m, acc[tm][tn][r]);
      }
    const float b = m == -INFINITY ? 0.0f : m;
    float s = 0.0f;
#pragma unroll
    for (int tm = 0; tm < T::kTM; ++tm)
#pragma unroll
      for (int r = 0; r < 4; ++r) s += exp_scaled(acc[tm][tn][r], b, kLog2e);
    join(m, s, __shfl_xor(m, 16), __shfl_xor(s, 16));
    join(m, s, __shfl_xor(m, 32), __shfl_xor(s, 32));
    if (g == 0 && in) p.part[((int64_t)tp * (T::NT / 64 / T::kWN) + wm) * p.Q.rows + t] = float2{m, s};
  }
}

// Token by token: the parts of its sum joined (four quarters of them at a time),
// the loss from the target's logit; a target outside the vocabulary gives NaN.
__global__ __launch_bounds__(256) void ce_join_kernel(const float2* part, int parts, const float* zt, const int64_t* y,
                                                      int64_t T, int64_t V, int64_t ignore, float* loss, float* lse) {
  __shared__ float2 sh[4][64];
  const int l = threadIdx.x & 63, q = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * 64 + l;
  float m = -INFINITY, s = 0.0f;
  if (t < T) {
    const int a = (int)((int64_t)parts * q / 4), b = (int)((int64_t)parts * (q + 1) / 4);
    const float2* at = part + (int64_t)a * T + t;
#pragma unroll 8
    for (int i = a; i < b; ++i, at += T) {
      const float2 v = *at;
      join(m, s, v.x, v.y);
    }
  }
  sh[q][l] = float2{m, s};
  __syncthreads();
  if (q || t >= T) return;
#pragma unroll
  for (int i = 1; i < 4; ++i) join(m, s, sh[i][l].x, sh[i][l].y);
  const float e = m + __builtin_amdgcn_logf(s) * kLn2;
  lse[t] = e;
  if (loss) {
    const int64_t k = y[t];
    loss[t] = k == ignore ? 0.0f : (uint64_t)k < (uint64_t)V ? e - zt[t] : __uint_as_float(0x7FC00000u);
  }
}

// c = w / max |w| (0 where the target is ignored) and that maximum: equal weights
// become 1, so that the bf16 of (softmax - 1) near a target is as exact as can be.
__global__ __launch_bounds__(1024) void ce_weights_kernel(const float* w, const int64_t* y, int64_t T, int64_t V, int64_t ignore,
                                                          float* c, float* top) {
  __shared__ float sh[16];
  float m = 0.0f;
  for (int64_t t = threadIdx.x; t < T; t += 1024)
    if (y[t] != ignore) m = fmaxf(m, fabsf(w[t]));
#pragma unroll
  for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = m;
  __syncthreads();
  m = sh[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) m = fmaxf(m, sh[i]);
  if (m == 0.0f) m = 1.0f;
  for (int64_t t = threadIdx.x; t < T; t += 1024) {
    const int64_t k = y[t];
    c[t] = k == ignore ? 0.0f : (uint64_t)k < (uint64_t)V ? w[t] / m : __uint_as_float(0x7FC00000u);
  }
  if (threadIdx.x == 0) *top = m;
}

template <class T>
__global__ __launch_bounds__(T::NT, 1) void ce_dz_kernel(CeArgs p) {
  __shared__ __attribute__((aligned(128))) typename T::Smem sm;
  uint32_t tp, tq;
  tile_of(blockIdx.x, gridDim.x, p.tiles_q, p.tiles_p, tq, tp);
  const int64_t p0 = (int64_t)tp * T::BM, q0 = (int64_t)tq * T::BN;
  typename T::Acc acc = {};
  T::run(p.P, p0, p.Q, q0, 0, p.nch, sm, acc);

  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
  const int64_t pw = p0 + (w / T::kWN) * T::kTM * 16 + g * 4 * T::PB, qw = q0 + (w % T::kWN) * T::kTN * 16 + n * T::kTN;
  const int64_t left = p.P.rows - pw;
  float c[T::kTN], b[T::kTN];
  int64_t y[T::kTN];
#pragma unroll
  for (int tn = 0; tn < T::kTN; ++tn) {
    const bool in = qw + tn < p.Q.rows;
    c[tn] = in ? p.c[qw + tn] : 0.0f;
    b[tn] = in ? p.lse[qw + tn] : 0.0f;
    y[tn] = in ? p.y[qw + tn] - p.v0 - pw : -1;
  }
#pragma unroll
  for (int tm = 0; tm < T::kTM; ++tm)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int v = T::p_row(tm, 0, r);
#pragma unroll
      for (int tn = 0; tn < T::kTN; ++tn) {
        float e = exp_scaled(acc[tm][tn][r], b[tn], kLog2e);
        e = c[tn] * (v == y[tn] ? e - 1.0f : e);
        // an ignored token has no gradient, whatever its logits are
        acc[tm][tn][r] = v < left && c[tn] != 0.0f ? e : 0.0f;
      }
      // four neighbouring tokens of one vocabulary entry
      if (pw + v < p.ldd && qw < p.ldt) {
        static_assert(T::kTN == 4, "four tokens a lane");
        *reinterpret_cast<uint2*>(p.dt + (pw + v) * p.ldt + qw) =
            uint2{bf16_pair(acc[tm][0][r], acc[tm][1][r]), bf16_pair(acc[tm][2][r], acc[tm][3][r])};
      }
    }
  // 4 PB neighbouring vocabulary entries of one token
#pragma unroll
  for (int tn = 0; tn < T::kTN; ++tn) {
    if (qw + tn >= p.Q.rows) continue;
#pragma unroll
    for (int tb = 0; tb < T::kTM / T::PB; ++tb) {
      const int64_t j = pw + tb * 16 * T::PB;
      if (j >= p.ldd) continue;  // ldd is a multiple of 64
      uint16_t* o = p.d + (qw + tn) * p.ldd + j;
#pragma unroll
      for (int k = 0; k < T::PB; k += 2) {
        const float4_t a = acc[tb * T::PB + k][tn], e = acc[tb * T::PB + k + 1][tn];
        *reinterpret_cast<uint4*>(o + 4 * k) =
            uint4{bf16_pair(a.x, a.y), bf16_pair(a.z, a.w), bf16_pair(e.x, e.y), bf16_pair(e.z, e.w)};
      }
    }
  }
}

// out[c][r] = in[r][c] for rows r < rows (zero up to ld) of a bf16 matrix with
// `cols` (a multiple of 16) columns: 64 x 64 through LDS.
__global__ __launch_bounds__(256) void transpose_kernel(const uint16_t* in, int64_t rows, int64_t cols, int64_t ldi, uint16_t* out,
                                                        int64_t ld) {
  __shared__ uint16_t tile[64][66];
  const int64_t r0 = (int64_t)blockIdx.x * 64, c0 = (int64_t)blockIdx.y * 64;
  const int t = threadIdx.x;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = i * 32 + (t >> 3), c = (t & 7) * 8;
    uint4 v = {0u, 0u, 0u, 0u};
    if (r0 + r < rows && c0 + c < cols) v = *reinterpret_cast<const uint4*>(in + (r0 + r) * ldi + c0 + c);
    uint32_t* s = reinterpret_cast<uint32_t*>(&tile[r][c]);
    s[0] = v.x; s[1] = v.y; s[2] = v.z; s[3] = v.w;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = i * 32 + (t >> 3), r = (t & 7) * 8;
    if (c0 + c >= cols) continue;
    uint32_t v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = tile[r + 2 * k][c] | ((uint32_t)tile[r + 2 * k + 1][c] << 16);
    *reinterpret_cast<uint4*>(out + (c0 + c) * ld + r0 + r) = uint4{v[0], v[1], v[2], v[3]};
  }
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

template <class T>
__global__ __launch_bounds__(T::NT, 1) void ce_product_kernel(ProductArgs p) {
  __shared__ __attribute__((aligned(128))) typename T::Smem sm;
  uint32_t tp, tq;
  const uint32_t tiles = p.tiles_p * p.tiles_q, z = blockIdx.x / tiles;
  tile_of(blockIdx.x - z * tiles, tiles, p.tiles_q, p.tiles_p, tq, tp);
  const int64_t p0 = (int64_t)tp * T::BM, q0 = (int64_t)tq * T::BN;
  const int c0 = (int)((int64_t)p.nch * z / p.splits), c1 = (int)((int64_t)p.nch * (z + 1) / p.splits);
  typename T::Acc acc = {};
  T::run(p.P, p0, p.Q, q0, c0, c1, sm, acc);

  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
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
}

// out = scale * (sum of `parts` fp32 slices), in order; 4 a thread (n a multiple of 16).
__global__ __launch_bounds__(256) void ce_sum_kernel(const float* sum, int parts, int64_t n, const float* scale, void* out, int bf16) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  float4_t v = *reinterpret_cast<const float4_t*>(sum + i);
  for (int z = 1; z < parts; ++z) v += *reinterpret_cast<const float4_t*>(sum + (size_t)z * (size_t)n + i);
  const float s = *scale;
  v *= s;
  if (bf16) *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(out) + i) = uint2{bf16_pair(v.x, v.y), bf16_pair(v.z, v.w)};
  else *reinterpret_cast<float4_t*>(reinterpret_cast<float*>(out) + i) = v;
}

// sum slice 0 (kept over the pieces) += the piece's slices, in order
__global__ __launch_bounds__(256) void ce_fold_kernel(float* kept, const float* part, int parts, int64_t n, int first) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  float4_t v = *reinterpret_cast<const float4_t*>(part + i);
  for (int z = 1; z < parts; ++z) v += *reinterpret_cast<const float4_t*>(part + (size_t)z * (size_t)n + i);
  if (!first) v += *reinterpret_cast<const float4_t*>(kept + i);
  *reinterpret_cast<float4_t*>(kept + i) = v;
}

using TileCe = Tile<EL_BF16, 2, 4, 8, 4>;

TileOp bf16_operand(const void* p, int64_t rows, int64_t cols, int64_t ld) {
  TileOp o = {};
  o.p = reinterpret_cast<const uint8_t*>(p);
  o.rows = rows;
  o.ld = ld * 2;
  o.kb = (int32_t)(cols * 2);
  return o;
}

int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// Vocabulary entries of a piece of the backward (a multiple of 256): dz of the
// piece, and its transpose, stay near the 256 MB of the memory-side cache.
int64_t ce_piece(int64_t T, int64_t V) {
  const int64_t most = ((int64_t)64 << 20) / std::max<int64_t>(up(T, 64), 1) / 256 * 256;
  return std::min(up(V, 256), std::max<int64_t>(most, 1024));
}

int ce_splits(int64_t p_rows, int64_t q_rows, int64_t k) {
  const int64_t tiles = up(p_rows, 256) / 256 * (up(q_rows, 256) / 256), nch = up(k, 64) / 64;
  return (int)std::max<int64_t>(1, std::min<int64_t>(256 / tiles, nch / 8));
}

struct CeBwdSpace {
  size_t c, top, xt, wt, d, dt, dx, part, bytes;
  int64_t piece, ldd, ldt;
  int sx, sw;
};
CeBwdSpace ce_bwd_space(int64_t T, int64_t K, int64_t V) {
  CeBwdSpace s;
  s.piece = ce_piece(T, V);
  s.ldd = s.piece;
  s.ldt = up(T, 64);
  s.sx = ce_splits(K, T, s.piece);
  s.sw = ce_splits(K, s.piece, T);
  size_t at = 0;
  auto take = [&](size_t n) { const size_t a = at; at += up256(n); return a; };
  s.c = take((size_t)T * 4);
  s.top = take(4);
  s.xt = take((size_t)(K * s.ldt * 2));
  s.wt = take((size_t)(K * s.ldd * 2));
  s.d = take((size_t)(T * s.ldd * 2));
  s.dt = take((size_t)(s.ldd * s.ldt * 2));
  s.dx = take((size_t)(T * K * 4));
  s.part = take(std::max(s.sx > 1 ? (size_t)s.sx * (size_t)(T * K * 4) : 0, s.sw > 1 ? (size_t)s.sw * (size_t)(s.piece * K * 4) : 0));
  s.bytes = at;
  return s;
}

}  // namespace

size_t ce_fwd_workspace_bytes(int64_t T, int64_t V) {
  const int64_t parts = up(V, TileCe::BM) / TileCe::BM * 2;
  return up256((size_t)parts * (size_t)T * 8) + up256((size_t)T * 4);
}

hipError_t launch_ce_fwd(const CeParams& c, void* ws, hipStream_t s) {
  CeArgs a = {};
  a.P = bf16_operand(c.W, c.V, c.K, c.ldw);
  a.Q = bf16_operand(c.X, c.T, c.K, c.ldx);
  a.y = c.y;
  a.V = c.V;
  a.ignore = c.ignore;
  a.tiles_p = (uint32_t)(up(c.V, TileCe::BM) / TileCe::BM);
  a.tiles_q = (uint32_t)(up(c.T, TileCe::BN) / TileCe::BN);
  a.nch = (int32_t)(up(c.K, 64) / 64);
  const int parts = (int)a.tiles_p * 2;
  a.part = reinterpret_cast<float2*>(ws);
  a.zt = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ws) + up256((size_t)parts * (size_t)c.T * 8));
  ce_fwd_kernel<TileCe><<<a.tiles_p * a.tiles_q, TileCe::NT, 0, s>>>(a);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  ce_join_kernel<<<(uint32_t)((c.T + 63) / 64), 256, 0, s>>>(a.part, parts, a.zt, c.y, c.T, c.V, c.ignore, c.loss, c.lse);
  return hipGetLastError();
}

size_t ce_bwd_workspace_bytes(int64_t T, int64_t K, int64_t V) { return ce_bwd_space(T, K, V).bytes; }

hipError_t launch_ce_bwd(const CeParams& c, void* ws, hipStream_t s) {
  const CeBwdSpace sp = ce_bwd_space(c.T, c.K, c.V);
  uint8_t* w = reinterpret_cast<uint8_t*>(ws);
  float* top = reinterpret_cast<float*>(w + sp.top);
  uint16_t *xt = reinterpret_cast<uint16_t*>(w + sp.xt), *wt = reinterpret_cast<uint16_t*>(w + sp.wt);
  uint16_t *d = reinterpret_cast<uint16_t*>(w + sp.d), *dt = reinterpret_cast<uint16_t*>(w + sp.dt);
  float *dx = reinterpret_cast<float*>(w + sp.dx), *part = reinterpret_cast<float*>(w + sp.part);
#define TJ2_STEP()                                                    \
  do {                                                                \
    if (hipError_t e_ = hipGetLastError(); e_ != hipSuccess) return e_; \
  } while (0)
  ce_weights_kernel<<<1, 1024, 0, s>>>(c.dloss, c.y, c.T, c.V, c.ignore, reinterpret_cast<float*>(w + sp.c), top);
  TJ2_STEP();
  const uint32_t kt = (uint32_t)((c.K + 63) / 64);
  transpose_kernel<<<dim3((uint32_t)(sp.ldt / 64), kt), 256, 0, s>>>(reinterpret_cast<const uint16_t*>(c.X), c.T, c.K, c.ldx, xt, sp.ldt);
  TJ2_STEP();
  const bool one = sp.piece >= c.V;
  for (int64_t v0 = 0; v0 < c.V; v0 += sp.piece) {
    const int64_t vn = std::min(sp.piece, c.V - v0), ldd = up(vn, 64);
    const uint16_t* W = reinterpret_cast<const uint16_t*>(c.W) + v0 * c.ldw;
    transpose_kernel<<<dim3((uint32_t)(ldd / 64), kt), 256, 0, s>>>(W, vn, c.K, c.ldw, wt, ldd);
    TJ2_STEP();
    CeArgs a = {};
    a.P = bf16_operand(W, vn, c.K, c.ldw);
    a.Q = bf16_operand(c.X, c.T, c.K, c.ldx);
    a.y = c.y;
    a.tiles_p = (uint32_t)(up(vn, TileCe::BM) / TileCe::BM);
    a.tiles_q = (uint32_t)(up(c.T, TileCe::BN) / TileCe::BN);
    a.nch = (int32_t)(up(c.K, 64) / 64);
    a.lse = c.lse;
    a.c = reinterpret_cast<float*>(w + sp.c);
    a.v0 = v0;
    a.d = d;
    a.dt = dt;
    a.ldd = ldd;
    a.ldt = sp.ldt;
    ce_dz_kernel<TileCe><<<a.tiles_p * a.tiles_q, TileCe::NT, 0, s>>>(a);
    TJ2_STEP();
    if (c.dX) {
      ProductArgs x = {};
      x.P = bf16_operand(wt, c.K, ldd, ldd);
      x.Q = bf16_operand(d, c.T, ldd, ldd);
      x.tiles_p = (uint32_t)(up(c.K, TileCe::BM) / TileCe::BM);
      x.tiles_q = a.tiles_q;
      x.nch = (int32_t)(ldd / 64);
      x.splits = std::min(sp.sx, std::max(1, x.nch));
      x.scale = top;
      x.bf16 = c.dx_dtype == TJ2_BF16;
      x.ldo = c.K;
      x.first = x.splits > 1 || v0 == 0;
      if (x.splits > 1) x.sum = part;
      else if (one) x.out = c.dX;
      else x.sum = dx;
      ce_product_kernel<TileCe><<<x.tiles_p * x.tiles_q * (uint32_t)x.splits, TileCe::NT, 0, s>>>(x);
      TJ2_STEP();
      const int64_t n = c.T * c.K;
      const uint32_t grid = (uint32_t)((n / 4 + 255) / 256);
      if (x.splits > 1 && one) {
        ce_sum_kernel<<<grid, 256, 0, s>>>(part, x.splits, n, top, c.dX, x.bf16);
      } else {
        if (x.splits > 1) ce_fold_kernel<<<grid, 256, 0, s>>>(dx, part, x.splits, n, v0 == 0);
        if (!one && v0 + vn == c.V) ce_sum_kernel<<<grid, 256, 0, s>>>(dx, 1, n, top, c.dX, x.bf16);
      }
      TJ2_STEP();
    }
    if (c.dW) {
      ProductArgs x = {};
      x.P = bf16_operand(xt, c.K, sp.ldt, sp.ldt);
      x.Q = bf16_operand(dt, vn, sp.ldt, sp.ldt);
      x.tiles_p = (uint32_t)(up(c.K, TileCe::BM) / TileCe::BM);
      x.tiles_q = (uint32_t)(up(vn, TileCe::BN) / TileCe::BN);
      x.nch = (int32_t)(sp.ldt / 64);
      x.splits = std::min(sp.sw, std::max(1, x.nch));
      x.scale = top;
      x.bf16 = c.dw_dtype == TJ2_BF16;
      x.ldo = c.K;
      x.first = 1;
      uint8_t* out = reinterpret_cast<uint8_t*>(c.dW) + (size_t)(v0 * c.K) * (x.bf16 ? 2 : 4);
      if (x.splits > 1) x.sum = part;
      else x.out = out;
      ce_product_kernel<TileCe><<<x.tiles_p * x.tiles_q * (uint32_t)x.splits, TileCe::NT, 0, s>>>(x);
      TJ2_STEP();
      const int64_t n = vn * c.K;
      if (x.splits > 1) ce_sum_kernel<<<(uint32_t)((n / 4 + 255) / 256), 256, 0, s>>>(part, x.splits, n, top, out, x.bf16);
      TJ2_STEP();
    }
  }
#undef TJ2_STEP
  return hipSuccess;
}

// ---- distillation -------------------------------------------------------------------
namespace {

constexpr int kDistillThreads = 512;
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

template <class F>
__device__ __forceinline__ float block_reduce(float v, float* sh, F f) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v = f(v, __shfl_xor(v, o));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  v = sh[0];
#pragma unroll
  for (int i = 1; i < kDistillThreads / 64; ++i) v = f(v, sh[i]);
  return v;
}

struct MaxOp {
  // NaN is kept: a row with one has a NaN loss
  __device__ __forceinline__ float operator()(float a, float b) const { return a > b || a != a ? a : b; }
};
struct SumOp {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};

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
// temperature 1).
template <class T, int R, bool HARD>
__global__ __launch_bounds__(kDistillThreads) void distill_kernel(DistillArgs p) {
  constexpr int N = Vec<T>::N;
  constexpr int RR = R > 0 ? R : 1;
  __shared__ float sh[kDistillThreads / 64];
  __shared__ int32_t id[kDistillMaxK];
  __shared__ float pr[kDistillMaxK], zi[kDistillMaxK];
  const int t = threadIdx.x;
  const int64_t row = blockIdx.x;
  const T* z = reinterpret_cast<const T*>(p.z) + row * p.ldz;
  T* dz = p.dz ? reinterpret_cast<T*>(p.dz) + row * p.ldd : nullptr;
  const int64_t V = p.V;
  const int64_t y = p.y ? p.y[row] : 0;
  const bool on = !p.y || y != p.ignore;
  const float w = p.w ? p.w[row] : 1.0f;

  // aligned middle [head, head + N * nv)
  const int head = (int)min((int64_t)(((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) / sizeof(T)), V);
  const int64_t nv = (V - head) / N;
  const int tail = (int)(V - head - nv * N);
  const uint4* zv = reinterpret_cast<const uint4*>(z + head);
  const bool edge = t < head + tail;
  const int64_t ei = t < head ? t : V - tail + (t - head);
  // the gradient's vectors: the same places, if its row is aligned alike
  const bool vec_out = dz && (((reinterpret_cast<uintptr_t>(dz) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0);

  if (!on) {  // no loss and no gradient
    if (t == 0 && p.loss) p.loss[row] = 0.0f;
    if (dz) {
      if (vec_out)
        for (int64_t i = t; i < nv; i += kDistillThreads) reinterpret_cast<uint4*>(dz + head)[i] = uint4{0u, 0u, 0u, 0u};
      else
        for (int64_t i = t; i < nv * N; i += kDistillThreads) dz[head + i] = from_f32<T>(0.0f);
      if (edge) dz[ei] = from_f32<T>(0.0f);
    }
    return;
  }

  uint4 q[RR];
  auto vec = [&](int r, int64_t i) __attribute__((always_inline)) -> uint4 {
    if constexpr (R > 0) return q[r];
    return zv[i];
  };
  // f(r, i) for each of this thread's vectors i
  auto each = [&](auto&& f) __attribute__((always_inline)) {
    if constexpr (R > 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int64_t i = t + r * kDistillThreads;
        if (i < nv) f(r, i);
      }
    } else {
      for (int64_t i = t; i < nv; i += kDistillThreads) f(0, i);
    }
  };
  if constexpr (R > 0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t i = t + r * kDistillThreads;
      if (i < nv) q[r] = zv[i];
    }
  }
  const float ze = edge ? to_f32<T>(z[ei]) : 0.0f;
  // read before anything is written: dz may be z
  float zy = 0.0f;
  if constexpr (HARD) zy = (uint64_t)y < (uint64_t)V ? to_f32<T>(z[y]) : __uint_as_float(0x7FC00000u);

  // the teacher's probabilities: softmax of its kept logits over tau
  const bool has_k = t < p.k;
  int32_t my = -1;
  float u = -INFINITY;
  if (has_k) {
    my = p.ids[row * p.k + t];
    if (my >= 0 && my < V) u = to_f32<T>(reinterpret_cast<const T*>(p.u)[row * p.k + t]) / p.tau;
    id[t] = my;
    zi[t] = my >= 0 && my < V ? to_f32<T>(z[my]) : 0.0f;
  }
  const bool kept = has_k && my >= 0;
  float m = edge ? ze : -INFINITY;
  each([&](int r, int64_t i) __attribute__((always_inline)) {
    float v[N];
    Vec<T>::get(vec(r, i), v);
#pragma unroll
    for (int k = 0; k < N; ++k) m = MaxOp{}(m, v[k]);
  });
  m = block_reduce(m, sh, MaxOp{});
  const float mu = block_reduce(u, sh, MaxOp{});
  const bool some = mu != -INFINITY;  // the teacher kept something of this row
  const float ctau = kLog2e / p.tau;
  float st = edge ? exp_scaled(ze, m, ctau) : 0.0f;
  float s1 = HARD && edge ? exp_scaled(ze, m, kLog2e) : 0.0f;
  each([&](int r, int64_t i) __attribute__((always_inline)) {
    float v[N];
    Vec<T>::get(vec(r, i), v);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      st += exp_scaled(v[k], m, ctau);
      if constexpr (HARD) s1 += exp_scaled(v[k], m, kLog2e);
    }
  });
  st = block_reduce(st, sh, SumOp{});
  if constexpr (HARD) s1 = block_reduce(s1, sh, SumOp{});
  const float eu = kept && some ? __builtin_amdgcn_exp2f((u - mu) * kLog2e) : 0.0f;
  const float su = block_reduce(eu, sh, SumOp{});
  const float pt = some ? eu / su : 0.0f;
  const float lt = __builtin_amdgcn_logf(st) * kLn2;  // lse / tau - m / tau
  // an id outside the vocabulary makes the row NaN
  const float wrong = kept && my >= V ? __uint_as_float(0x7FC00000u) : 0.0f;
  float kl = wrong;
  if (pt > 0.0f || pt != pt) kl += pt * ((u - mu) - __builtin_amdgcn_logf(su) * kLn2 - ((zi[t] - m) / p.tau - lt));
  kl = block_reduce(kl, sh, SumOp{});
  float loss = p.alpha > 0.0f ? p.alpha * p.tau * p.tau * kl : 0.0f;
  if constexpr (HARD) loss += (1.0f - p.alpha) * (m + __builtin_amdgcn_logf(s1) * kLn2 - zy);
  if (t == 0 && p.loss) p.loss[row] = loss;
  if (!dz) return;

  // dz = w (alpha tau (q_tau - p) + (1 - alpha)(q_1 - [target])): the softmax
  // parts everywhere, then the few entries with a teacher's or target's part
  const float bad = loss != loss ? __uint_as_float(0x7FC00000u) : 0.0f;
  const float at = some ? p.alpha * p.tau * w : 0.0f, gt = at / st + bad;
  const float a1 = (1.0f - p.alpha) * w, g1 = HARD ? a1 / s1 : 0.0f;
  auto grad = [&](float v) __attribute__((always_inline)) {
    float g = gt * exp_scaled(v, m, ctau);
    if constexpr (HARD) g = fmaf(g1, exp_scaled(v, m, kLog2e), g);
    return g;
  };
  if (has_k) pr[t] = pt;
  each([&](int r, int64_t i) __attribute__((always_inline)) {
    float v[N];
    Vec<T>::get(vec(r, i), v);
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = grad(v[k]);
    if (vec_out) {
      reinterpret_cast<uint4*>(dz + head)[i] = Vec<T>::put(v);
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) dz[head + i * N + k] = from_f32<T>(v[k]);
    }
  });
  if (edge) dz[ei] = from_f32<T>(grad(ze));
  __syncthreads();  // the row is written, pr and id are there
  // an entry that is listed twice is written once, by its first place
  if (has_k && my >= 0 && my < V) {
    float sum = 0.0f;
    bool first = true;
    for (int j = 0; j < p.k; ++j) {
      if (id[j] != my) continue;
      if (j < t) first = false;
      sum += pr[j];
    }
    if (first) {
      float g = grad(zi[t]) - at * sum;
      if (HARD && my == y) g -= a1;
      dz[my] = from_f32<T>(g);
    }
  }
  if constexpr (HARD) {
    if (t == 0 && (uint64_t)y < (uint64_t)V) {
      bool listed = false;
      for (int j = 0; j < p.k; ++j) listed |= id[j] == y;
      if (!listed) dz[y] = from_f32<T>(grad(zy) - a1);
    }
  }
}

template <class T, bool HARD>
void launch_distill_r(const DistillArgs& a, hipStream_t s) {
  const int64_t nv = a.V / Vec<T>::N, r = (nv + kDistillThreads - 1) / kDistillThreads;
  const uint32_t grid = (uint32_t)a.T;
  if (r <= 4) distill_kernel<T, 4, HARD><<<grid, kDistillThreads, 0, s>>>(a);
  else if (r <= 8) distill_kernel<T, 8, HARD><<<grid, kDistillThreads, 0, s>>>(a);
  else if (r <= 13) distill_kernel<T, 13, HARD><<<grid, kDistillThreads, 0, s>>>(a);
  else if (r <= 20) distill_kernel<T, 20, HARD><<<grid, kDistillThreads, 0, s>>>(a);
  else distill_kernel<T, 0, HARD><<<grid, kDistillThreads, 0, s>>>(a);
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
