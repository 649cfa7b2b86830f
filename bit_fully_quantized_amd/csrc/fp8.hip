// FP8 linear layers for gfx950: E4M3 elements under one fp32 scale per 128 elements of a
// row (activations and gradients) or per 128 x 128 (weights), quantisers, values and the
// product
//
//   C[i, j] = sum over chunks c of 128  sA[i, c] sB[j, c] (sum_k qA[i, k] qB[j, k]).
//
// gfx950's 8-bit instruction takes 128 elements of the reduction at once, a chunk, so its
// result is what the two scales multiply; they are arbitrary fp32 numbers, which the
// instruction's own power-of-two scales could not hold.  Results in fp32 take exact
// products of decoded codes instead (tj2_tile.h): the instruction's own sums are off by
// 1.4e-5.
#include <algorithm>

#include "tj2_fp8.h"
#include "tj2_skinny.h"

namespace tj2 {
namespace {

// ---- quantisers ------------------------------------------------------------------
// scale = max|x| / 448 and its reciprocal in fp32, codes of x / scale rounded to the nearest
// even by the hardware's conversion.  All are bound by memory: each element is read once
// and stays in registers (or, turned, in LDS) between its group's maximum and its code.
// 16384 x 4096, us (TB/s of what is read and written; a copy reaches 5.3): along the rows
// bf16 35.0 (5.8), fp32 57.9 (5.8), per 128 x 128 bf16 35.3 (5.7), fp32 58.9 (5.7), along the
// columns bf16 33.7 (6.0), fp32 67.2 (5.0), from codes 29.6 (4.7).
// Where an operand's groups go: row r's chunk of 128 elements c has its codes at at(r, c)
// and its scale at scale[r srs + c scs].  Row-major, or (what only the backward's own
// products read) blocked as TileOp says, the scales of a chunk then next to each other.
struct Fp8Out {
  uint8_t* codes;
  float* scale;
  int64_t ld, bs, cs, srs, scs;
  __device__ __forceinline__ int64_t at(int64_t row, int64_t c) const { return (row >> 7) * bs + (row & 127) * ld + c * cs; }
};
Fp8Out fp8_out(const QView& q, bool blocked) {
  if (blocked) return Fp8Out{q.codes, q.s128, 128, q.nb * 16384, 16384, 1, (q.rows + 127) / 128 * 128};
  return Fp8Out{q.codes, q.s128, q.nb * 128, q.nb * 128 * 128, 128, q.nb, 1};
}

struct Fp8RowArgs {
  const void* x;
  Fp8Out out;
  int64_t rows;
  int32_t cols, nb;
};
// Groups along the rows: 8 neighbouring elements a thread, 16 lanes a group.
template <class T>
__device__ __forceinline__ void fp8_row(const Fp8RowArgs& p, uint32_t block) {
  const uint32_t per = (uint32_t)p.nb * 16, id = block * 256 + threadIdx.x;
  const uint32_t row = id / per;
  if (row >= p.rows) return;
  const int32_t c = (int32_t)(id - row * per) * 8;
  float v[8];
  if (c < p.cols) {
    load8(reinterpret_cast<const T*>(p.x) + (int64_t)row * p.cols + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  }
  const Fp8Scale s = fp8_scale(max16_lanes(top_bits8(v)));
  *reinterpret_cast<uint2*>(p.out.codes + p.out.at(row, c >> 7) + (c & 127)) = fp8_codes8(v, s);
  if ((c & 127) == 0) p.out.scale[row * p.out.srs + (c >> 7) * p.out.scs] = s.S;
}

// One scale for 128 x 128: a workgroup a block, 8 rows of 8 elements a thread, in registers
// between the block's maximum and its codes.
template <class T>
__device__ __forceinline__ void fp8_block(const Fp8RowArgs& p, uint32_t block) {
  __shared__ uint32_t sh[4];
  const uint32_t br = block / (uint32_t)p.nb, bc = block - br * (uint32_t)p.nb;
  const int t = threadIdx.x;
  const int32_t c = (int32_t)bc * 128 + (t & 15) * 8;
  float v[8][8];
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = (int64_t)br * 128 + i * 16 + (t >> 4);
    if (r < p.rows && c < p.cols) {
      load8(reinterpret_cast<const T*>(p.x) + r * p.cols + c, v[i]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] = 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, top_bits8(v[i]));
  top = max16_lanes(top);
  top = max(top, (uint32_t)__shfl_xor((int)top, 16));
  top = max(top, (uint32_t)__shfl_xor((int)top, 32));
  if ((t & 63) == 0) sh[t >> 6] = top;
  __syncthreads();
  const Fp8Scale s = fp8_scale(max(max(sh[0], sh[1]), max(sh[2], sh[3])));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = (int64_t)br * 128 + i * 16 + (t >> 4);
    if (r < p.rows) *reinterpret_cast<uint2*>(p.out.codes + r * p.out.ld + c) = fp8_codes8(v[i], s);
  }
  if (t == 0) p.out.scale[(int64_t)br * p.nb + bc] = s.S;
}

template <class T>
__global__ __launch_bounds__(256) void fp8_row_kernel(Fp8RowArgs p) {
  fp8_row<T>(p, blockIdx.x);
}
template <class T>
__global__ __launch_bounds__(256) void fp8_block_kernel(Fp8RowArgs p) {
  fp8_block<T>(p, blockIdx.x);
}
// The forward's operands: bf16 activations (nx workgroups) and fp32 weights.  16384 x 1024 and
// 4096 x 1024 22 us (72 MB, 3.3 TB/s: too short to get to the copy's rate).
__global__ __launch_bounds__(256) void fp8_forward_kernel(Fp8RowArgs x, Fp8RowArgs w, uint32_t nx) {
  if (blockIdx.x < nx) fp8_row<uint16_t>(x, blockIdx.x);
  else fp8_block<float>(w, blockIdx.x - nx);
}

// Groups along the columns, stored transposed: a workgroup takes 128 rows by 4 CQ columns
// through LDS, in quads of 4 columns that change places by the row's eighth, so that 16
// lanes, each with 8 rows of one quad, read different banks.
struct Fp8ColArgs {
  const void* x;       // dense [rows, cols], or codes
  const float* xs;     // codes: their scales [rows][nbx]
  int64_t ldx;         // elements (bytes) between rows
  Fp8Out out;          // [cols, rows]
  int64_t rows;
  int32_t cols, nbx;
};
struct Codes {};  // tag: E4M3 input under a scale per 128 of a row, grouped anew
struct Turn {};   // tag: E4M3 input whose codes are only transposed (a scale per 128 x 128)
template <class T>
struct ColOf {
  using Quad = uint32_t;
  static constexpr int CQ = 32;
};
template <>
struct ColOf<uint16_t> {
  using Quad = uint2;
  static constexpr int CQ = 32;
};
template <>
struct ColOf<float> {
  using Quad = float4;
  static constexpr int CQ = 16;
};

__device__ __forceinline__ void quad_values(uint2 q, float, float v[4]) {
  v[0] = __uint_as_float(q.x << 16);
  v[1] = __uint_as_float(q.x & 0xFFFF0000u);
  v[2] = __uint_as_float(q.y << 16);
  v[3] = __uint_as_float(q.y & 0xFFFF0000u);
}
__device__ __forceinline__ void quad_values(float4 q, float, float v[4]) { v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w; }
__device__ __forceinline__ void quad_values(uint32_t q, float s, float v[4]) {
  const f32x2v_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q, 1.0f, false), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q, 1.0f, true);
  v[0] = a.x * s; v[1] = a.y * s; v[2] = b.x * s; v[3] = b.y * s;
}

// The tile is in LDS, a barrier crossed: the columns' groups (or transposed codes).
constexpr int kColThreads = 512;
template <class T>
__device__ __forceinline__ void fp8_col_out(const Fp8Out& out, int32_t cols, int32_t c0, uint32_t by,
                                            typename ColOf<T>::Quad (*tile)[ColOf<T>::CQ], const float* rs) {
  constexpr int CQ = ColOf<T>::CQ;
  const int rg = threadIdx.x & 15;
#pragma unroll
  for (int k = 0; k < CQ * 16; k += kColThreads) {
    if (CQ * 16 < kColThreads && threadIdx.x >= CQ * 16) break;
    const int q = k / 16 + (threadIdx.x >> 4), col = c0 + q * 4;
    typename ColOf<T>::Quad raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[i] = tile[rg * 8 + i][q ^ rg];
    if constexpr (std::is_same<T, Turn>::value) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t pick = 0x0C0C0000u | (uint32_t)((j + 4) << 8) | (uint32_t)j;  // byte j of both
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __builtin_amdgcn_perm(raw[2 * i + 1], raw[2 * i], pick);
        if (col + j < cols) *reinterpret_cast<uint2*>(out.codes + out.at(col + j, by) + rg * 8) = uint2{h[0] | h[1] << 16, h[2] | h[3] << 16};
      }
    } else {
      float v[4][8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float u[4];
        quad_values(raw[i], std::is_same<T, Codes>::value ? rs[rg * 8 + i] : 1.0f, u);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j][i] = u[j];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const Fp8Scale s = fp8_scale(max16_lanes(top_bits8(v[j])));
        if (col + j < cols) {
          *reinterpret_cast<uint2*>(out.codes + out.at(col + j, by) + rg * 8) = fp8_codes8(v[j], s);
          if (rg == 0) out.scale[(col + j) * out.srs + by * out.scs] = s.S;
        }
      }
    }
  }
}

template <class T>
__device__ __forceinline__ void fp8_col(const Fp8ColArgs& p, uint32_t bx, uint32_t by, typename ColOf<T>::Quad (*tile)[ColOf<T>::CQ], float* rs) {
  constexpr int CQ = ColOf<T>::CQ;
  constexpr bool kDense = std::is_same<T, float>::value || std::is_same<T, uint16_t>::value;
  constexpr int VQ = std::is_same<T, float>::value ? 1 : kDense ? 2 : 4;  // quads of 16 bytes
  const int t = threadIdx.x;
  const int64_t r0 = (int64_t)by * 128;
  const int32_t c0 = (int32_t)bx * (4 * CQ);
#pragma unroll
  for (int i = t; i < 128 * CQ / VQ; i += kColThreads) {
    const int r = i / (CQ / VQ), q = i % (CQ / VQ) * VQ;
    const bool in = r0 + r < p.rows && c0 + q * 4 < p.cols;
    if constexpr (std::is_same<T, float>::value) {
      float4 a = {0.0f, 0.0f, 0.0f, 0.0f};
      if (in) a = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.x) + (r0 + r) * p.ldx + c0 + q * 4);
      tile[r][q ^ (r >> 3)] = a;
    } else {
      constexpr int es = kDense ? 2 : 1;
      uint4 a = {0u, 0u, 0u, 0u};
      if (in) a = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(p.x) + ((r0 + r) * p.ldx + c0 + q * 4) * es);
      if constexpr (kDense) {
        tile[r][q ^ (r >> 3)] = uint2{a.x, a.y};
        tile[r][(q + 1) ^ (r >> 3)] = uint2{a.z, a.w};
      } else {
        tile[r][q ^ (r >> 3)] = a.x;
        tile[r][(q + 1) ^ (r >> 3)] = a.y;
        tile[r][(q + 2) ^ (r >> 3)] = a.z;
        tile[r][(q + 3) ^ (r >> 3)] = a.w;
      }
    }
  }
  if constexpr (std::is_same<T, Codes>::value)
    if (t < 128) rs[t] = r0 + t < p.rows ? p.xs[(r0 + t) * p.nbx + bx] : 0.0f;
  __syncthreads();
  fp8_col_out<T>(p.out, p.cols, c0, by, tile, rs);
}
template <class T>
__global__ __launch_bounds__(kColThreads) void fp8_col_kernel(Fp8ColArgs p) {
  __shared__ __attribute__((aligned(16))) typename ColOf<T>::Quad tile[128][ColOf<T>::CQ];
  __shared__ float rs[128];
  fp8_col<T>(p, blockIdx.x, blockIdx.y, tile, rs);
}

// Both groupings of a dense bf16 matrix from one read: an output gradient is the left
// operand of both backward products.  128 x 128 a workgroup; a thread quantises 8
// neighbours of a row as it loads them.
struct Fp8DualArgs {
  const uint16_t* x;
  Fp8Out row, col;  // [rows, cols] and [cols, rows]
  int64_t rows;
  int32_t cols, nbc;
};
__device__ __forceinline__ void fp8_dual(const Fp8DualArgs& p, uint32_t bx, uint32_t by, uint2 (*tile)[32]) {
  const int t = threadIdx.x, h = t & 15;
  const int64_t r0 = (int64_t)by * 128;
  const int32_t c = (int32_t)bx * 128 + h * 8;
  constexpr int N = 128 * 16 / kColThreads, R = kColThreads / 16;  // loads of a thread, rows of one of all threads
  uint4 raw[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t r = r0 + i * R + (t >> 4);
    raw[i] = uint4{0u, 0u, 0u, 0u};
    if (r < p.rows && c < p.cols) raw[i] = *reinterpret_cast<const uint4*>(p.x + r * p.cols + c);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = i * R + (t >> 4);
    tile[r][(2 * h) ^ (r >> 3)] = uint2{raw[i].x, raw[i].y};
    tile[r][(2 * h + 1) ^ (r >> 3)] = uint2{raw[i].z, raw[i].w};
    float v[8];
    quad_values(uint2{raw[i].x, raw[i].y}, 1.0f, v);
    quad_values(uint2{raw[i].z, raw[i].w}, 1.0f, v + 4);
    const Fp8Scale s = fp8_scale(max16_lanes(top_bits8(v)));
    if (r0 + r < p.rows) {
      *reinterpret_cast<uint2*>(p.row.codes + p.row.at(r0 + r, bx) + h * 8) = fp8_codes8(v, s);
      if (h == 0) p.row.scale[(r0 + r) * p.row.srs + bx * p.row.scs] = s.S;
    }
  }
  __syncthreads();
  fp8_col_out<uint16_t>(p.col, p.cols, (int32_t)bx * 128, by, tile, nullptr);
}

// All operands of the backward pass in one launch: nd workgroups for dY, nw for the
// weights' codes turned, the others for the activations' grouped along the tokens.
// 16384 x 1024 -> 4096 65 us for 316 MB (4.9 TB/s): dY read once, written twice.
__global__ __launch_bounds__(kColThreads) void fp8_backward_kernel(Fp8DualArgs d, uint32_t nd, Fp8ColArgs w, uint32_t nw, Fp8ColArgs x) {
  __shared__ __attribute__((aligned(16))) uint2 tile[128][32];
  __shared__ float rs[128];
  uint32_t b = blockIdx.x;
  if (b < nd) return fp8_dual(d, b % (uint32_t)d.nbc, b / (uint32_t)d.nbc, tile);
  b -= nd;
  const bool is_w = b < nw;
  if (!is_w) b -= nw;
  uint32_t(*codes)[32] = reinterpret_cast<uint32_t(*)[32]>(tile);
  const uint32_t n = (uint32_t)((is_w ? w.cols : x.cols) + 127) / 128;
  if (is_w) fp8_col<Turn>(w, b % n, b / n, codes, rs);
  else fp8_col<Codes>(x, b % n, b / n, codes, rs);
}

// ---- values ----------------------------------------------------------------------
// 8 elements a thread; len is a multiple of 16.  16384 x 4096 to bf16 30.8 us (6.6 TB/s), to
// fp32 60.7.
template <bool F32>
__global__ __launch_bounds__(256) void fp8_values_kernel(const uint8_t* codes, const float* scale, int64_t rows, int32_t len,
                                                         int32_t nb, int block, void* out) {
  const uint32_t per = (uint32_t)len / 8, id = blockIdx.x * 256 + threadIdx.x, row = id / per;
  if (row >= rows) return;
  const int32_t c = (int32_t)(id - row * per) * 8;
  const uint2 q = *reinterpret_cast<const uint2*>(codes + (int64_t)row * nb * 128 + c);
  const float s = scale[(int64_t)(block ? row >> 7 : row) * nb + (c >> 7)];
  float v[8];
  quad_values(q.x, s, v);
  quad_values(q.y, s, v + 4);
  const int64_t at = (int64_t)row * len + c;
  if constexpr (F32) {
    float4* o = reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + at);
    o[0] = float4{v[0], v[1], v[2], v[3]};
    o[1] = float4{v[4], v[5], v[6], v[7]};
  } else {
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(out) + at) =
        uint4{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
  }
}

// ---- product ---------------------------------------------------------------------
// Per chunk of 128 the products of a tile's 16 x 16 part start from zero, and what they are
// is multiplied by both scales and added to the fp32 sum: two vector operations a result
// and chunk, between the matrix instructions of the next part.  With a scale per 128 rows
// of P they are one multiplication by a number and one fma.  PFLOP/s of C in bf16, P per
// 128 x 128 / per row, and in fp32 (exact products of codes decoded to f16, which
// vector operations bound): 8192^3 2.31 / 1.93, 0.93; 16384 x 1024 over 4096 2.07 / 1.75,
// 0.85; 16384 x 4096 over 1024, whose 134 MB of results are not covered by products, 1.54 /
// 1.44, 0.69.  The same instructions in the library, under one scale, do 2.90, 2.31 and 1.89.
struct Fp8GemmArgs {
  TileOp P, Q;        // P: B [J, K] (columns of C), Q: A [I, K] (rows of C)
  void* C;            // split: fp32 partial sums [splits][I][J], joined by fp8_join_kernel
  int64_t ldc, zstride;
  const float* partial;
  uint32_t tiles_p, tiles_q;
  int32_t nch, splits;
  int32_t bf16, accumulate, vec;  // vec: rows of C may be stored 16 bytes at a time
};

// N (a multiple of 4) neighbouring results from column j on of the row that starts at
// element `row` of C
template <int N>
__device__ __forceinline__ void fp8_store(const Fp8GemmArgs& p, int64_t row, int64_t j, const float (&v)[N]) {
  const int64_t J = p.P.rows;
  if (j >= J) return;
  const bool whole = p.vec && j + N <= J;
  if (p.bf16) {
    uint16_t* o = reinterpret_cast<uint16_t*>(p.C) + row + j;
    if (whole) {
      if constexpr (N == 4) {
        *reinterpret_cast<uint2*>(o) = uint2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
      } else {
#pragma unroll
        for (int k = 0; k < N; k += 8)
          *reinterpret_cast<uint4*>(o + k) = uint4{bf16_pair(v[k], v[k + 1]), bf16_pair(v[k + 2], v[k + 3]),
                                                  bf16_pair(v[k + 4], v[k + 5]), bf16_pair(v[k + 6], v[k + 7])};
      }
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (j + k < J) o[k] = (uint16_t)bf16_pair(v[k], 0.0f);
    }
  } else {
    float* o = reinterpret_cast<float*>(p.C) + row + j;
    if (whole) {
#pragma unroll
      for (int k = 0; k < N; k += 4) {
        float4 a = {v[k], v[k + 1], v[k + 2], v[k + 3]};
        if (p.accumulate) {
          const float4 c = *reinterpret_cast<const float4*>(o + k);
          a.x += c.x; a.y += c.y; a.z += c.z; a.w += c.w;
        }
        *reinterpret_cast<float4*>(o + k) = a;
      }
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (j + k < J) o[k] = p.accumulate ? o[k] + v[k] : v[k];
    }
  }
}

template <class T>
__device__ __forceinline__ void fp8_tiles(const Fp8GemmArgs& p, typename T::Smem& sm, uint32_t block, uint32_t blocks) {
  const typename T::Items items(p.tiles_p, p.tiles_q, (uint32_t)p.nch, (uint32_t)p.splits, block, blocks);
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
  T::run(p.P, p.Q, items, sm, [&](int64_t p0, int64_t q0, uint32_t z, typename T::Acc& acc) __attribute__((always_inline)) {
    const int64_t pw = p0 + (w / T::kWN) * T::kTM * 16 + g * 4 * T::PB, qw = q0 + (w % T::kWN) * T::kTN * 16;
    const int64_t at = p.zstride * z;
#pragma unroll
    for (int tn = 0; tn < T::kTN; ++tn) {
      const int64_t i = qw + T::q_row(tn, n);
      if (i < p.Q.rows) {
#pragma unroll
        for (int tb = 0; tb < T::kTM / T::PB; ++tb) {
          float v[4 * T::PB];
#pragma unroll
          for (int k = 0; k < 4 * T::PB; ++k) v[k] = acc[tb * T::PB + k / 4][tn][k % 4];
          fp8_store<4 * T::PB>(p, at + i * p.ldc, pw + tb * 16 * T::PB, v);
        }
      }
    }
  });
}
template <class T>
__global__ __launch_bounds__(T::NT, T::WAVES) void fp8_gemm_kernel(Fp8GemmArgs p) {
  __shared__ __attribute__((aligned(128))) typename T::Smem sm;
  fp8_tiles<T>(p, sm, blockIdx.x, gridDim.x);
}
// The backward's two products in tiles of one size, where the second fills what the first
// leaves idle: A's workgroups first.
template <class A, class B>
__global__ __launch_bounds__(A::NT, A::WAVES) void fp8_gemm_pair_kernel(Fp8GemmArgs a, Fp8GemmArgs b, uint32_t first) {
  static_assert(A::NT == B::NT && sizeof(typename A::Smem) == sizeof(typename B::Smem), "one tile");
  __shared__ __attribute__((aligned(128))) typename A::Smem sm;
  if (blockIdx.x < first) fp8_tiles<A>(a, sm, blockIdx.x, first);
  else fp8_tiles<B>(b, reinterpret_cast<typename B::Smem&>(sm), blockIdx.x - first, gridDim.x - first);
}

// Few rows of A (decoding): A whole in LDS, B read once.  From bf16 X (the linear layer's
// forward) each workgroup quantises X for itself, the first one storing the codes too,
// which saves the launch that would do it.  N 4096, K 1024: 1 row 5.7 us, 8 rows 6.9 (6 of
// them a chain of quantizing, one barrier, the codes' loads and the join of the waves).
struct Fp8FewArgs {
  Fp8GemmArgs g;
  const uint16_t* x;  // quantise [I, cols] bf16 into codes and scale [I][nb]; NULL: they are given
  int32_t cols, nb;
  uint8_t* codes;
  float* scale;
};
template <class S>
__global__ __launch_bounds__(S::NT, 2) void fp8_few_kernel(Fp8FewArgs a) {
  __shared__ typename S::Smem sm;
  const Fp8GemmArgs& p = a.g;
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4, I = (int)p.Q.rows;
  const int px = S::pitch(p.P.kb), per = a.nb * 16, all = I * per;  // 8-element pieces of a row, whole chunks
  float* xs = reinterpret_cast<float*>(sm.xs);
  auto put = [&](int t, int c, uint2 q, float s) __attribute__((always_inline)) {
    *reinterpret_cast<uint2*>(sm.x + t * px + c) = q;
    if ((c & 127) == 0) xs[(c >> 7) * S::TOKENS + t] = s;
  };
  auto stage = [&]() __attribute__((always_inline)) {
    // four pieces a thread at once, so that their loads are in flight together
    for (int i0 = threadIdx.x; i0 < all; i0 += 4 * S::NT) {
      if (a.x) {
        float v[4][8];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int i = i0 + u * S::NT, t = i / per, c = (i - t * per) * 8;
          if (i < all && c < a.cols) {
            load8(a.x + (int64_t)t * a.cols + c, v[u]);
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[u][k] = 0.0f;
          }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int i = i0 + u * S::NT, t = i / per, c = (i - t * per) * 8;
          const Fp8Scale f = fp8_scale(max16_lanes(top_bits8(v[u])));
          const uint2 q = fp8_codes8(v[u], f);
          if (i >= all) break;  // (whole groups of 16 lanes: a row's pieces are a multiple of 16)
          if (blockIdx.x == 0) {
            *reinterpret_cast<uint2*>(a.codes + (int64_t)t * a.nb * 128 + c) = q;
            if ((c & 127) == 0) a.scale[(int64_t)t * a.nb + (c >> 7)] = f.S;
          }
          put(t, c, q, f.S);
        }
      } else {
        uint2 q[4];
        float s[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int i = i0 + u * S::NT, t = i / per, c = (i - t * per) * 8;
          q[u] = uint2{0u, 0u};
          s[u] = 0.0f;
          if (i < all) {
            if (c < a.cols) q[u] = *reinterpret_cast<const uint2*>(a.codes + (int64_t)t * a.nb * 128 + c);
            s[u] = a.scale[(int64_t)t * a.nb + (c >> 7)];
          }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int i = i0 + u * S::NT, t = i / per, c = (i - t * per) * 8;
          if (i < all) put(t, c, q[u], s[u]);
        }
      }
    }
    __syncthreads();
  };
  S::run(p.P, sm, [&](uint32_t group, const typename S::Acc& acc) __attribute__((always_inline)) {
    static_assert(S::TOKENS == 16, "one tile of tokens");
    if (n < I) {
      const float v[4] = {acc[0].x, acc[0].y, acc[0].z, acc[0].w};
      fp8_store<4>(p, (int64_t)n * p.ldc, (int64_t)group * 16 + g * 4, v);
    }
  }, stage);
}

// C = (C +) the sum of the splits' results in order, 4 a thread; of one product or two.
// Memory: dW of 4096 x 1024 in 4 splits 10 us (84 MB).
__global__ __launch_bounds__(256) void fp8_join_kernel(Pair<Fp8GemmArgs> jobs) {
  const Share mine(jobs.first);
  const Fp8GemmArgs& p = jobs.x[mine.job];
  const int64_t I = p.Q.rows, J = p.P.rows, n = I * J, per = (J + 3) / 4;
  const int64_t id = (int64_t)mine.block * 256 + threadIdx.x, i = id / per, j = (id - i * per) * 4;
  if (i >= I) return;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const float* s = p.partial + i * J + j;
  if ((J & 3) == 0) {
#pragma unroll 4
    for (int z = 0; z < p.splits; ++z) {
      const float4 a = *reinterpret_cast<const float4*>(s + (int64_t)z * n);
      v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
    }
  } else {
    for (int z = 0; z < p.splits; ++z)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (j + k < J) v[k] += s[(int64_t)z * n + k];
  }
  fp8_store<4>(p, i * p.ldc, j, v);
}

template <int EL>
using TileBig = Tile<EL, 2, 4, 8, 4>;    // 256 x 256
template <int EL>
using TileMid = Tile<EL, 2, 2, 4, 4>;    // 128 x 128
template <int EL>
using TileSmall = Tile<EL, 2, 2, 2, 2>;  // 64 x 64

template <class T>
uint32_t tile_grid(Fp8GemmArgs& a) {
  a.tiles_p = (uint32_t)((a.P.rows + T::BM - 1) / T::BM);
  a.tiles_q = (uint32_t)((a.Q.rows + T::BN - 1) / T::BN);
  return T::grid((uint64_t)a.tiles_p * a.tiles_q * (uint32_t)a.splits);
}
template <class T>
void launch_tile(Fp8GemmArgs a, hipStream_t s) {
  const uint32_t grid = tile_grid<T>(a);
  fp8_gemm_kernel<T><<<grid, T::NT, 0, s>>>(a);
}
template <class A, class B>
void launch_pair(Fp8GemmArgs a, Fp8GemmArgs b, hipStream_t s) {
  const uint32_t first = tile_grid<A>(a), others = tile_grid<B>(b);
  fp8_gemm_pair_kernel<A, B><<<first + others, A::NT, 0, s>>>(a, b, first);
}

TileOp fp8_operand(const QView& q, bool blocked) {
  const Fp8Out at = fp8_out(q, blocked);
  TileOp o = {};
  o.p = q.codes;
  o.s = reinterpret_cast<const uint8_t*>(q.s128);
  o.rows = q.rows;
  o.ld = at.ld;
  o.bs = at.bs;
  o.cs = (int32_t)at.cs;
  o.kb = (int32_t)(blocked ? q.nb * 128 : q.len);  // (what lies beyond a caller's row is not read)
  o.srs = at.srs * 4;
  o.scs = at.scs * 4;
  return o;
}

// Rows of A that fp8_few_kernel takes: up to 16, an instruction tile, of up to 8192
// elements in all, as every workgroup quantises them.  Linear forward here and in tiles
// with the quantisation's launch, us: N 4096, K 1024: 1 row 5.7 and 9.2, 8 rows 6.9 and
// 10.1, 16 rows 9.1 and 10.1; K 2048: 1 row 8.5 and 9.2, 4 rows 9.6 and 9.6, 8 rows 11.7 and
// 9.8; K 256: 16 rows 4.9 and 6.4; N 50304, K 1024: 1 row 14.4 and 14.9, 8 rows 15.7 and 15.5,
// 16 rows 17.8 and 15.7.  (Tiles of 32 and 64 rows here: 24 rows of N 50304, K 1024 22.0
// and 15.7, 64 rows 38.8 and 16.6.)
using Few = Skinny<EL_FP8BX, 1, 34 * 1024>;
static_assert(Few::TOKENS * (2048 + 16) <= 34 * 1024 && Few::TOKENS * (2048 + 128 + 16) > 34 * 1024, "2048 elements");
bool is_few(int64_t M, int64_t K) { return Few::fits(M, K) && M * K <= 8192; }

// Tile and splits of a product, by an estimate of its time from what the tiles measure
// (us on MI355X; a chunk is 128 elements of the reduction): alone on its CU a tile of 64 /
// 128 / 256 takes 0.7 / 0.98 / 1.7 a chunk, with the CU full (4 / 2 / 1 workgroups) 0.94 /
// 1.09 / 1.7; with exact products 0.95 / 1.48 and 1.4 / 2.1 (decoded operands of a 256 x 256
// tile would not fit the registers).  A split costs a launch and its fp32 partial sums,
// written and read.
struct Fp8Plan {
  int tile, splits;
  double time, packed;  // packed: where other tiles take the places that it leaves idle
};
Fp8Plan fp8_plan(int64_t I, int64_t J, int64_t K, bool exact, int tile) {
  const double kAlone[3] = {exact ? 0.95 : 0.7, exact ? 1.48 : 0.98, 1.7}, kFull[3] = {exact ? 1.4 : 0.94, exact ? 2.1 : 1.09, 1.7},
               kFixed[3] = {2.5, 3.5, 5.0};
  constexpr int kSlots[3] = {4, 2, 1};
  const int64_t nch = (K + 127) / 128;
  const int64_t b = 64 << tile, n = ((I + b - 1) / b) * ((J + b - 1) / b), slots = kCus * kSlots[tile];
  Fp8Plan best = {tile, 1, 1e30, 1e30};
  for (int z = 1; z <= 16 && z * 4 <= std::max<int64_t>(nch, 4); z *= 2) {
    const int64_t items = n * z, full = items / slots, rest = items % slots, deep = (rest + kCus - 1) / kCus;
    const double chunks = (double)((nch + z - 1) / z);
    double t = (double)full * (chunks * kFull[tile] + kFixed[tile]);
    if (rest) {
      const double per = kSlots[tile] > 1 ? kAlone[tile] + (kFull[tile] - kAlone[tile]) * (double)(deep - 1) / (kSlots[tile] - 1) : kFull[tile];
      t += chunks * per + kFixed[tile];
    }
    const double join = z > 1 ? 3.0 + (double)I * (double)J * 8.0 * z / 5e6 : 0.0;
    if (t + join < best.time)
      best = Fp8Plan{tile, z, t + join, (double)items * (chunks * kFull[tile] + kFixed[tile]) / (double)slots + join};
  }
  return best;
}
Fp8Plan fp8_plan(int64_t I, int64_t J, int64_t K, bool exact) {
  Fp8Plan best = fp8_plan(I, J, K, exact, 0);
  for (int tile = 1; tile < (exact ? 2 : 3); ++tile)
    if (const Fp8Plan p = fp8_plan(I, J, K, exact, tile); p.time < best.time) best = p;
  return best;
}

size_t split_bytes(int64_t I, int64_t J, int64_t K, bool exact) {
  const int z = fp8_plan(I, J, K, exact).splits;
  return z > 1 ? (size_t)z * (size_t)I * (size_t)J * 4 : 0;
}

Fp8GemmArgs fp8_args(const TileOp& Q, const TileOp& P, int64_t K, void* C, int c_dtype, int64_t ldc, int accumulate) {
  Fp8GemmArgs a = {};
  a.P = P;
  a.Q = Q;
  a.C = C;
  a.ldc = ldc;
  a.nch = (int32_t)((K + 127) / 128);
  a.splits = 1;
  a.bf16 = c_dtype == TJ2_BF16;
  a.accumulate = accumulate;
  a.vec = (reinterpret_cast<uintptr_t>(C) & 15u) == 0 && (ldc * (a.bf16 ? 2 : 4)) % 16 == 0;
  return a;
}

// A planned product; split: `part` is what the tiles write, joined into `out`.
struct Fp8Product {
  Fp8GemmArgs part, out;
  int tile;
  bool exact, block;
};
Fp8Product fp8_product(const Fp8GemmArgs& a, const Fp8Plan& plan, bool block, float* partial) {
  Fp8Product x = {a, a, plan.tile, !a.bf16, block};
  x.part.splits = x.out.splits = partial ? plan.splits : 1;
  if (x.part.splits > 1) {
    x.out.partial = partial;
    x.part.C = partial;
    x.part.ldc = a.P.rows;
    x.part.zstride = a.Q.rows * a.P.rows;
    x.part.bf16 = x.part.accumulate = 0;
    x.part.vec = (a.P.rows & 3) == 0;
  }
  return x;
}
hipError_t launch_product(const Fp8Product& x, hipStream_t s) {
  auto tiles = [&](auto el) {
    constexpr int EL = decltype(el)::value;
    if constexpr (EL == EL_FP8 || EL == EL_FP8B)
      if (x.tile == 2) return launch_tile<TileBig<EL>>(x.part, s);
    if (x.tile == 1) launch_tile<TileMid<EL>>(x.part, s);
    else launch_tile<TileSmall<EL>>(x.part, s);
  };
  if (x.exact && x.block) tiles(std::integral_constant<int, EL_FP8BX>{});
  else if (x.exact) tiles(std::integral_constant<int, EL_FP8X>{});
  else if (x.block) tiles(std::integral_constant<int, EL_FP8B>{});
  else tiles(std::integral_constant<int, EL_FP8>{});
  return hipGetLastError();
}
// The joins of those that are split.
hipError_t launch_joins(const Fp8Product* x, int n, hipStream_t s) {
  Pair<Fp8GemmArgs> jobs = {};
  uint32_t grid[2] = {0, 0};
  int k = 0;
  for (int i = 0; i < n; ++i) {
    if (x[i].out.splits == 1) continue;
    jobs.x[k] = x[i].out;
    grid[k++] = (uint32_t)((x[i].out.Q.rows * ((x[i].out.P.rows + 3) / 4) + 255) / 256);
  }
  if (!k) return hipSuccess;
  jobs.first = grid[0];
  fp8_join_kernel<<<grid[0] + grid[1], 256, 0, s>>>(jobs);
  return hipGetLastError();
}
hipError_t run_product(const Fp8GemmArgs& a, int64_t K, bool block, float* partial, hipStream_t s) {
  const Fp8Product x = fp8_product(a, fp8_plan(a.Q.rows, a.P.rows, K, !a.bf16), block, partial);
  if (hipError_t e = launch_product(x, s); e != hipSuccess) return e;
  return launch_joins(&x, 1, s);
}

hipError_t run_few(const Fp8GemmArgs& g, const QView& A, const void* x, hipStream_t s) {
  Fp8FewArgs f = {};
  f.g = g;
  f.x = reinterpret_cast<const uint16_t*>(x);
  f.cols = (int32_t)A.len;
  f.nb = (int32_t)A.nb;
  f.codes = A.codes;
  f.scale = A.s128;
  fp8_few_kernel<Few><<<Few::grid(g.P.rows), Few::NT, 0, s>>>(f);
  return hipGetLastError();
}

Fp8RowArgs row_args(const void* x, const QView& out) { return Fp8RowArgs{x, fp8_out(out, false), out.rows, (int32_t)out.len, (int32_t)out.nb}; }
uint32_t row_grid(const Fp8RowArgs& a) { return (uint32_t)(((uint64_t)a.rows * (uint64_t)a.nb * 16 + 255) / 256); }
uint32_t block_grid(const Fp8RowArgs& a) { return (uint32_t)((a.rows + 127) / 128 * a.nb); }
Fp8ColArgs col_args(const void* x, const float* xs, int64_t ldx, int64_t rows, int64_t cols, const QView& out, bool blocked) {
  return Fp8ColArgs{x, xs, ldx, fp8_out(out, blocked), rows, (int32_t)cols, (int32_t)((cols + 127) / 128)};
}

}  // namespace

hipError_t launch_fp8_quant(const Fp8QuantParams& q, hipStream_t s) {
  if (q.out.fmt == TJ2_FP8_BLOCK) {
    const Fp8RowArgs a = row_args(q.x, q.out);
    if (q.in_dtype == TJ2_BF16) fp8_block_kernel<uint16_t><<<block_grid(a), 256, 0, s>>>(a);
    else fp8_block_kernel<float><<<block_grid(a), 256, 0, s>>>(a);
  } else if (q.grouping == TJ2_GROUP_ROW) {
    const Fp8RowArgs a = row_args(q.x, q.out);
    if (q.in_dtype == TJ2_BF16) fp8_row_kernel<uint16_t><<<row_grid(a), 256, 0, s>>>(a);
    else fp8_row_kernel<float><<<row_grid(a), 256, 0, s>>>(a);
  } else {
    const uint32_t by = (uint32_t)((q.rows + 127) / 128);
    if (q.in_dtype == TJ2_FP8) {
      fp8_col_kernel<Codes><<<dim3((uint32_t)((q.cols + 127) / 128), by), kColThreads, 0, s>>>(
          col_args(q.xq.codes, q.xq.s128, q.xq.nb * 128, q.rows, q.cols, q.out, false));
    } else if (q.in_dtype == TJ2_BF16) {
      fp8_col_kernel<uint16_t><<<dim3((uint32_t)((q.cols + 127) / 128), by), kColThreads, 0, s>>>(
          col_args(q.x, nullptr, q.cols, q.rows, q.cols, q.out, false));
    } else {
      fp8_col_kernel<float><<<dim3((uint32_t)((q.cols + 63) / 64), by), kColThreads, 0, s>>>(
          col_args(q.x, nullptr, q.cols, q.rows, q.cols, q.out, false));
    }
  }
  return hipGetLastError();
}

hipError_t launch_fp8_values(const QView& q, void* out, int dtype, hipStream_t s) {
  const uint32_t grid = (uint32_t)(((uint64_t)q.rows * (uint64_t)(q.len / 8) + 255) / 256);
  const int block = q.fmt == TJ2_FP8_BLOCK;
  if (dtype == TJ2_F32) fp8_values_kernel<true><<<grid, 256, 0, s>>>(q.codes, q.s128, q.rows, (int32_t)q.len, (int32_t)q.nb, block, out);
  else fp8_values_kernel<false><<<grid, 256, 0, s>>>(q.codes, q.s128, q.rows, (int32_t)q.len, (int32_t)q.nb, block, out);
  return hipGetLastError();
}

// of either type of results
size_t fp8_gemm_workspace_bytes(int64_t I, int64_t J, int64_t K) { return std::max(split_bytes(I, J, K, false), split_bytes(I, J, K, true)); }

hipError_t launch_fp8_gemm(const QView& A, const QView& B, void* C, int c_dtype, int64_t ldc, int accumulate, float* partial,
                           hipStream_t s) {
  const Fp8GemmArgs a = fp8_args(fp8_operand(A, false), fp8_operand(B, false), A.len, C, c_dtype, ldc, accumulate);
  const bool block = B.fmt == TJ2_FP8_BLOCK;
  if (block && is_few(A.rows, A.len)) return run_few(a, A, nullptr, s);
  return run_product(a, A.len, block, partial, s);
}

size_t fp8_linear_fwd_workspace_bytes(int64_t M, int64_t N, int64_t K) { return is_few(M, K) ? 0 : fp8_gemm_workspace_bytes(M, N, K); }

hipError_t launch_fp8_linear_fwd(const void* X, const float* W, const QView& Xq, const QView& Wq, void* Y, int y_dtype,
                                 float* partial, hipStream_t s) {
  const Fp8RowArgs x = row_args(X, Xq), w = row_args(W, Wq);
  const Fp8GemmArgs a = fp8_args(fp8_operand(Xq, false), fp8_operand(Wq, false), Xq.len, Y, y_dtype, Wq.rows, 0);
  const bool few = is_few(Xq.rows, Xq.len);
  if (few || !X) {
    if (W) fp8_block_kernel<float><<<block_grid(w), 256, 0, s>>>(w);
  } else if (W) {
    fp8_forward_kernel<<<row_grid(x) + block_grid(w), 256, 0, s>>>(x, w, row_grid(x));
  } else {
    fp8_row_kernel<uint16_t><<<row_grid(x), 256, 0, s>>>(x);
  }
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  if (few) return run_few(a, Xq, X, s);
  return run_product(a, Xq.len, true, partial, s);
}

namespace {
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
// a blocked operand of the backward pass: codes, and the scales that follow them
size_t blocked_codes(int64_t rows, int64_t len) { return (size_t)((rows + 127) / 128 * 128) * (size_t)((len + 127) / 128 * 128); }
size_t blocked_bytes(int64_t rows, int64_t len) { return up256(blocked_codes(rows, len)) + up256(blocked_codes(rows, len) / 32); }
// The backward's plans: of tiles of 64 or 128 for both, they run in one launch.
struct Fp8BwdPlan {
  Fp8Plan x, w;
  Fp8BwdPlan(int64_t M, int64_t N, int64_t K, bool exact_dx) : x(fp8_plan(M, K, N, exact_dx)), w(fp8_plan(N, K, M, true)) {
    double least = x.time + w.time;
    for (int tile = 0; tile < 2; ++tile) {
      const Fp8Plan a = fp8_plan(M, K, N, exact_dx, tile), b = fp8_plan(N, K, M, true, tile);
      // the launch saved, and the CUs that either leaves idle
      const double t = std::max({a.time, b.time, a.packed + b.packed});
      if (t < least) {
        least = t;
        x = a;
        w = b;
      }
    }
  }
  bool together() const { return x.tile == w.tile; }
};
struct Fp8BwdSpace {
  size_t dy, dyt, wt, xt, px, pw, bytes;
  Fp8BwdSpace(int64_t M, int64_t N, int64_t K) {
    // (of either type of dX)
    const Fp8BwdPlan plan[2] = {{M, N, K, false}, {M, N, K, true}};
    auto part = [](const Fp8Plan& p, int64_t I, int64_t J) { return p.splits > 1 ? (size_t)p.splits * (size_t)(I * J) * 4 : 0; };
    size_t at = 0;
    auto take = [&](size_t n) { const size_t a = at; at += up256(n); return a; };
    dy = take(blocked_bytes(M, N));
    dyt = take(blocked_bytes(N, M));
    wt = take(blocked_codes(K, N));
    xt = take(blocked_bytes(K, M));
    px = take(std::max(part(plan[0].x, M, K), part(plan[1].x, M, K)));
    pw = take(std::max(part(plan[0].w, N, K), part(plan[1].w, N, K)));
    bytes = at;
  }
};
QView blocked_view(uint8_t* at, int64_t rows, int64_t len) {
  QView q = {};
  q.codes = at;
  q.s128 = reinterpret_cast<float*>(at + up256(blocked_codes(rows, len)));
  q.rows = rows;
  q.len = len;
  q.nb = (len + 127) / 128;
  q.fmt = TJ2_FP8;
  return q;
}
}  // namespace

size_t fp8_linear_bwd_workspace_bytes(int64_t M, int64_t N, int64_t K) { return Fp8BwdSpace(M, N, K).bytes; }

hipError_t launch_fp8_linear_bwd(const void* dY, const QView& Xq, const QView& Wq, void* dX, int dx_dtype, float* dW, void* ws,
                                 hipStream_t s) {
  const int64_t M = Xq.rows, N = Wq.rows, K = Xq.len;
  const Fp8BwdSpace sp(M, N, K);
  uint8_t* w = reinterpret_cast<uint8_t*>(ws);
  const QView dy = blocked_view(w + sp.dy, M, N), dyt = blocked_view(w + sp.dyt, N, M), wt = blocked_view(w + sp.wt, K, N),
              xt = blocked_view(w + sp.xt, K, M);
  const Fp8DualArgs d = {reinterpret_cast<const uint16_t*>(dY), fp8_out(dy, true), fp8_out(dyt, true), M, (int32_t)N, (int32_t)((N + 127) / 128)};
  const Fp8ColArgs tw = col_args(Wq.codes, nullptr, Wq.nb * 128, N, K, wt, true), tx = col_args(Xq.codes, Xq.s128, Xq.nb * 128, M, K, xt, true);
  const uint32_t kb = (uint32_t)((K + 127) / 128), mb = (uint32_t)((M + 127) / 128), nb = (uint32_t)((N + 127) / 128);
  fp8_backward_kernel<<<nb * mb + kb * nb + kb * mb, kColThreads, 0, s>>>(d, nb * mb, tw, kb * nb, tx);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  TileOp P = fp8_operand(wt, true);
  P.s = reinterpret_cast<const uint8_t*>(Wq.s128);  // of the turned codes: the same scales, read the other way
  P.srs = 4;
  P.scs = Wq.nb * 4;
  const Fp8BwdPlan plan(M, N, K, dx_dtype == TJ2_F32);
  const Fp8Product x[2] = {
      fp8_product(fp8_args(fp8_operand(dy, true), P, N, dX, dx_dtype, K, 0), plan.x, true, reinterpret_cast<float*>(w + sp.px)),
      fp8_product(fp8_args(fp8_operand(dyt, true), fp8_operand(xt, true), M, dW, TJ2_F32, K, 0), plan.w, false,
                  reinterpret_cast<float*>(w + sp.pw))};
  if (plan.together()) {
    if (x[0].exact && x[0].tile) launch_pair<TileMid<EL_FP8X>, TileMid<EL_FP8BX>>(x[1].part, x[0].part, s);
    else if (x[0].exact) launch_pair<TileSmall<EL_FP8X>, TileSmall<EL_FP8BX>>(x[1].part, x[0].part, s);
    else if (x[0].tile) launch_pair<TileMid<EL_FP8X>, TileMid<EL_FP8B>>(x[1].part, x[0].part, s);
    else launch_pair<TileSmall<EL_FP8X>, TileSmall<EL_FP8B>>(x[1].part, x[0].part, s);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  } else {
    for (const Fp8Product& p : x)
      if (hipError_t e = launch_product(p, s); e != hipSuccess) return e;
  }
  return launch_joins(x, 2, s);
}

}  // namespace tj2
