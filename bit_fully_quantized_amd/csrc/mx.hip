// Microscaled 4-bit floating point (MXFP4) for gfx950: quantiser, its inverse and
// the product.
//
// A group of 32 consecutive elements shares one power of two, v = q 2^e with q
// in E2M1 {0, .5, 1, 1.5, 2, 3, 4, 6} and the byte e + 127.  gfx950 multiplies the
// format as it is stored (v_mfma_scale_f32_16x16x128_f8f6f4: four times the bf16
// rate, a quarter of the bytes), where the double block's E4M3 scales have to be
// decoded to f16 first.
#include <algorithm>

#include "tj2_skinny.h"

namespace tj2 {
namespace {

// ---- quantiser -------------------------------------------------------------------
// Scale byte of a group whose largest magnitude has the fp32 bits `top`.
//   RTN: e = floor(log2 top) - 2, so the group's top binade is E2M1's (4 to 8; values
//        above 6 saturate), the rule of the OCP microscaling formats.
//   SR:  the smallest e with top <= 6 2^e: nothing saturates, so the rounding stays
//        unbiased.
// Clamped to byte 0 (2^-127); a group with an infinity or NaN gets 255 (NaN).
template <bool SR>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
  if (top >= 0x7F800000u) return 255u;
  const int e = (int)(top >> 23) - ((SR && (top & 0x7FFFFFu) > 0x400000u) ? 1 : 2);
  return (uint32_t)max(e, 0);
}

// 2^-e of a scale byte: exact, and v * 2^-e too (below 8; subnormal v become normal)
__device__ __forceinline__ float mx_inverse(uint32_t byte) {
  return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}
// 2^e of a scale byte
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7FC00000u) : byte ? __uint_as_float(byte << 23) : 0x1p-127f;
}

// 16 values to 8 bytes of codes; a group with a NaN scale gets zeros.
template <bool SR>
__device__ __forceinline__ uint2 mx_codes16(const float v[16], uint32_t byte, uint64_t block, uint64_t seed, uint64_t offset) {
  const float inv = mx_inverse(byte);
  float y[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = v[i] * inv;
  uint32_t c[2];
  if constexpr (SR) {
    uint32_t r[16];
    draws8(block, seed, offset, r);
    draws8(block + 1, seed, offset, r + 8);
    e2m1_sr16(y, r, c);
  } else {
    e2m1_rtn16(y, c);
  }
  return byte == 255u ? uint2{0u, 0u} : uint2{c[0], c[1]};
}

__device__ __forceinline__ uint32_t top_bits16(const float v[16]) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

template <class T>
__device__ __forceinline__ void load16(const T* p, float v[16]);
template <>
__device__ __forceinline__ void load16<uint16_t>(const uint16_t* p, float v[16]) {
  const uint4* q = reinterpret_cast<const uint4*>(p);
  const uint4 a = q[0], b = q[1];
  const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
template <>
__device__ __forceinline__ void load16<float>(const float* p, float v[16]) {
  const float4* q = reinterpret_cast<const float4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 a = q[i];
    v[4 * i] = a.x; v[4 * i + 1] = a.y; v[4 * i + 2] = a.z; v[4 * i + 3] = a.w;
  }
}

struct MxRowArgs {
  const void* x;
  uint8_t* codes;
  uint8_t* scale;
  int64_t rows;
  int32_t cols, nb;  // elements and 128-element blocks per row
  uint32_t mask;
  uint64_t seed, offset;
};

// Groups along the rows.  A thread takes 16 neighbouring elements, a pair of lanes
// a group (the pair's larger top by one DPP swap), eight threads a 128-element
// block, padding included.  Bound by memory: 16384 x 1024 bf16 in 8.7 us, 4.9 TB/s.
template <class T, bool SR, bool RHT>
__device__ __forceinline__ void mx_row(const MxRowArgs& p, uint32_t block) {
  const int64_t id = (int64_t)block * 256 + threadIdx.x;
  const int32_t per = p.nb * 8;
  const int64_t row = id / per;
  if (row >= p.rows) return;
  const int32_t h = (int32_t)(id - row * per), c = h * 16;
  float v[16];
  if (c < p.cols) {
    load16<T>(reinterpret_cast<const T*>(p.x) + row * p.cols + c, v);
    if constexpr (RHT) rht16(v, p.mask);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.0f;
  }
  uint32_t top = top_bits16(v);
  top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0xB1, 0xF, 0xF, false));  // the other half of the group
  const uint32_t byte = mx_scale_byte<SR>(top);
  const int64_t padded = ((int64_t)p.cols + 31) / 32 * 32;
  const uint2 q = mx_codes16<SR>(v, byte, (uint64_t)(row * padded + c) >> 3, p.seed, p.offset);
  *reinterpret_cast<uint2*>(p.codes + (row * per + h) * 8) = c < p.cols ? q : uint2{0u, 0u};
  if (!(h & 1)) p.scale[(row * per + h) >> 1] = (uint8_t)byte;
}

template <class T, bool SR, bool RHT>
__global__ __launch_bounds__(256) void mx_row_kernel(MxRowArgs p) {
  mx_row<T, SR, RHT>(p, blockIdx.x);
}
// The forward's operands: bf16 activations (nx workgroups) and fp32 weights.
__global__ __launch_bounds__(256) void mx_row_pair_kernel(MxRowArgs x, MxRowArgs w, uint32_t nx) {
  if (blockIdx.x < nx) mx_row<uint16_t, false, false>(x, blockIdx.x);
  else mx_row<float, false, false>(w, blockIdx.x - nx);
}

// Where an operand's groups go: row r's block of 128 elements b has its 64 bytes of
// codes at at(r, b) and its 4 scale bytes at a sixteenth of that.  Row-major, or (what
// only the backward's own products read) blocked as TileOp says: with rows a power of
// two apart a product's loads meet in few channels of the L2 (4096 x 4096 over 16384:
// 158 us, and 144 at a pitch of 33 lines; backward of 4096 x 4096 over 1024 61.2 us
// row-major, 59.6 blocked).
struct MxOut {
  uint8_t *codes, *scale;
  int64_t ld, bs, cs;
  __device__ __forceinline__ int64_t at(int64_t row, uint32_t block) const {
    return (row >> 7) * bs + (row & 127) * ld + (int64_t)(block >> 1) * cs + (block & 1) * 64;
  }
};
MxOut mx_out(const QView& q, bool blocked) {
  if (blocked) return MxOut{q.codes, q.s16, 128, (q.nb + 1) / 2 * 16384, 16384};
  return MxOut{q.codes, q.s16, q.nb * 64, q.nb * 64 * 128, 128};
}

struct MxColArgs {
  const void* x;       // dense [rows, cols], or codes of an MXFP4 operand [rows, cols]
  const uint8_t* xs;   // its scale bytes
  int64_t ldx, lds;    // codes and scale bytes per row of it
  MxOut out;           // [cols, rows]
  int32_t rows, cols, nb;
  uint32_t mask;
  uint64_t seed, offset;
};

struct MxIn {};  // tag: MXFP4 input

// Groups along the columns, stored transposed.  A workgroup takes 128 rows by 64
// columns through LDS: rows are read whole, then each thread owns 32 rows of one
// column, a group, and writes its 16 bytes (four groups of a column make a line of
// 64).  MXFP4 input is decoded to bf16 on the way, which holds its values exactly.
// Bound by memory: 16384 x 4096 bf16 in 34 us, 5 TB/s (35 with the transform, 44 with
// stochastic rounding too, which its draws bound; from memory that no cache holds 45
// with the transform).  128 columns a workgroup and two a thread: 35, 37 and 46.
template <class T>
using MxColElement = std::conditional_t<std::is_same<T, float>::value, float, uint16_t>;
template <class T, bool SR, bool RHT>
__device__ __forceinline__ void mx_col(const MxColArgs& p, uint32_t bx, uint32_t by, MxColElement<T> (*tile)[64], uint8_t (*sb)[4]) {
  constexpr bool kMx = std::is_same<T, MxIn>::value;
  constexpr bool kF32 = std::is_same<T, float>::value;
  using E = MxColElement<T>;
  const int t = threadIdx.x;
  const int32_t r0 = (int32_t)by * 128, c0 = (int32_t)bx * 64;
  // 8 elements a load: 8 loads a row
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int q = i * 256 + t, r = q >> 3, c = (q & 7) * 8;
    const bool in = r0 + r < p.rows && c0 + c < p.cols;
    const int64_t row = r0 + r;
    if constexpr (kF32) {
      float4 a = {0.0f, 0.0f, 0.0f, 0.0f}, b = a;
      if (in) {
        const float4* s = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.x) + row * p.ldx + c0 + c);
        a = s[0];
        b = s[1];
      }
      *reinterpret_cast<float4*>(&tile[r][c]) = a;
      *reinterpret_cast<float4*>(&tile[r][c + 4]) = b;
    } else if constexpr (!kMx) {
      uint4 a = {0u, 0u, 0u, 0u};
      if (in) a = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.x) + row * p.ldx + c0 + c);
      *reinterpret_cast<uint4*>(&tile[r][c]) = a;
    } else {
      uint4 a = {0u, 0u, 0u, 0u};
      if (in) {
        const uint32_t codes = *reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint8_t*>(p.x) + row * p.ldx + (c0 + c) / 2);
        const float s = mx_scale(p.xs[row * p.lds + (c0 + c) / 32]);
        uint32_t w[4];
        static_for<4>([&](auto k) __attribute__((always_inline)) {
          constexpr int b = decltype(k)::value;
          const f32x2v_t v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, b);
          // exact in bf16: an E2M1 value times a power of two (2^-128 and up)
          w[b] = (__float_as_uint(v.x * s) >> 16) | (__float_as_uint(v.y * s) & 0xFFFF0000u);
        });
        a = uint4{w[0], w[1], w[2], w[3]};
      }
      *reinterpret_cast<uint4*>(&tile[r][c]) = a;
    }
  }
  __syncthreads();
  const int c = t & 63, rg = t >> 6;
  float v[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const E e = tile[rg * 32 + i][c];
    if constexpr (kF32) v[i] = e;
    else v[i] = __uint_as_float((uint32_t)e << 16);
  }
  const int32_t first = r0 + rg * 32;
  if constexpr (RHT) {
    // a last piece of fewer than 16 rows stays as it is
    if (first + 16 <= p.rows) rht16(v, p.mask);
    if (first + 32 <= p.rows) rht16(v + 16, p.mask);
  }
  const uint32_t byte = mx_scale_byte<SR>(max(top_bits16(v), top_bits16(v + 16)));
  const int64_t col = c0 + c;
  const int64_t padded = ((int64_t)p.rows + 31) / 32 * 32;
  const uint64_t block = (uint64_t)(col * padded + first) >> 3;
  const uint2 a = mx_codes16<SR>(v, byte, block, p.seed, p.offset);
  const uint2 b = mx_codes16<SR>(v + 16, byte, block + 2, p.seed, p.offset);
  sb[c][rg] = (uint8_t)byte;
  if (col < p.cols)
    *reinterpret_cast<uint4*>(p.out.codes + p.out.at(col, by) + rg * 16) = uint4{a.x, a.y, b.x, b.y};
  __syncthreads();
  if (t < 64 && c0 + t < p.cols)
    *reinterpret_cast<uint32_t*>(p.out.scale + p.out.at(c0 + t, by) / 16) = *reinterpret_cast<const uint32_t*>(sb[t]);
}
template <class T, bool SR, bool RHT>
__global__ __launch_bounds__(256) void mx_col_kernel(MxColArgs p) {
  __shared__ __attribute__((aligned(16))) MxColElement<T> tile[128][64];
  __shared__ __attribute__((aligned(4))) uint8_t sb[64][4];
  mx_col<T, SR, RHT>(p, blockIdx.x, blockIdx.y, tile, sb);
}

// Both groupings of a dense bf16 matrix from one read: an output gradient is the left
// operand of both backward products.  A workgroup takes 128 x 128 elements; a thread
// quantises 16 neighbouring elements of a row as it loads them (mx_row_kernel), leaves
// them in LDS and then owns 32 rows of two neighbouring columns.  Paddings of both
// outputs lie in the tiles and are written with them.  (16384 x 4096: 51 us, 4 TB/s, where
// the two kernels one after the other took 38 + 34; 76 us with the transform and
// stochastic rounding, whose draws, ten rounds of two 64-bit products for eight
// elements, then bound it.)
struct MxDualArgs {
  const uint16_t* x;       // [rows, cols]
  MxOut row, col;          // [rows, cols] and [cols, rows]
  int32_t rows, cols, nbr, nbc;    // 128-element blocks of a column and of a row
  uint32_t row_mask, col_mask;
  uint64_t seed, row_offset, col_offset;
};

template <bool SR, bool RHT>
__device__ __forceinline__ void mx_dual(const MxDualArgs& p, uint32_t bx, uint32_t by, uint16_t (*tile)[128], uint8_t (*sb)[4]) {
  const int t = threadIdx.x;
  const int32_t r0 = (int32_t)by * 128, c0 = (int32_t)bx * 128;
  const int h = t & 7, c = c0 + h * 16;
  uint4 raw[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + i * 32 + (t >> 3);
    raw[i][0] = raw[i][1] = uint4{0u, 0u, 0u, 0u};
    if (r < p.rows && c < p.cols) {
      const uint4* s = reinterpret_cast<const uint4*>(p.x + r * p.cols + c);
      raw[i][0] = s[0];
      raw[i][1] = s[1];
    }
  }
  const int64_t padded_c = ((int64_t)p.cols + 31) / 32 * 32;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 32 + (t >> 3);
    uint4* s = reinterpret_cast<uint4*>(&tile[r][h * 16]);
    s[0] = raw[i][0];
    s[1] = raw[i][1];
    float v[16];
    load16<uint16_t>(reinterpret_cast<const uint16_t*>(raw[i]), v);
    if constexpr (RHT) rht16(v, p.row_mask);
    uint32_t top = top_bits16(v);
    top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0xB1, 0xF, 0xF, false));
    const uint32_t byte = mx_scale_byte<SR>(top);
    const int64_t row = r0 + r;
    const uint2 q = mx_codes16<SR>(v, byte, (uint64_t)(row * padded_c + c) >> 3, p.seed, p.row_offset);
    if (row < p.rows) {
      const int64_t at = p.row.at(row, bx) + h * 8;
      *reinterpret_cast<uint2*>(p.row.codes + at) = c < p.cols ? q : uint2{0u, 0u};
      if (!(h & 1)) p.row.scale[at / 16] = (uint8_t)byte;
    }
  }
  __syncthreads();
  const int64_t padded_r = ((int64_t)p.rows + 31) / 32 * 32;
  const int cc = 2 * (t & 63), rg = t >> 6;
  const int32_t first = r0 + rg * 32;
  uint32_t w[32];
#pragma unroll
  for (int k = 0; k < 32; ++k) w[k] = *reinterpret_cast<const uint32_t*>(&tile[rg * 32 + k][cc]);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float v[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(i ? w[k] & 0xFFFF0000u : w[k] << 16);
    if constexpr (RHT) {
      // a last piece of fewer than 16 rows stays as it is
      if (first + 16 <= p.rows) rht16(v, p.col_mask);
      if (first + 32 <= p.rows) rht16(v + 16, p.col_mask);
    }
    const uint32_t byte = mx_scale_byte<SR>(max(top_bits16(v), top_bits16(v + 16)));
    const int64_t col = c0 + cc + i;
    const uint64_t block = (uint64_t)(col * padded_r + first) >> 3;
    const uint2 a = mx_codes16<SR>(v, byte, block, p.seed, p.col_offset);
    const uint2 b = mx_codes16<SR>(v + 16, byte, block + 2, p.seed, p.col_offset);
    sb[cc + i][rg] = (uint8_t)byte;
    if (col < p.cols)
      *reinterpret_cast<uint4*>(p.col.codes + p.col.at(col, by) + rg * 16) = uint4{a.x, a.y, b.x, b.y};
  }
  __syncthreads();
  if (t < 128 && c0 + t < p.cols)
    *reinterpret_cast<uint32_t*>(p.col.scale + p.col.at(c0 + t, by) / 16) = *reinterpret_cast<const uint32_t*>(sb[t]);
}

// All operands of the backward pass in one launch: nd workgroups for dY, the others for
// the codes of the weights and of the activations.
// (Passes over few tokens are as long as their launches: backward of 700 x 2000 over 400
// 32 us with a launch for each operand, product and join, 20 with one for each kind.)
template <bool SR, bool RHT>
__global__ __launch_bounds__(256) void mx_backward_kernel(MxDualArgs d, uint32_t nd, Pair<MxColArgs> codes) {
  __shared__ __attribute__((aligned(16))) uint16_t tile[128][128];
  __shared__ __attribute__((aligned(4))) uint8_t sb[128][4];
  uint32_t b = blockIdx.x;
  if (b < nd) return mx_dual<SR, RHT>(d, b % (uint32_t)d.nbc, b / (uint32_t)d.nbc, tile, sb);
  b -= nd;
  const int job = b < codes.first ? 0 : 1;
  const MxColArgs& p = codes.x[job];
  if (job) b -= codes.first;
  const uint32_t n = (uint32_t)(p.cols + 63) / 64;
  mx_col<MxIn, SR, RHT>(p, b % n, b / n, reinterpret_cast<uint16_t (*)[64]>(tile), sb);
}

// ---- values ----------------------------------------------------------------------
// 8 elements (one code word) a thread; rows of the output are `len` elements.  Bound by
// memory: 16384 x 4096 to bf16 in 25 us, 6.7 TB/s.
template <bool F32>
__global__ __launch_bounds__(256) void mx_values_kernel(const uint8_t* codes, const uint8_t* scale, int64_t rows, int32_t len,
                                                        int32_t nb, void* out) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int32_t per = (len + 7) / 8;
  const int64_t row = id / per;
  if (row >= rows) return;
  const int32_t c = (int32_t)(id - row * per) * 8;
  const uint32_t q = *reinterpret_cast<const uint32_t*>(codes + row * nb * 64 + c / 2);
  const float s = mx_scale(scale[row * nb * 4 + c / 32]);
  float v[8];
  static_for<4>([&](auto k) __attribute__((always_inline)) {
    constexpr int b = decltype(k)::value;
    const f32x2v_t f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, b);
    v[2 * b] = f.x * s;
    v[2 * b + 1] = f.y * s;
  });
  const int64_t at = row * len + c;
  if constexpr (F32) {
    float* o = reinterpret_cast<float*>(out) + at;
    if (!(len & 3) && c + 8 <= len) {
      reinterpret_cast<float4*>(o)[0] = float4{v[0], v[1], v[2], v[3]};
      reinterpret_cast<float4*>(o)[1] = float4{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < len) o[i] = v[i];
    }
  } else {
    uint16_t* o = reinterpret_cast<uint16_t*>(out) + at;
    if (!(len & 7)) {
      *reinterpret_cast<uint4*>(o) = uint4{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < len) o[i] = (uint16_t)bf16_pair(v[i], 0.0f);
    }
  }
}

// ---- product ---------------------------------------------------------------------
struct MxGemmArgs {
  TileOp P, Q;        // P: B [J, K] (columns of C), Q: A [I, K] (rows of C)
  void* C;            // split: fp32 partial sums [splits][I][J], joined by mx_join_kernel
  int64_t ldc, zstride;
  const float* partial;
  uint32_t tiles_p, tiles_q;
  int32_t nch, splits;
  int32_t bf16, accumulate, vec;  // vec: rows of C may be stored 16 bytes at a time
};

// N (a multiple of 4) neighbouring results from column j on of the row that starts
// at element `row` of C
template <int N>
__device__ __forceinline__ void store_run(const MxGemmArgs& p, int64_t row, int64_t j, const float (&v)[N]) {
  const int64_t J = p.P.rows;
  if (j >= J) return;
  const bool whole = p.vec && j + N <= J;
  if (p.bf16) {
    uint16_t* o = reinterpret_cast<uint16_t*>(p.C) + row + j;
    if (whole && N == 4) {
      *reinterpret_cast<uint2*>(o) = uint2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    } else if (whole) {
#pragma unroll
      for (int k = 0; k + 8 <= N; k += 8)
        *reinterpret_cast<uint4*>(o + k) = uint4{bf16_pair(v[k], v[k + 1]), bf16_pair(v[k + 2], v[k + 3]),
                                                bf16_pair(v[k + 4], v[k + 5]), bf16_pair(v[k + 6], v[k + 7])};
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

// One product or two.  C = sum over groups of 2^(ea + eb) sum qa qb, the scales applied
// by the instruction.  4096 x 4096 over 16384 in 154 us, 3.6 PFLOP/s (4.6 on operands of
// zeros: with others the GPU's power bounds it, and the loads' way through L2 and LDS);
// 16384 x 4096 over 1024 in 56, of which the 134 MB of results alone take 26.
template <class T>
__global__ __launch_bounds__(T::NT, T::WAVES) void mx_gemm_kernel(Pair<MxGemmArgs> jobs) {
  __shared__ __attribute__((aligned(128))) typename T::Smem sm;
  const Share mine(jobs.first);
  const MxGemmArgs& p = jobs.x[mine.job];
  const typename T::Items items(p.tiles_p, p.tiles_q, (uint32_t)p.nch, (uint32_t)p.splits, mine.block, mine.blocks);
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
          store_run<4 * T::PB>(p, at + i * p.ldc, pw + tb * 16 * T::PB, v);
        }
      }
    }
  });
}

// Up to 16 rows of A (decoding): A whole in LDS, B read once.  From bf16 X (the
// linear layer's forward) each workgroup quantizes X for itself, the first one
// storing the codes too, which saves the launch that would do it.  1 x 1024 to 4096 in
// 4.5 us, which is a launch, the quantization and one round of loads.
struct MxFewArgs {
  MxGemmArgs g;
  const uint16_t* x;  // quantize [I, cols] bf16 into g.Q's arrays; NULL: they are given
  int32_t cols;
  uint8_t* codes;
  uint8_t* scale;
};
template <class S>
__global__ __launch_bounds__(S::NT, 2) void mx_few_kernel(MxFewArgs a) {
  __shared__ typename S::Smem sm;
  const MxGemmArgs& p = a.g;
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4, I = (int)p.Q.rows;
  const int px = S::pitch(p.P.kb), ps = S::scale_pitch(p.P.kb);
  const int chunks = (p.P.kb + 127) / 128, halves = chunks * 16;  // 16-element pieces of a row, whole chunks
  for (int i = threadIdx.x; i < S::TOKENS * halves; i += S::NT) {
    const int t = i / halves, h = i - t * halves;
    uint2 q = {0u, 0u};
    uint32_t byte = 0u;
    if (a.x) {
      float v[16];
      if (t < I && h * 16 < a.cols) {
        load16<uint16_t>(a.x + (int64_t)t * a.cols + h * 16, v);
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = 0.0f;
      }
      uint32_t top = top_bits16(v);
      top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0xB1, 0xF, 0xF, false));
      byte = mx_scale_byte<false>(top);
      q = mx_codes16<false>(v, byte, 0, 0, 0);
      if (h * 16 >= a.cols) q = uint2{0u, 0u};
      if (blockIdx.x == 0 && t < I && h * 8 < p.P.kb) {
        *reinterpret_cast<uint2*>(a.codes + (int64_t)t * p.P.kb + h * 8) = q;
        if (!(h & 1)) a.scale[(int64_t)t * (p.P.kb / 16) + h / 2] = (uint8_t)byte;
      }
    } else if (t < I && h * 8 < p.P.kb) {
      q = *reinterpret_cast<const uint2*>(p.Q.p + (int64_t)t * p.P.kb + h * 8);
      byte = p.Q.s[(int64_t)t * (p.P.kb / 16) + h / 2];
    }
    *reinterpret_cast<uint2*>(sm.x + t * px + h * 8) = q;
    if (!(h & 1)) sm.xs[t * ps + h / 2] = (uint8_t)byte;
  }
  __syncthreads();
  S::run(p.P, sm, [&](uint32_t group, const typename S::Acc& acc) __attribute__((always_inline)) {
    static_assert(S::TOKENS == 16, "one tile of tokens");
    if (n < I) {
      const float v[4] = {acc[0].x, acc[0].y, acc[0].z, acc[0].w};
      store_run<4>(p, (int64_t)n * p.ldc, (int64_t)group * 16 + g * 4, v);
    }
  });
}

// C = (C +) the sum of the splits' results in order, 4 a thread; of one product or two.
// Bound by memory (or, most often, the last cache): two splits of 4096 x 1024 in 10 us.
__global__ __launch_bounds__(256) void mx_join_kernel(Pair<MxGemmArgs> jobs) {
  const Share mine(jobs.first);
  const MxGemmArgs& p = jobs.x[mine.job];
  const int64_t I = p.Q.rows, J = p.P.rows, n = I * J, per = (J + 3) / 4;
  const int64_t id = (int64_t)mine.block * 256 + threadIdx.x, i = id / per, j = (id - i * per) * 4;
  if (i >= I) return;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const float* s = p.partial + i * J + j;
  if ((J & 3) == 0) {
    for (int z = 0; z < p.splits; ++z, s += n) {
      const float4 a = *reinterpret_cast<const float4*>(s);
      v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
    }
  } else {
    for (int z = 0; z < p.splits; ++z, s += n)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (j + k < J) v[k] += s[k];
  }
  store_run<4>(p, i * p.ldc, j, v);
}

using TileBig = Tile<EL_MX, 2, 4, 8, 4>;    // 256 x 256
using TileMid = Tile<EL_MX, 2, 2, 4, 4>;    // 128 x 128
using TileSmall = Tile<EL_MX, 2, 2, 2, 2>;  // 64 x 64

template <class T>
uint32_t tile_grid(MxGemmArgs& a) {
  a.tiles_p = (uint32_t)((a.P.rows + T::BM - 1) / T::BM);
  a.tiles_q = (uint32_t)((a.Q.rows + T::BN - 1) / T::BN);
  return T::grid((uint64_t)a.tiles_p * a.tiles_q * (uint32_t)a.splits);
}
template <class T>
void launch_tile(const MxGemmArgs& a, const MxGemmArgs* second, hipStream_t s) {
  Pair<MxGemmArgs> jobs = {{a, second ? *second : a}, 0};
  jobs.first = tile_grid<T>(jobs.x[0]);
  const uint32_t others = second ? tile_grid<T>(jobs.x[1]) : 0;
  mx_gemm_kernel<T><<<jobs.first + others, T::NT, 0, s>>>(jobs);
}

TileOp mx_operand(const QView& q, bool blocked) {
  TileOp o = {};
  o.p = q.codes;
  o.s = q.s16;
  o.rows = q.rows;
  const MxOut at = mx_out(q, blocked);
  o.ld = at.ld;
  o.bs = at.bs;
  o.cs = (int32_t)at.cs;
  o.kb = (int32_t)(q.nb * 64);
  return o;
}

// Rows of A that mx_few_kernel takes: one instruction tile (with more, the 64 x 64
// tiles are as fast: 24 x 50304 over 1024 11.8 us here and 9.8 there, 64 x 4096 9.2 and
// 5.3), over up to 2048 elements, whose codes fit this LDS.  Beyond, every workgroup's
// quantization of all of A and a wave's way through whole rows of B take longer than
// tiles, which split the reduction.  Linear forward of 1 row here and in tiles with the
// quantization's launch, N 4096: over 256 3.5 and 5.5 us, 1024 4.9 and 6.7, 2048 7.8 and
// 8.7, 3968 13.0 and 10.0, 7936 24.4 and 12.0; N 50304: 1024 9.4 and 10.1, 2048 17.3 and
// 15.0, 3968 28.9 and 24.1.  16 rows, N 4096: 1024 5.7 and 7.4, 2048 9.7 and 9.7.
using Few = Skinny<EL_MX, 1, 17 * 1024>;
static_assert(Few::TOKENS * (2048 / 2 + 16) <= 17 * 1024 && Few::TOKENS * (2048 / 2 + 128 + 16) > 17 * 1024, "2048 elements");

// Tile and splits of a product, by an estimate of its time from what the tiles
// measure (us on MI355X; a chunk is 256 elements of the reduction): alone on its CU
// a tile of 64 / 128 / 256 takes 0.6 / 1.15 / 2.3 a chunk, with the CU full (4 / 2 / 1
// workgroups) 1.3 / 1.6 / 2.3, and 2 to 5 for its start and its results.  A split
// costs a launch and its fp32 partial sums, written and read.  Of 4096 x 1024
// results over 4096: 23.6, 20.8, 36.5 unsplit; over 16384: 79.8, 68.7 unsplit, 65.0
// (128, two splits); of 256 x 4096 over 4096: 11.3 (64), 18.1, 30.7.
struct MxPlan {
  int tile, splits;
  double time, packed;  // packed: where other tiles take the places that it leaves idle
};
MxPlan mx_plan(int64_t I, int64_t J, int64_t K, int tile) {
  constexpr double kAlone[3] = {0.6, 1.15, 2.3}, kFull[3] = {1.3, 1.6, 2.3}, kFixed[3] = {2.0, 2.5, 5.0};
  constexpr int kSlots[3] = {4, 2, 1};
  const int64_t nch = (K + 255) / 256;
  const int64_t b = 64 << tile, n = ((I + b - 1) / b) * ((J + b - 1) / b), slots = kCus * kSlots[tile];
  MxPlan best = {tile, 1, 1e30, 1e30};
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
      best = MxPlan{tile, z, t + join, (double)items * (chunks * kFull[tile] + kFixed[tile]) / (double)slots + join};
  }
  return best;
}
MxPlan mx_plan(int64_t I, int64_t J, int64_t K) {
  MxPlan best = mx_plan(I, J, K, 0);
  for (int tile = 1; tile < 3; ++tile)
    if (const MxPlan p = mx_plan(I, J, K, tile); p.time < best.time) best = p;
  return best;
}
// Two products that do not depend on each other: of one tile they run in one launch,
// the second in the places that the first leaves idle (backward of 16384 x 1024 over
// 1024: 85 us with tiles of 256 and 128 in two launches, 79 with 128 for both).
struct MxPlans {
  MxPlan a, b;
};
MxPlans mx_plans(int64_t I, int64_t J, int64_t K, int64_t I2, int64_t J2, int64_t K2) {
  MxPlans best = {mx_plan(I, J, K), mx_plan(I2, J2, K2)};
  double least = best.a.time + best.b.time;
  for (int tile = 0; tile < 3; ++tile) {
    const MxPlans c = {mx_plan(I, J, K, tile), mx_plan(I2, J2, K2, tile)};
    const double t = std::max({c.a.packed + c.b.packed, c.a.time, c.b.time});
    if (t < least) {
      least = t;
      best = c;
    }
  }
  return best;
}

}  // namespace

bool mx_is_few(int64_t M, int64_t K) { return Few::fits(M, (K + 127) / 128 * 64); }

bool mx_blocked(int64_t I, int64_t K) { return !mx_is_few(I, K); }

namespace {
size_t split_bytes(int z, int64_t I, int64_t J) { return z > 1 ? (size_t)z * (size_t)I * (size_t)J * 4 : 0; }
}  // namespace

size_t mx_gemm_workspace_bytes(int64_t I, int64_t J, int64_t K) {
  return mx_is_few(I, K) ? 0 : split_bytes(mx_plan(I, J, K).splits, I, J);
}

namespace {
// The product of few rows; x: quantize them first, into `q`.
hipError_t launch_few(const MxGemmArgs& a, const void* x, int64_t cols, const QView* q, hipStream_t s) {
  MxFewArgs f = {};
  f.g = a;
  f.x = reinterpret_cast<const uint16_t*>(x);
  f.cols = (int32_t)cols;
  if (q) {
    f.codes = q->codes;
    f.scale = q->s16;
  }
  mx_few_kernel<Few><<<Few::grid(a.P.rows), Few::NT, 0, s>>>(f);
  return hipGetLastError();
}

MxGemmArgs mx_gemm_args(const QView& A, const QView& B, void* C, int c_dtype, int64_t ldc, int accumulate, bool blocked = false) {
  MxGemmArgs a = {};
  a.P = mx_operand(B, blocked);
  a.Q = mx_operand(A, blocked);
  a.C = C;
  a.ldc = ldc;
  a.nch = (int32_t)((A.nb + 1) / 2);
  a.splits = 1;
  a.bf16 = c_dtype == TJ2_BF16;
  a.accumulate = accumulate;
  const int64_t es = a.bf16 ? 2 : 4;
  a.vec = (reinterpret_cast<uintptr_t>(C) & 15u) == 0 && (ldc * es) % 16 == 0;
  return a;
}
}  // namespace

hipError_t launch_mx_linear_few(const void* X, const QView& Xq, const QView& Wq, void* Y, int y_dtype, hipStream_t s) {
  return launch_few(mx_gemm_args(Xq, Wq, Y, y_dtype, Wq.rows, 0), X, Xq.len, &Xq, s);
}

namespace {
// A planned product; split: `part` is what the tiles write, joined into `out`.
struct MxProduct {
  MxGemmArgs part, out;
  int tile;
};
MxProduct mx_product(const MxGemmArgs& a, const MxPlan& plan, float* partial) {
  MxProduct x = {a, a, plan.tile};
  x.part.splits = x.out.splits = partial ? plan.splits : 1;
  x.out.partial = partial;
  if (x.out.splits > 1) {
    x.part.C = partial;
    x.part.ldc = a.P.rows;
    x.part.zstride = a.Q.rows * a.P.rows;
    x.part.bf16 = 0;
    x.part.accumulate = 0;
    x.part.vec = (a.P.rows & 3) == 0;
  }
  return x;
}
// One product, or two of one tile.
hipError_t launch_products(const MxProduct* x, int n, hipStream_t s) {
  const MxGemmArgs* second = n > 1 ? &x[1].part : nullptr;
  if (x[0].tile == 2) launch_tile<TileBig>(x[0].part, second, s);
  else if (x[0].tile == 1) launch_tile<TileMid>(x[0].part, second, s);
  else launch_tile<TileSmall>(x[0].part, second, s);
  return hipGetLastError();
}
// The joins of those that are split.
hipError_t launch_joins(const MxProduct* x, int n, hipStream_t s) {
  Pair<MxGemmArgs> jobs = {};
  uint32_t grid[2] = {0, 0};
  int k = 0;
  for (int i = 0; i < n; ++i) {
    if (x[i].out.splits == 1) continue;
    jobs.x[k] = x[i].out;
    grid[k] = (uint32_t)((x[i].out.Q.rows * ((x[i].out.P.rows + 3) / 4) + 255) / 256);
    ++k;
  }
  if (!k) return hipSuccess;
  jobs.first = grid[0];
  mx_join_kernel<<<grid[0] + grid[1], 256, 0, s>>>(jobs);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_mx_gemm(const QView& A, const QView& B, void* C, int c_dtype, int64_t ldc, int accumulate, float* partial,
                          hipStream_t s) {
  const MxGemmArgs a = mx_gemm_args(A, B, C, c_dtype, ldc, accumulate);
  if (mx_is_few(A.rows, A.len)) return launch_few(a, nullptr, 0, nullptr, s);
  const MxProduct x = mx_product(a, mx_plan(A.rows, B.rows, A.len), partial);
  if (hipError_t e = launch_products(&x, 1, s); e != hipSuccess) return e;
  return launch_joins(&x, 1, s);
}

namespace {
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
// the plans of a pair, of which either may be a product of few rows instead
MxPlans pair_plans(int64_t I, int64_t J, int64_t K, int64_t I2, int64_t J2, int64_t K2) {
  if (mx_is_few(I, K) || mx_is_few(I2, K2)) return MxPlans{mx_plan(I, J, K), mx_plan(I2, J2, K2)};
  return mx_plans(I, J, K, I2, J2, K2);
}
}  // namespace

size_t mx_gemm_pair_workspace_bytes(int64_t I, int64_t J, int64_t K, int64_t I2, int64_t J2, int64_t K2) {
  const MxPlans plans = pair_plans(I, J, K, I2, J2, K2);
  return up256(mx_is_few(I, K) ? 0 : split_bytes(plans.a.splits, I, J)) + (mx_is_few(I2, K2) ? 0 : split_bytes(plans.b.splits, I2, J2));
}

hipError_t launch_mx_gemm_pair(const QView& A, const QView& B, void* C, int c_dtype, const QView& A2, const QView& B2, void* C2,
                               int c2_dtype, float* partial, hipStream_t s) {
  const MxGemmArgs a[2] = {mx_gemm_args(A, B, C, c_dtype, B.rows, 0, mx_blocked(A.rows, A.len)),
                           mx_gemm_args(A2, B2, C2, c2_dtype, B2.rows, 0, mx_blocked(A2.rows, A2.len))};
  const MxPlans plans = pair_plans(A.rows, B.rows, A.len, A2.rows, B2.rows, A2.len);
  const bool few[2] = {mx_is_few(A.rows, A.len), mx_is_few(A2.rows, A2.len)};
  const size_t first = up256(few[0] ? 0 : split_bytes(plans.a.splits, A.rows, B.rows));
  MxProduct x[2];
  int n = 0;
  for (int i = 0; i < 2; ++i) {
    if (few[i]) {
      if (hipError_t e = launch_few(a[i], nullptr, 0, nullptr, s); e != hipSuccess) return e;
    } else {
      x[n++] = mx_product(a[i], i ? plans.b : plans.a, i ? partial + first / 4 : partial);
    }
  }
  for (int i = 0; i < n;) {
    const int k = i + 1 < n && x[i].tile == x[i + 1].tile ? 2 : 1;
    if (hipError_t e = launch_products(x + i, k, s); e != hipSuccess) return e;
    i += k;
  }
  return launch_joins(x, n, s);
}

hipError_t launch_mx_values(const QView& q, void* out, int dtype, hipStream_t s) {
  const int64_t n = q.rows * ((q.len + 7) / 8);
  const uint32_t grid = (uint32_t)((n + 255) / 256);
  if (dtype == TJ2_F32) mx_values_kernel<true><<<grid, 256, 0, s>>>(q.codes, q.s16, q.rows, (int32_t)q.len, (int32_t)q.nb, out);
  else mx_values_kernel<false><<<grid, 256, 0, s>>>(q.codes, q.s16, q.rows, (int32_t)q.len, (int32_t)q.nb, out);
  return hipGetLastError();
}

namespace {
template <class T>
hipError_t launch_row(const MxRowArgs& a, bool sr, bool rht, uint32_t grid, hipStream_t s) {
  if (sr) {
    if (rht) mx_row_kernel<T, true, true><<<grid, 256, 0, s>>>(a);
    else mx_row_kernel<T, true, false><<<grid, 256, 0, s>>>(a);
  } else {
    if (rht) mx_row_kernel<T, false, true><<<grid, 256, 0, s>>>(a);
    else mx_row_kernel<T, false, false><<<grid, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}
template <class T>
hipError_t launch_col(const MxColArgs& a, bool sr, bool rht, dim3 grid, hipStream_t s) {
  if (sr) {
    if (rht) mx_col_kernel<T, true, true><<<grid, 256, 0, s>>>(a);
    else mx_col_kernel<T, true, false><<<grid, 256, 0, s>>>(a);
  } else {
    if (rht) mx_col_kernel<T, false, true><<<grid, 256, 0, s>>>(a);
    else mx_col_kernel<T, false, false><<<grid, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}
}  // namespace

namespace {
MxRowArgs row_args(const MxQuantParams& q) {
  MxRowArgs a = {};
  a.x = q.x;
  a.codes = q.out.codes;
  a.scale = q.out.s16;
  a.rows = q.rows;
  a.cols = (int32_t)q.cols;
  a.nb = (int32_t)q.out.nb;
  a.mask = q.rht_mask;
  a.seed = q.seed;
  a.offset = q.offset;
  return a;
}
uint32_t row_grid(const MxRowArgs& a) { return (uint32_t)((a.rows * a.nb * 8 + 255) / 256); }
MxColArgs col_args(const MxQuantParams& q) {
  MxColArgs a = {};
  a.x = q.x;
  a.ldx = q.cols;
  if (q.in_dtype == TJ2_MXFP4) {
    a.x = q.xq.codes;
    a.xs = q.xq.s16;
    a.ldx = q.xq.nb * 64;
    a.lds = q.xq.nb * 4;
  }
  a.out = mx_out(q.out, q.blocked);
  a.rows = (int32_t)q.rows;
  a.cols = (int32_t)q.cols;
  a.nb = (int32_t)q.out.nb;
  a.mask = q.rht_mask;
  a.seed = q.seed;
  a.offset = q.offset;
  return a;
}
dim3 col_grid(const MxColArgs& a) { return dim3((uint32_t)(a.cols + 63) / 64, (uint32_t)a.nb); }
}  // namespace

hipError_t launch_mx_quant(const MxQuantParams& q, hipStream_t s) {
  const bool sr = q.rounding == TJ2_SR;
  if (q.grouping == TJ2_GROUP_ROW) {
    const MxRowArgs a = row_args(q);
    const uint32_t grid = row_grid(a);
    return q.in_dtype == TJ2_BF16 ? launch_row<uint16_t>(a, sr, q.rht, grid, s) : launch_row<float>(a, sr, q.rht, grid, s);
  }
  const MxColArgs a = col_args(q);
  const dim3 grid = col_grid(a);
  if (q.in_dtype == TJ2_MXFP4) return launch_col<MxIn>(a, sr, q.rht, grid, s);
  return q.in_dtype == TJ2_BF16 ? launch_col<uint16_t>(a, sr, q.rht, grid, s) : launch_col<float>(a, sr, q.rht, grid, s);
}

hipError_t launch_mx_forward_operands(const MxQuantParams& x, const MxQuantParams& w, hipStream_t s) {
  const MxRowArgs a = row_args(x), b = row_args(w);
  mx_row_pair_kernel<<<row_grid(a) + row_grid(b), 256, 0, s>>>(a, b, row_grid(a));
  return hipGetLastError();
}

hipError_t launch_mx_backward_operands(const MxQuantParams& dy_row, const MxQuantParams& dy_col, const MxQuantParams& w,
                                       const MxQuantParams& x, hipStream_t s) {
  MxDualArgs d = {};
  d.x = reinterpret_cast<const uint16_t*>(dy_row.x);
  d.row = mx_out(dy_row.out, dy_row.blocked);
  d.col = mx_out(dy_col.out, dy_col.blocked);
  d.rows = (int32_t)dy_row.rows;
  d.cols = (int32_t)dy_row.cols;
  d.nbr = (int32_t)dy_col.out.nb;
  d.nbc = (int32_t)dy_row.out.nb;
  d.row_mask = dy_row.rht_mask;
  d.col_mask = dy_col.rht_mask;
  d.seed = dy_row.seed;
  d.row_offset = dy_row.offset;
  d.col_offset = dy_col.offset;
  const dim3 gw = col_grid(col_args(w)), gx = col_grid(col_args(x));
  const Pair<MxColArgs> codes = {{col_args(w), col_args(x)}, gw.x * gw.y};
  const uint32_t nd = (uint32_t)d.nbc * (uint32_t)d.nbr, grid = nd + codes.first + gx.x * gx.y;
  if (dy_row.rounding == TJ2_SR) {
    if (dy_row.rht) mx_backward_kernel<true, true><<<grid, 256, 0, s>>>(d, nd, codes);
    else mx_backward_kernel<true, false><<<grid, 256, 0, s>>>(d, nd, codes);
  } else {
    if (dy_row.rht) mx_backward_kernel<false, true><<<grid, 256, 0, s>>>(d, nd, codes);
    else mx_backward_kernel<false, false><<<grid, 256, 0, s>>>(d, nd, codes);
  }
  return hipGetLastError();
}

}  // namespace tj2
