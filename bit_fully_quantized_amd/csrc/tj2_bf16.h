// bf16 operands, tiles and plans of the products in the head's cross entropy (loss.hip)
// and the gated feed-forward block (ffn.hip).
#pragma once
#include <algorithm>

#include "tj2_skinny.h"

namespace tj2 {
namespace {

// A bf16 matrix [rows, cols] (cols a multiple of 16) into blocked operands: `copy`
// [rows, cols] and `turned` [cols, rows], zero up to whole chunks; either may be
// NULL.  64 x 64 through LDS.  Rows of ignored tokens (y, if not NULL) become zero:
// their dz is, but an infinity or NaN in them times zero would not be.
struct BlockArgs {
  const uint16_t* in;
  int64_t rows, cols, ld;
  uint16_t *copy, *turned;
  uint32_t nr, nc;  // chunks of rows and of columns
  uint32_t pitch;   // chunks of a row of `turned` (nr, or more where it is part of a longer operand)
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
    *reinterpret_cast<uint4*>(p.turned + ((c0 >> 7) * p.pitch + br) * 8192 + ((c0 & 127) + c) * 64 + r) = uint4{v[0], v[1], v[2], v[3]};
  }
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

// Tokens from which the operands of a product over the features are copied into blocks first.
constexpr int64_t kBlockTokens = 2048;

BlockArgs block_args(const void* in, int64_t rows, int64_t cols, int64_t ld, void* copy, void* turned) {
  return BlockArgs{reinterpret_cast<const uint16_t*>(in), rows,
                   cols, ld, reinterpret_cast<uint16_t*>(copy),
                   reinterpret_cast<uint16_t*>(turned), (uint32_t)((rows + 63) / 64), (uint32_t)((cols + 63) / 64), (uint32_t)((rows + 63) / 64), nullptr, 0};
}

int64_t tiles_of(int64_t p, int64_t q, int64_t b) { return (p + b - 1) / b * ((q + b - 1) / b); }

// Estimated time (us on MI355X) of `items` tiles over `chunks` chunks of 64 elements:
// a tile of 256 takes 1.9 a chunk and `fixed` for its start and results, one of 128
// 1.1 alone on its CU and 1.5 beside another, and half of `fixed`.
double tile_time(bool big, int64_t items, double chunks, double fixed) {
  if (big) return (double)((items + kCus - 1) / kCus) * (chunks * 1.9 + fixed);
  const int64_t full = items / (2 * kCus), rest = items % (2 * kCus);
  return (double)full * (chunks * 1.5 + fixed / 2) + (rest ? chunks * (rest > kCus ? 1.5 : 1.1) + fixed / 2 : 0.0);
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
}  // namespace
}  // namespace tj2
