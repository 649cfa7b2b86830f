// Root-mean-square norm with the residual's addition for gfx950:
//
//   s = x + residual (rounded to the stream's type, the new residual stream),
//   r = 1 / sqrt(mean(s^2) + eps),   y = (s r) w,
//
// y in the stream's type or as E4M3 under amax / 448 per 128 elements of a row (an FP8
// linear's operand, which then is never written in 16 bits), and its backward pass
//
//   ds = r (dy w - s r mean(dy w s r)) + dsum,   dw = sum over the rows of dy s r.
//
// Both are bound by memory: a row is read once, kept in registers as fp32 between the sum
// and its use, and written once.  The statistics, the products and dw's sums are fp32.
#include <algorithm>

#include "tj2_fp8.h"
#include "tj2_internal.h"
#include "tj2_tile.h"

namespace tj2 {
namespace {

struct NormArgs {
  const void *x, *res;
  int64_t ldx, ldr;
  void *sum, *y;        // dense; y NULL: FP8
  const void* w;
  float* rstd;
  uint8_t* codes;       // [rows][nb * 128]
  float* scale;         // [rows][nb]
  int64_t rows;
  int32_t cols, nb, w_bf16;
  float eps;
};

struct NormGradArgs {
  const void *dy, *s, *dsum;
  int64_t lddy, lds, ldd;
  const void* w;
  const float* rstd;
  void* ds;
  float* part;          // [workgroups][cols], NULL: dw is not asked for
  int64_t rows;
  int32_t cols, w_bf16;
};

// How a row's elements are dealt out over its threads, 8 and 8 or one and one:
//   Whole   vectors of 8 neighbours, 16-byte accesses at any element's address
//   Tail    the same where a row's last vector is part of one (bf16): its thread loads the
//           row's last 8 elements and shifts them, without a branch, so that the loads of
//           all vectors and tensors are on their way together
//   Single  single elements (fp32 rows that are no multiple of 8)
// Forward and backward with the residual's, in us: 16384 x 1023 bf16 25 and 42 as Tail, 32
// and 42 where a branch loads the last vector's elements, 33 and 68 in pairs, 56 and 70 as
// Single (16384 x 1024: 22 and 28); 1555 x 1003 fp32 5.7 and 10.3 as Single, 7.3 and 12.1 as Tail.
// What Tail still costs: 16-byte accesses at odd elements, several of the L1 each (backward of
// 16384 x 1023: 3.3 times the L1 accesses of 1024 columns for the same bytes of memory), and 1.7
// times the vector instructions.
enum class Deal { Whole, Tail, Single };

template <int TPR, Deal D>
struct Row {
  typedef uint32_t Words __attribute__((ext_vector_type(4), aligned(2)));
  typedef float Floats __attribute__((ext_vector_type(4), aligned(4)));
  static __device__ __forceinline__ int at(int v, int e, int t) { return D == Deal::Single ? (v * 8 + e) * TPR + t : (v * TPR + t) * 8 + e; }
  static __device__ __forceinline__ float get(const float* p) { return *p; }
  static __device__ __forceinline__ float get(const uint16_t* p) { return bf16_to_f32(*p); }
  static __device__ __forceinline__ void get8(const float* p, float out[8]) {
    const Floats a = *reinterpret_cast<const Floats*>(p), b = *reinterpret_cast<const Floats*>(p + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      out[e] = a[e];
      out[4 + e] = b[e];
    }
  }
  static __device__ __forceinline__ void get8(const uint16_t* p, float out[8]) {
    const Words u = *reinterpret_cast<const Words*>(p);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      out[2 * e] = __uint_as_float(u[e] << 16);
      out[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void put(float* p, float v) { *p = v; }
  static __device__ __forceinline__ void put(uint16_t* p, float v) { *p = (uint16_t)bf16_pair(v, 0.0f); }
  static __device__ __forceinline__ void put8(float* p, const float in[8]) {
    *reinterpret_cast<Floats*>(p) = Floats{in[0], in[1], in[2], in[3]};
    *reinterpret_cast<Floats*>(p + 4) = Floats{in[4], in[5], in[6], in[7]};
  }
  static __device__ __forceinline__ void put8(uint16_t* p, const float in[8]) {
    *reinterpret_cast<Words*>(p) = Words{bf16_pair(in[0], in[1]), bf16_pair(in[2], in[3]), bf16_pair(in[4], in[5]), bf16_pair(in[6], in[7])};
  }
  // vector v of a row, zeros past its end
  template <class T>
  static __device__ __forceinline__ void load(const T* p, int v, int t, int cols, float out[8]) {
    const int c = at(v, 0, t);
    if constexpr (D == Deal::Whole) {
      if (c < cols) {
        get8(p + c, out);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) out[e] = 0.0f;
      }
      return;
    }
    if (D == Deal::Single || cols < 8) {
#pragma unroll
      for (int e = 0; e < 8; ++e) out[e] = at(v, e, t) < cols ? get(p + at(v, e, t)) : 0.0f;
      return;
    }
    const int past = max(c + 8 - cols, 0);
    get8(p + (c - past), out);
#pragma unroll
    for (int o = 1; o < 8; o *= 2)
#pragma unroll
      for (int e = 0; e < 8; ++e) out[e] = past & o ? (e + o < 8 ? out[e + o] : 0.0f) : out[e];
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = past < 8 ? out[e] : 0.0f;
  }
  static __device__ __forceinline__ void weight(const void* w, int bf16, int v, int t, int cols, float out[8]) {
    if (bf16) load(reinterpret_cast<const uint16_t*>(w), v, t, cols, out);
    else load(reinterpret_cast<const float*>(w), v, t, cols, out);
  }
  template <class T>
  static __device__ __forceinline__ void store(T* p, int v, int t, int cols, const float in[8]) {
    const int c = at(v, 0, t);
    if (D != Deal::Single && c + 8 <= cols) {
      put8(p + c, in);
    } else if constexpr (D != Deal::Whole) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at(v, e, t) < cols) put(p + at(v, e, t), in[e]);
    }
  }
};

// in[] rounded to T and back
template <class T>
__device__ __forceinline__ void as_stored(float v[8]) {
  if constexpr (!std::is_same<T, float>::value) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const uint32_t u = bf16_pair(v[e], v[e + 1]);
      v[e] = __uint_as_float(u << 16);
      v[e + 1] = __uint_as_float(u & 0xFFFF0000u);
    }
  }
}

// Sum over the TPR threads of a row (64: a wave, else the workgroup), the same in all.
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float* sh) {
#pragma unroll
  for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o);
  if constexpr (TPR > 64) {
    __syncthreads();  // the last row's sums have been read
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = x;
    __syncthreads();
    x = sh[0];
#pragma unroll
    for (int k = 1; k < TPR / 64; ++k) x += sh[k];
  }
  return x;
}

// 8 neighbouring elements from column c of a row in FP8; 16 lanes make a group.
__device__ __forceinline__ void store_fp8(const NormArgs& p, int64_t row, int c, const float v[8]) {
  const Fp8Scale s = fp8_scale(max16_lanes(top_bits8(v)));
  if (c >= p.nb * 128) return;
  *reinterpret_cast<uint2*>(p.codes + row * p.nb * 128 + c) = fp8_codes8(v, s);
  if ((c & 127) == 0) p.scale[row * p.nb + (c >> 7)] = s.S;
}

constexpr int kNormThreads = 256;

// Rows whose elements the registers hold, a wave or a workgroup a row.  Bound by memory:
// 16384 x 1024 bf16 with the residual 22 us (134 MB at 6.0 TB/s; a copy reaches 5.1), fp32
// 41 us (6.5 TB/s); with the FP8 result instead of the bf16 one 22 us (117 MB, 5.3 TB/s).
template <class T, int TPR, int NV, Deal D, bool RES, bool FP8>
__global__ __launch_bounds__(kNormThreads) void norm_kernel(NormArgs p) {
  using R = Row<TPR, D>;
  constexpr int RPW = kNormThreads / TPR;
  __shared__ float sh[4];
  const int t = threadIdx.x % TPR;
  float w[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) R::weight(p.w, p.w_bf16, v, t, p.cols, w[v]);
  for (int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / TPR; row < p.rows; row += (int64_t)gridDim.x * RPW) {
    float s[NV][8];
    const T* x = reinterpret_cast<const T*>(p.x) + row * p.ldx;
#pragma unroll
    for (int v = 0; v < NV; ++v) R::load(x, v, t, p.cols, s[v]);
    if constexpr (RES) {
      const T* res = reinterpret_cast<const T*>(p.res) + row * p.ldr;
      float q[NV][8];
#pragma unroll
      for (int v = 0; v < NV; ++v) R::load(res, v, t, p.cols, q[v]);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s[v][e] += q[v][e];
        as_stored<T>(s[v]);
        R::store(reinterpret_cast<T*>(p.sum) + row * p.cols, v, t, p.cols, s[v]);
      }
    }
    float a = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) a = fmaf(s[v][e], s[v][e], a);
    a = row_sum<TPR>(a, sh);
    const float r = 1.0f / sqrtf(a / (float)p.cols + p.eps);
    if (p.rstd && t == 0) p.rstd[row] = r;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int e = 0; e < 8; ++e) s[v][e] = s[v][e] * r * w[v][e];
      if constexpr (FP8) store_fp8(p, row, R::at(v, 0, t), s[v]);
      else R::store(reinterpret_cast<T*>(p.y) + row * p.cols, v, t, p.cols, s[v]);
    }
  }
}

// Longer rows: a workgroup a row, which is read again for its results (1000 x 20000 bf16
// with the residual 31 us, 5.1 TB/s of the first reading and the results: L2 holds the row).
template <class T, Deal D, bool RES, bool FP8>
__global__ __launch_bounds__(kNormThreads) void norm_long_kernel(NormArgs p) {
  using R = Row<kNormThreads, D>;
  __shared__ float sh[4];
  const int t = threadIdx.x, nv = (p.cols + kNormThreads * 8 - 1) / (kNormThreads * 8);
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = reinterpret_cast<const T*>(p.x) + row * p.ldx;
    T* sum = reinterpret_cast<T*>(p.sum) + row * p.cols;
    float a = 0.0f;
    for (int v = 0; v < nv; ++v) {
      float s[8];
      R::load(x, v, t, p.cols, s);
      if constexpr (RES) {
        float q[8];
        R::load(reinterpret_cast<const T*>(p.res) + row * p.ldr, v, t, p.cols, q);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] += q[e];
        as_stored<T>(s);
        R::store(sum, v, t, p.cols, s);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) a = fmaf(s[e], s[e], a);
    }
    a = row_sum<kNormThreads>(a, sh);
    const float r = 1.0f / sqrtf(a / (float)p.cols + p.eps);
    if (p.rstd && t == 0) p.rstd[row] = r;
    for (int v = 0; v < nv; ++v) {
      float s[8], w[8];
      R::load(RES ? sum : x, v, t, p.cols, s);  // (this thread's own stores)
      R::weight(p.w, p.w_bf16, v, t, p.cols, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] = s[e] * r * w[e];
      if constexpr (FP8) store_fp8(p, row, R::at(v, 0, t), s);
      else R::store(reinterpret_cast<T*>(p.y) + row * p.cols, v, t, p.cols, s);
    }
  }
}

// Bound by memory and, from 4 vectors a thread on, by the few waves that run: 16384 x 1024
// bf16 with dsum 24 us (134 MB at 5.6 TB/s) and 4 us for norm_dw_kernel, fp32 47 us.
// A thread keeps its columns' sums of dw over the workgroup's rows; each workgroup writes
// its sums, which norm_dw_kernel adds up in order (no atomics: the same bits every run).
template <class T, int TPR, int NV, Deal D, bool DSUM>
__global__ __launch_bounds__(kNormThreads) void norm_grad_kernel(NormGradArgs p) {
  using R = Row<TPR, D>;
  constexpr int RPW = kNormThreads / TPR;
  __shared__ float sh[4];
  const int t = threadIdx.x % TPR;
  float w[NV][8], dw[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    R::weight(p.w, p.w_bf16, v, t, p.cols, w[v]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[v][e] = 0.0f;
  }
  for (int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / TPR; row < p.rows; row += (int64_t)gridDim.x * RPW) {
    float x[NV][8], g[NV][8], d[DSUM ? NV : 1][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      R::load(reinterpret_cast<const T*>(p.s) + row * p.lds, v, t, p.cols, x[v]);
      R::load(reinterpret_cast<const T*>(p.dy) + row * p.lddy, v, t, p.cols, g[v]);
      if constexpr (DSUM) R::load(reinterpret_cast<const T*>(p.dsum) + row * p.ldd, v, t, p.cols, d[v]);
    }
    const float r = p.rstd[row];
    float a = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[v][e] *= r;
        dw[v][e] = fmaf(g[v][e], x[v][e], dw[v][e]);
        g[v][e] *= w[v][e];
        a = fmaf(g[v][e], x[v][e], a);
      }
    if (p.ds) {
      a = row_sum<TPR>(a, sh) / (float)p.cols;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          g[v][e] = r * fmaf(-x[v][e], a, g[v][e]);
          if constexpr (DSUM) g[v][e] += d[v][e];
        }
        R::store(reinterpret_cast<T*>(p.ds) + row * p.cols, v, t, p.cols, g[v]);
      }
    }
  }
  if (!p.part) return;
  float* part = p.part + (int64_t)blockIdx.x * p.cols;
  if constexpr (TPR == 64) {
    // the waves' sums, in their order
    __shared__ float sums[NV * 8][64];
    for (int q = 0; q < RPW; ++q) {
      if (q == (int)threadIdx.x / 64) {
#pragma unroll
        for (int i = 0; i < NV * 8; ++i) {
          if (q) dw[i / 8][i % 8] += sums[i][t];
          if (q < RPW - 1) sums[i][t] = dw[i / 8][i % 8];
        }
      }
      __syncthreads();
    }
    if (threadIdx.x / 64 != RPW - 1) return;
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) R::store(part, v, t, p.cols, dw[v]);
}

// Longer rows: ds with the row read twice (L2 holds it), and dw's sums over a slab of rows by
// columns, which reads s and dy again, as a lane's columns of dw do not fit its registers (1000
// x 20000 bf16 55 us: ds 37, the slabs 15 for 80 MB, norm_dw_kernel 5).
template <class T, Deal D, bool DSUM>
__global__ __launch_bounds__(kNormThreads) void norm_grad_long_kernel(NormGradArgs p) {
  using R = Row<kNormThreads, D>;
  __shared__ float sh[4];
  const int t = threadIdx.x, nv = (p.cols + kNormThreads * 8 - 1) / (kNormThreads * 8);
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T *s = reinterpret_cast<const T*>(p.s) + row * p.lds, *dy = reinterpret_cast<const T*>(p.dy) + row * p.lddy;
    const float r = p.rstd[row];
    float a = 0.0f, x[8], g[8], w[8];
    auto fetch = [&](int v) __attribute__((always_inline)) {
      R::load(s, v, t, p.cols, x);
      R::load(dy, v, t, p.cols, g);
      R::weight(p.w, p.w_bf16, v, t, p.cols, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] *= r;
        g[e] *= w[e];
      }
    };
    for (int v = 0; v < nv; ++v) {
      fetch(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) a = fmaf(g[e], x[e], a);
    }
    a = row_sum<kNormThreads>(a, sh) / (float)p.cols;
    for (int v = 0; v < nv; ++v) {
      fetch(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = r * fmaf(-x[e], a, g[e]);
      if constexpr (DSUM) {
        float d[8];
        R::load(reinterpret_cast<const T*>(p.dsum) + row * p.ldd, v, t, p.cols, d);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] += d[e];
      }
      R::store(reinterpret_cast<T*>(p.ds) + row * p.cols, v, t, p.cols, g);
    }
  }
}

// dw's sums over rows [slab y, slab y + 1) of 256 columns
template <class T>
__global__ __launch_bounds__(kNormThreads) void norm_grad_slab_kernel(NormGradArgs p, int64_t slab) {
  const int64_t c = (int64_t)blockIdx.x * kNormThreads + threadIdx.x;
  if (c >= p.cols) return;
  const int64_t first = (int64_t)blockIdx.y * slab, last = min(first + slab, p.rows);
  float a = 0.0f;
#pragma unroll 4
  for (int64_t row = first; row < last; ++row) {
    float s, g;
    if constexpr (std::is_same<T, float>::value) {
      s = reinterpret_cast<const T*>(p.s)[row * p.lds + c];
      g = reinterpret_cast<const T*>(p.dy)[row * p.lddy + c];
    } else {
      s = bf16_to_f32(reinterpret_cast<const T*>(p.s)[row * p.lds + c]);
      g = bf16_to_f32(reinterpret_cast<const T*>(p.dy)[row * p.lddy + c]);
    }
    a = fmaf(g, s * p.rstd[row], a);
  }
  p.part[(int64_t)blockIdx.y * p.cols + c] = a;
}

// dw = the workgroups' sums in order: 32 columns a workgroup, 32 threads a column.
__global__ __launch_bounds__(1024) void norm_dw_kernel(const float* part, int parts, int64_t cols, void* dw, int bf16) {
  __shared__ float sh[32][33];
  const int l = threadIdx.x & 31, q = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + l;
  float a = 0.0f;
  if (c < cols) {
    const int first = (int)((int64_t)parts * q / 32), last = (int)((int64_t)parts * (q + 1) / 32);
#pragma unroll 8
    for (int i = first; i < last; ++i) a += part[(int64_t)i * cols + c];
  }
  sh[q][l] = a;
  __syncthreads();
  if (q || c >= cols) return;
#pragma unroll
  for (int k = 1; k < 32; ++k) a += sh[k][l];
  if (bf16) reinterpret_cast<uint16_t*>(dw)[c] = (uint16_t)bf16_pair(a, 0.0f);
  else reinterpret_cast<float*>(dw)[c] = a;
}

// Columns that registers hold: up to 32 elements a thread, of a wave up to 2048 and of a
// workgroup up to 8192 (dw and w take as many again in the backward pass).
constexpr int64_t kNormWave = 2048, kNormHeld = 8192;

template <bool B>
using Is = std::integral_constant<bool, B>;
template <class F>
void pick(bool b, F&& f) {
  if (b) f(Is<true>{});
  else f(Is<false>{});
}
template <class T, class F>
void pick_deal(int64_t cols, F&& f) {
  constexpr Deal odd = std::is_same<T, float>::value ? Deal::Single : Deal::Tail;
  if (cols % 8 == 0) f(std::integral_constant<Deal, Deal::Whole>{});
  else f(std::integral_constant<Deal, odd>{});
}
// f(threads a row, vectors a thread) for rows of `cols`
template <class F>
void pick_row(int64_t cols, F&& f) {
  if (cols <= 512) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
  else if (cols <= 1024) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
  else if (cols <= kNormWave) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 4>{});
  else if (cols <= 4096) f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
  else f(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{});
}

int64_t norm_rows_per_group(int64_t cols) { return cols <= kNormWave ? 4 : 1; }
// Workgroups of the forward pass: up to 8 a CU, so that a weight is read for several rows.
uint32_t norm_grid(int64_t rows, int64_t cols) {
  const int64_t per = norm_rows_per_group(cols);
  return (uint32_t)std::min<int64_t>((rows + per - 1) / per, 8 * kCus);
}
// Workgroups of the backward pass, each with a row of dw's sums: as many as the registers
// let run at once, 2 a CU with 4 vectors a thread (8192 x 2048 bf16: 31 us, with 4 a CU 35,
// with 1 48; 2048 x 8192: 35, 41 and 46) and else 4 (16384 x 1024: 28 us, with 2 32, with 8
// 32; 4096 x 4096: 31, 34 and 38).
int64_t norm_parts(int64_t rows, int64_t cols) {
  if (cols > kNormHeld) return std::min<int64_t>((rows + 63) / 64, 64);
  const int64_t per = norm_rows_per_group(cols);
  const bool four = (cols > 1024 && cols <= kNormWave) || cols > 4096;
  return std::min<int64_t>((rows + per - 1) / per, (four ? 2 : 4) * kCus);
}

template <class T>
hipError_t run_norm(const NormParams& n, hipStream_t s) {
  NormArgs a = {};
  a.x = n.x;
  a.res = n.residual;
  a.ldx = n.ldx;
  a.ldr = n.ldr;
  a.sum = n.sum;
  a.y = n.y;
  a.w = n.w;
  a.w_bf16 = n.w_dtype == TJ2_BF16;
  a.rstd = n.rstd;
  a.codes = n.yq.codes;
  a.scale = n.yq.s128;
  a.nb = (int32_t)n.yq.nb;
  a.rows = n.rows;
  a.cols = (int32_t)n.cols;
  a.eps = n.eps;
  const uint32_t grid = norm_grid(n.rows, n.cols);
  pick_deal<T>(n.cols, [&](auto deal) {
    pick(n.residual != nullptr, [&](auto res) {
      pick(!n.y, [&](auto fp8) {
        if constexpr (fp8.value && deal.value != Deal::Whole) return;  // (whole groups of 128)
        if (n.cols > kNormHeld) return (void)norm_long_kernel<T, deal.value, res.value, fp8.value><<<grid, kNormThreads, 0, s>>>(a);
        pick_row(n.cols, [&](auto tpr, auto nv) {
          norm_kernel<T, tpr.value, nv.value, deal.value, res.value, fp8.value><<<grid, kNormThreads, 0, s>>>(a);
        });
      });
    });
  });
  return hipGetLastError();
}

template <class T>
hipError_t run_norm_grad(const NormGradParams& n, float* part, hipStream_t s) {
  NormGradArgs a = {};
  a.dy = n.dy;
  a.s = n.s;
  a.dsum = n.dsum;
  a.lddy = n.lddy;
  a.lds = n.lds;
  a.ldd = n.ldd;
  a.w = n.w;
  a.w_bf16 = n.w_dtype == TJ2_BF16;
  a.rstd = n.rstd;
  a.ds = n.ds;
  a.part = n.dw ? part : nullptr;
  a.rows = n.rows;
  a.cols = (int32_t)n.cols;
  const int64_t parts = norm_parts(n.rows, n.cols);
  if (n.cols > kNormHeld && n.dw) {  // first: ds may take dy's or s' place
    const dim3 grid((uint32_t)((n.cols + kNormThreads - 1) / kNormThreads), (uint32_t)parts);
    norm_grad_slab_kernel<T><<<grid, kNormThreads, 0, s>>>(a, (n.rows + parts - 1) / parts);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  pick_deal<T>(n.cols, [&](auto deal) {
    pick(n.dsum && n.ds, [&](auto dsum) {
      if (n.cols > kNormHeld) {
        if (n.ds) norm_grad_long_kernel<T, deal.value, dsum.value><<<norm_grid(n.rows, n.cols), kNormThreads, 0, s>>>(a);
      } else {
        pick_row(n.cols, [&](auto tpr, auto nv) {
          norm_grad_kernel<T, tpr.value, nv.value, deal.value, dsum.value><<<(uint32_t)parts, kNormThreads, 0, s>>>(a);
        });
      }
    });
  });
  if (hipError_t e = hipGetLastError(); e != hipSuccess || !n.dw) return e;
  norm_dw_kernel<<<(uint32_t)((n.cols + 31) / 32), 1024, 0, s>>>(part, (int)parts, n.cols, n.dw, n.w_dtype == TJ2_BF16);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormParams& n, hipStream_t s) {
  return n.dtype == TJ2_BF16 ? run_norm<uint16_t>(n, s) : run_norm<float>(n, s);
}
size_t norm_grad_workspace_bytes(int64_t rows, int64_t cols) { return (size_t)norm_parts(rows, cols) * (size_t)cols * 4; }
hipError_t launch_norm_grad(const NormGradParams& n, void* ws, hipStream_t s) {
  float* part = reinterpret_cast<float*>(ws);
  return n.dtype == TJ2_BF16 ? run_norm_grad<uint16_t>(n, part, s) : run_norm_grad<float>(n, part, s);
}

}  // namespace tj2
