// Product of a few rows (tokens) with a long operand, for decoding and scoring:
// D[t, v] = sum_k X[t, k] W[v, k] for up to 64 tokens, bound by one read of W.
//
// The tokens' operand sits in LDS whole; W goes from memory straight into
// registers, 16 rows a wave, a batch of U chunks (128 bytes of each row) ahead of
// the one in the matrix units, so a CU keeps 64 to 128 KB in flight where a staged
// tile is limited by its LDS stage and a barrier a chunk.  A wave takes
// groups of 16 rows in turn, its loads running on into the next group; no barrier
// after the tokens are in place.
#pragma once
#include "tj2_tile.h"

namespace tj2 {

template <int EL, int TN, int LDS_BYTES>
struct Skinny {
  static constexpr int NT = 256, WAVES = NT / 64, U = EL == EL_MX ? 4 : 8;
  static constexpr int TOKENS = 16 * TN;
  static constexpr int PER_CU = 160 * 1024 / (LDS_BYTES + LDS_BYTES / 16 + 512) >= 2 ? 2 : 1;

  struct Smem {
    __attribute__((aligned(16))) uint8_t x[LDS_BYTES];
    __attribute__((aligned(16))) uint8_t xs[EL == EL_MX ? LDS_BYTES / 16 + 2 * TOKENS : 16];  // MXFP4 scale bytes
  };

  // LDS row pitch of a token: whole chunks and 16 bytes, so that 16 tokens' pieces lie in different banks
  static __host__ __device__ __forceinline__ int pitch(int kb) { return (kb + 127) / 128 * 128 + 16; }
  // scale bytes of a token in LDS: 8 per chunk
  static __host__ __device__ __forceinline__ int scale_pitch(int kb) { return (kb + 127) / 128 * 8 + 2; }
  static bool fits(int64_t tokens, int64_t kb) {
    return tokens <= TOKENS && TOKENS * (int64_t)pitch((int)kb) <= LDS_BYTES;
  }
  // Workgroups whose waves share `rows` in groups of 16 evenly, at most what runs at once.
  static uint32_t grid(int64_t rows) {
    const int64_t groups = (rows + 15) / 16, most = (int64_t)kCus * PER_CU * WAVES, rounds = (groups + most - 1) / most;
    return (uint32_t)((groups + rounds * WAVES - 1) / (rounds * WAVES));
  }

  typedef float4_t Acc[TN];

  // The tokens are in sm (zero beyond them and beyond their kb bytes), a barrier
  // crossed.  epilogue(group, acc): acc[tn][r] is the result of W row
  // 16 group + 4 g + r and token 16 tn + n (lane n + 16 g).
  template <class Epilogue>
  static __device__ __forceinline__ void run(const TileOp& P, const Smem& sm, Epilogue&& epilogue) {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const uint32_t wave = blockIdx.x * WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = gridDim.x * WAVES;
    const uint32_t groups = (uint32_t)((P.rows + 15) >> 4);
    if (wave >= groups) return;
    const int chunks = (P.kb + 127) >> 7, batches = (chunks + U - 1) / U;
    const int px = pitch(P.kb), ps = scale_pitch(P.kb);
    const uint8_t* xl = sm.x + n * px + g * 32;
    const uint8_t* sl = sm.xs + n * ps + g * 2;

    struct Batch {
      i32x4_t a[U][2];
      uint16_t s[EL == EL_MX ? U : 1];
    };
    // batch b of group gr
    auto fetch = [&](Batch& f, uint32_t gr, int b) __attribute__((always_inline)) {
      const int64_t r0 = (int64_t)gr * 16;
      const bool in = r0 + n < P.rows;
      const auto d = __builtin_amdgcn_make_buffer_rsrc((void*)(P.p + r0 * P.ld), 0, 0x7FFFFFFF, 0x00020000);
      const uint32_t row = (uint32_t)n * (uint32_t)P.ld;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t at = (uint32_t)(b * U + u) * 128u + (uint32_t)g * 32u;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          f.a[u][h] = __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                          d, in && at + h * 16 < (uint32_t)P.kb ? row + at + h * 16 : kOutside, 0, 0));
      }
      if constexpr (EL == EL_MX) {
        const auto ds = __builtin_amdgcn_make_buffer_rsrc((void*)(P.s + r0 * P.ld / 16), 0, 0x7FFFFFFF, 0x00020000);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t at = (uint32_t)(b * U + u) * 8u + (uint32_t)g * 2u;
          f.s[u] = __builtin_amdgcn_raw_buffer_load_b16(ds, in && at < (uint32_t)P.kb / 16 ? (uint32_t)n * (uint32_t)(P.ld / 16) + at : kOutside, 0, 0);
        }
      }
    };
    Acc acc = {};
    auto multiply = [&](const Batch& f, int b) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = b * U + u;
        if (c >= chunks) break;
#pragma unroll
        for (int tn = 0; tn < TN; ++tn) {
          const i32x4_t* x = reinterpret_cast<const i32x4_t*>(xl + tn * 16 * px + c * 128);
          if constexpr (EL == EL_BF16) {
            acc[tn] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, f.a[u][0]),
                                                              __builtin_bit_cast(bf16x8_t, x[0]), acc[tn], 0, 0, 0);
            acc[tn] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, f.a[u][1]),
                                                              __builtin_bit_cast(bf16x8_t, x[1]), acc[tn], 0, 0, 0);
          } else {
            const int sx = *reinterpret_cast<const uint16_t*>(sl + tn * 16 * ps + c * 8), sw = f.s[u];
            const i32x4_t z = {0, 0, 0, 0};
            acc[tn] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_shufflevector(f.a[u][0], z, 0, 1, 2, 3, 4, 5, 6, 7),
                                                                       __builtin_shufflevector(x[0], z, 0, 1, 2, 3, 4, 5, 6, 7),
                                                                       acc[tn], 4, 4, 0, sw, 0, sx);
            acc[tn] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_shufflevector(f.a[u][1], z, 0, 1, 2, 3, 4, 5, 6, 7),
                                                                       __builtin_shufflevector(x[1], z, 0, 1, 2, 3, 4, 5, 6, 7),
                                                                       acc[tn], 4, 4, 1, sw, 1, sx);
          }
        }
      }
    };
    uint32_t gr = wave;   // of the batch in the matrix units
    int b = 0;
    Batch f0, f1;
    fetch(f0, gr, 0);
    // two batches a turn, so that each has its own registers
    auto turn = [&](const Batch& now, Batch& next) __attribute__((always_inline)) -> bool {
      uint32_t ng = gr;
      int nb = b + 1;
      if (nb == batches) {
        nb = 0;
        ng += waves;
      }
      if (ng < groups) fetch(next, ng, nb);
      multiply(now, b);
      if (ng != gr) {
        epilogue(gr, acc);
#pragma unroll
        for (int tn = 0; tn < TN; ++tn) acc[tn] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
      }
      gr = ng;
      b = nb;
      return gr < groups;
    };
    while (turn(f0, f1) && turn(f1, f0)) {
    }
  }
};

}  // namespace tj2
