// E4M3 groups of 128 elements under one fp32 scale, as the FP8 quantisers (fp8.hip) and
// the norm that writes them (norm.hip) form them.
#pragma once
#include "tj2_device.h"

namespace tj2 {

// Largest of the 16 lanes of an aligned group (DPP: quad swaps, half-row mirror, and the
// rotation by 8 of a row of 16).  Bit patterns of magnitudes order as unsigned integers,
// an infinity and NaNs above every finite value.
__device__ __forceinline__ uint32_t max16_lanes(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xF, 0xF, false));
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xF, 0xF, false));
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x141, 0xF, 0xF, false));
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x128, 0xF, 0xF, false));
  return x;
}

__device__ __forceinline__ uint32_t top_bits8(const float v[8]) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

// The scale S = amax / 448 of a group whose largest magnitude has the bits `top`, and what
// its elements are multiplied by, fl(1 / S); a group below 2^-100 is empty (S = 0), one
// that holds an infinity or NaN has the scale NaN and zero codes.
struct Fp8Scale {
  float S, inv;
};
__device__ __forceinline__ Fp8Scale fp8_scale(uint32_t top) {
  if (top >= 0x7F800000u) return {__uint_as_float(0x7FC00000u), 0.0f};
  const float a = __uint_as_float(top);
  if (a < kTiny) return {0.0f, 0.0f};
  const float S = a / kFp8Div;
  return {S, 1.0f / S};
}

// 8 elements to 8 bytes: v = clamp(fl(y inv), +-448) to the nearest E4M3 value, ties to even.
__device__ __forceinline__ uint2 fp8_codes8(const float v[8], const Fp8Scale& s) {
  typedef short short2_t __attribute__((ext_vector_type(2)));
  uint32_t out[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    short2_t d = {0, 0};
    d = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(d, fp8_scaled(v[4 * w], s.inv), fp8_scaled(v[4 * w + 1], s.inv), 1.0f, false);
    d = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(d, fp8_scaled(v[4 * w + 2], s.inv), fp8_scaled(v[4 * w + 3], s.inv), 1.0f, true);
    out[w] = __builtin_bit_cast(uint32_t, d);
  }
  // (a group with a NaN scale has inv 0: its infinities and NaNs times 0 are NaN)
  return s.S != s.S ? uint2{0u, 0u} : uint2{out[0], out[1]};
}

// 8 neighbouring elements at p, 16-byte aligned
__device__ __forceinline__ void load8(const uint16_t* p, float v[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float v[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

}  // namespace tj2
