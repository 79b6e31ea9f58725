// Pieces of the kernels that work row by row on 16-bit activations: eight values to and from 16 bytes, and
// their int8 codes.
#pragma once

#include "qg_device.h"

namespace qg {

template <int T>   // O_F16 / O_BF16
__device__ __forceinline__ float to_f32(uint32_t bits16) {
  if constexpr (T == O_BF16) return bf16_bits_to_f32(bits16);
  else return f16_bits_to_f32(bits16);
}

template <int T>
__device__ __forceinline__ void unpack8(const u32x4 v, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = to_f32<T>(v[i] & 0xFFFFu);
    f[2 * i + 1] = to_f32<T>(v[i] >> 16);
  }
}

template <int T>
__device__ __forceinline__ u32x4 pack8(const float* f) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = (uint32_t)f32_to_out<T>(f[2 * i]) | ((uint32_t)f32_to_out<T>(f[2 * i + 1]) << 16);
  return o;
}

// int8 codes of four values of a row with the scale sc and its reciprocal inv.
//
// The quotients of a row share their divisor, so its reciprocal is divided out once and each quotient
// takes two corrections by its exact remainder: the first leaves less than a unit in the last place, from
// where the second gives the correctly rounded quotient (Markstein, IBM J. Res. Dev. 34, 1990).  Divisors
// whose remainders could leave the range of float32 go through the division itself.
__device__ __forceinline__ uint32_t int8_codes(const float* v, float sc, float inv) {
  uint32_t b[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float q = v[e] * inv;
    q = __builtin_fmaf(__builtin_fmaf(-q, sc, v[e]), inv, q);
    q = __builtin_fmaf(__builtin_fmaf(-q, sc, v[e]), inv, q);
    // |q| <= 127: the sum's last bit is 1, so it rounds to an integer, whose low byte is the code
    b[e] = __float_as_uint(q + 12582912.0f);
  }
  const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x0C0C0400u);
  return lo | (hi << 16);
}
__device__ __forceinline__ uint32_t int8_codes_divided(const float* v, float sc) {
  if (sc != sc) return 0;
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float q = fminf(fmaxf(__builtin_rintf(v[e] / sc), -127.0f), 127.0f);
    w |= ((uint32_t)(int)q & 0xFFu) << (8 * e);
  }
  return w;
}

// e4m3 codes of four values of a row.  One correction: a quotient that lies halfway between two codes is a float32 number,
// which it gives exactly, and of the others one is a unit in the last place off at most.  |quotient| <= 448 to such a unit,
// which the conversion (nearest even) takes to 448.  A row that is not finite has scale NaN and codes 0.
__device__ __forceinline__ uint32_t e4m3_of(const float* q) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);   // bytes 0, 1
  v = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], v, true);        // bytes 2, 3
  return (uint32_t)v;
}
__device__ __forceinline__ uint32_t e4m3_codes(const float* v, float sc, float inv) {
  float q[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    q[e] = v[e] * inv;
    q[e] = __builtin_fmaf(__builtin_fmaf(-q[e], sc, v[e]), inv, q[e]);
  }
  return e4m3_of(q);
}
__device__ __forceinline__ uint32_t e4m3_codes_divided(const float* v, float sc) {
  if (sc != sc) return 0;
  float q[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) q[e] = fminf(fmaxf(v[e] / sc, -448.0f), 448.0f);
  return e4m3_of(q);
}

// MXFP4 codes of 8 of a block's 32 values, whose largest magnitude (of all 32) is amax: the rule of mxfp4_encode32.  The
// conversion divides by the power of two and rounds to the nearest code, halves to the even one, 6 at most; it keeps
// the sign of values that round to zero, which is taken out.
// Returns the UE8M0 byte; a block that is not finite has the byte of NaN (255) and codes 0.
__device__ __forceinline__ uint32_t mxfp4_encode8(const float* v, float amax, uint32_t& codes) {
  codes = 0;
  if (!(amax < __builtin_inff())) return 255;
  // (exponents below -126 would need scales that float32 holds as subnormals: brought up by 2^32 first)
  const int e = amax > 0.f ? max(-127, min(127, __builtin_amdgcn_frexp_expf(amax) - 3)) : -127;
  const bool low = e < -126;
  const float up = low ? 0x1p32f : 1.0f, s = __uint_as_float((uint32_t)(e + 127 + (low ? 32 : 0)) << 23);
  codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0] * up, v[1] * up, s, 0);
  codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[2] * up, v[3] * up, s, 1);
  codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[4] * up, v[5] * up, s, 2);
  codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[6] * up, v[7] * up, s, 3);
  const uint32_t some = (codes | (codes >> 1) | (codes >> 2)) & 0x11111111u;      // bit 0 of each code that is not zero
  codes &= 0x77777777u | (some << 3);
  return (uint32_t)(e + 127);
}

// The value of another lane of its 16: M = 0xB1 and 0x4E the one whose place is this one's XOR 1 or 2, 0x141 and 0x140 its
// mirror image in eight and in sixteen.
template <int M>
__device__ __forceinline__ float neighbour(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), M, 0xF, 0xF, true));
}

// A symmetric operation over 16 or all 64 lanes, the same bits in each.  (in the vector unit: exchanges through LDS take several
// times as long)
template <int N, typename F>
__device__ __forceinline__ float over_lanes(float v, F with) {
  static_assert(N == 16 || N == 64, "rows of lanes or a wave");
  v = with(v, neighbour<0xB1>(v));
  v = with(v, neighbour<0x4E>(v));
  v = with(v, neighbour<0x141>(v));
  v = with(v, neighbour<0x140>(v));
  if constexpr (N == 64) {
    const uint32_t w = __float_as_uint(v);
    const auto rows = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    v = with(__uint_as_float(rows[0]), __uint_as_float(rows[1]));
    const uint32_t h = __float_as_uint(v);
    const auto halves = __builtin_amdgcn_permlane32_swap(h, h, false, false);
    v = with(__uint_as_float(halves[0]), __uint_as_float(halves[1]));
  }
  return v;
}

}  // namespace qg
