// e4m3 codes (no infinities, 0x7F and 0xFF are NaN) with a power of two per
// block, as the 8-bit cache holds them.
#pragma once

#include "attn_common.hpp"

namespace qg {

// An exponent byte as it counts: 0 and 255 are not written by any call, and count
// as 1 and 254.
__device__ __forceinline__ uint32_t exp_of(uint32_t byte) { return byte < 1 ? 1 : byte > 254 ? 254 : byte; }
// 2^(byte - 127) of an exponent byte
__device__ __forceinline__ float exp_scale(uint32_t byte) { return __uint_as_float(exp_of(byte) << 23); }
// 2^(127 - e) of an exponent e from 1 to 254 (2^-127 is subnormal)
__device__ __forceinline__ float exp_inverse(int e) {
  return __uint_as_float(e < 254 ? (uint32_t)(254 - e) << 23 : 0x400000u);
}

// Two codes, the low or high half of `codes`, times a power of two, as two
// 16-bit values: one instruction, exact where the type holds the value (with its
// four significant bits from 2^-21 to 65504 in fp16, from 2^-130 on in bf16),
// rounded to nearest even below, subnormal ones too, infinite above.
template <typename E, bool HI>
__device__ __forceinline__ uint32_t decode2(uint32_t codes, float scale);
template <>
__device__ __forceinline__ uint32_t decode2<F16, false>(uint32_t codes, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, scale, false));
}
template <>
__device__ __forceinline__ uint32_t decode2<F16, true>(uint32_t codes, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, scale, true));
}
template <>
__device__ __forceinline__ uint32_t decode2<BF16, false>(uint32_t codes, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, false));
}
template <>
__device__ __forceinline__ uint32_t decode2<BF16, true>(uint32_t codes, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, true));
}
// eight codes -> eight 16-bit values
template <typename E>
__device__ __forceinline__ u4 decode8(uint32_t lo, uint32_t hi, float scale) {
  return u4{decode2<E, false>(lo, scale), decode2<E, true>(lo, scale), decode2<E, false>(hi, scale),
            decode2<E, true>(hi, scale)};
}

// four floats (at most 448, or NaN) -> four codes, rounded to nearest even
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  return __builtin_amdgcn_cvt_pk_fp8_f32(c, d, __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false), true);
}

// codes of a block whose exponent grew, under the new one: by = 2^(old - new)
__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float by) {
  const f2v lo = __builtin_amdgcn_cvt_pk_f32_fp8(codes, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(codes, true);
  return encode4(lo[0] * by, lo[1] * by, hi[0] * by, hi[1] * by);
}
// 2^(from - to), 0 where it is below 2^-126, for from <= to
__device__ __forceinline__ float exp_ratio(int from, int to) {
  return to - from < 127 ? __uint_as_float((uint32_t)(127 + from - to) << 23) : 0.f;
}

// The exponent byte of a block: the least e with amax <= 448 * 2^e (448, the
// largest code, is 1.75 * 2^8), at least -64, plus 127.  amax is finite.
constexpr int EXP_LEAST = 127 - 64;
__device__ __forceinline__ int exp_byte(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < EXP_LEAST ? EXP_LEAST : e;
}

}  // namespace qg
