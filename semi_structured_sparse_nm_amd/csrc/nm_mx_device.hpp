// Rounding to the microscaled 4-bit format, shared by the quantiser and the
// few-token product.
//
// A block's scale exponent is floor(log2(amax)) - 2: with amax as a binary32
// number (every fp16 and bf16 value is one exactly), the biased exponent
// byte of the scale is amax's own biased exponent - 2, at least 0 (amax's
// subnormals have exponent 0, so they land there too).  Elements are rounded
// half to even, with saturation, by v_cvt_scalef32_pk_fp4_*, which divides by
// a power of two exactly.
#pragma once

#include "nm_ffn.hpp"

namespace nm {

#if defined(__HIP_DEVICE_COMPILE__)
namespace {

typedef unsigned short v2u16 __attribute__((ext_vector_type(2)));

// E8M0 byte of a block whose largest magnitude is amax (a binary32's bits,
// sign cleared); 0xFF where it is not finite
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
// the scale as binary32: 2^(byte - 127), byte 0 the subnormal 2^-127
__device__ __forceinline__ float mx_scale_f32(uint32_t byte) {
  return __builtin_bit_cast(float, byte ? byte << 23 : 0x00400000u);
}

// larger of two pairs of sign-cleared 16-bit floats (their bits order them)
__device__ __forceinline__ uint32_t max_16x2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(
      uint32_t, __builtin_elementwise_max(__builtin_bit_cast(v2u16, a), __builtin_bit_cast(v2u16, b)));
}

// amax as binary32 bits from 16-bit pairs' running maximum
template <int DT>
__device__ __forceinline__ uint32_t amax_bits_16(uint32_t m) {
  const uint32_t lo = m & 0xFFFFu, hi = m >> 16;
  return __builtin_bit_cast(uint32_t, from_16<DT>(lo > hi ? lo : hi));
}

// eight values (four dwords of 16-bit pairs, or eight binary32) -> eight
// codes, element i in bits 4 i ..
template <int DT>
__device__ __forceinline__ uint32_t mx_codes8(const uint32_t* x, float scale) {
  uint32_t r = 0;
  if constexpr (DT == NM_F16) {
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(v2h_, x[0]), scale, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(v2h_, x[1]), scale, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(v2h_, x[2]), scale, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(v2h_, x[3]), scale, 3);
  } else if constexpr (DT == NM_BF16) {
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(v2bf_, x[0]), scale, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(v2bf_, x[1]), scale, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(v2bf_, x[2]), scale, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(v2bf_, x[3]), scale, 3);
  } else {
    const float* f = reinterpret_cast<const float*>(x);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[0], f[1], scale, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[2], f[3], scale, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[4], f[5], scale, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[6], f[7], scale, 3);
  }
  return r;
}

// largest of the four lanes 4 i .. 4 i + 3 (lane exchanges inside the vector unit)
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));   // lane ^ 1
  return max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));   // lane ^ 2
}

// bits of the largest magnitude (as binary32) among eight values
template <int DT>
__device__ __forceinline__ uint32_t mx_amax8(const uint32_t* x) {
  if constexpr (DT == NM_F32) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, x[i] & 0x7FFFFFFFu);
    return m;
  } else {
    uint32_t m = x[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 4; ++i) m = max_16x2(m, x[i] & 0x7FFF7FFFu);
    return amax_bits_16<DT>(m);
  }
}

}  // namespace
#endif

}  // namespace nm
