// Device parts of the 8-bit rows: shared by the quantiser and the product that
// quantises its own rows.
//
// Nearest element: the sum of x r (r the reciprocal unit's 1 / scale, 1 ulp) and
// 1.5 2^23, rounded once, holds in its last bits a whole number q that is off by
// at most one, and only where x lies within 2^-15 scale of a border.  d = x - q
// scale is exact in one fused multiply-add there (a multiple of the scale's last
// place no larger than the scale), so comparing |d| with half the scale finds the
// nearest without a division; on a tie an odd q is the wrong one, so for odd q the
// half's predecessor is compared with.
#pragma once

#include "nm_rows.hpp"

namespace nm {

namespace {

// eight elements k .. k + 7 of a row, as sign-cleared bits' maximum and values
template <int DT>
struct Eight {
  uint32_t x[DT == NM_F32 ? 8 : 4];
  __device__ __forceinline__ void load(const void* row, int64_t k, int64_t K) {
    if constexpr (DT == NM_F32) {
      const uint32_t* p = static_cast<const uint32_t*>(row) + k;
      if (k + 8 <= K) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const v4f v = *reinterpret_cast<const v4f_any*>(p + 4 * i);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[4 * i + e] = __builtin_bit_cast(uint32_t, (float)v[e]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = k + i < K ? p[i] : 0u;
      }
    } else {
      const v4i v = load_piece(static_cast<const uint16_t*>(row), k, K);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = (uint32_t)v[i];
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (uint32_t& v : x) v = 0;
  }
  // largest magnitude's bits (in binary32's order; infinities and NaN on top)
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
    if constexpr (DT == NM_F32) {
#pragma unroll
      for (const uint32_t v : x) m = max(m, v & 0x7FFFFFFFu);
    } else {
      typedef uint16_t v2u __attribute__((ext_vector_type(2)));
      v2u a = {0, 0};
#pragma unroll
      for (const uint32_t v : x) a = __builtin_elementwise_max(a, __builtin_bit_cast(v2u, v & 0x7FFF7FFFu));
      m = max((uint32_t)a[0], (uint32_t)a[1]);
    }
    return m;
  }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (DT == NM_F32)
      return __builtin_bit_cast(float, x[i]);
    else
      return from_16<DT>((x[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
  }
};

constexpr float kInv127 = 0x1.020408p-7f;              // 1 / 127, rounded
// the row's scale from its largest magnitude's bits; NaN where that is no number
template <int DT>
__device__ __forceinline__ float scale_of(uint32_t top) {
  constexpr uint32_t inf = DT == NM_F32 ? 0x7F800000u : DT == NM_BF16 ? 0x7F80u : 0x7C00u;
  if (top >= inf) return __builtin_bit_cast(float, 0x7FC00000u);
  const float amax = DT == NM_F32 ? __builtin_bit_cast(float, top) : from_16<DT == NM_F32 ? NM_BF16 : DT>(top);
  return fmaxf(amax * kInv127, 0x1p-126f);
}

// x / s to the nearest whole number, half to even, in the low byte (r: 1 / s
// within 1 ulp, h: the bits of s / 2)
__device__ __forceinline__ uint32_t nearest_byte(float x, float s, float r, uint32_t h) {
  const float m = 12582912.0f;                          // 1.5 2^23
  const float u = __builtin_fmaf(x, r, m);
  const float d = __builtin_fmaf(m - u, s, x);
  const uint32_t b = __builtin_bit_cast(uint32_t, u);
  const float half = __builtin_bit_cast(float, h - (b & 1u));
  const int step = (__builtin_bit_cast(int, d) >> 31) | 1;
  return b + (__builtin_fabsf(d) > half ? step : 0);
}

template <int DT>
__device__ __forceinline__ v2i codes_of(const Eight<DT>& e, float s, float r) {
  v2i c;
#if defined(__HIP_DEVICE_COMPILE__)
  const uint32_t h = __builtin_bit_cast(uint32_t, 0.5f * s);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) q[k] = nearest_byte(e.value(4 * i + k), s, r, h);
    const uint32_t lo = __builtin_amdgcn_perm(q[1], q[0], 0x0C0C0400u);
    c[i] = (int)__builtin_amdgcn_perm(__builtin_amdgcn_perm(q[3], q[2], 0x0C0C0400u), lo, 0x05040100u);
  }
#endif
  return c;
}

// the largest of a wave's values (sign-cleared bits)
__device__ __forceinline__ uint32_t wave_max(uint32_t m) {
#if defined(__HIP_DEVICE_COMPILE__)
  return (uint32_t)__builtin_amdgcn_readlane(wave_scan_max((int)m), 63);
#else
  return m;
#endif
}

}  // namespace

}  // namespace nm
