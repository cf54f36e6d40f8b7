// 8-bit rows: quantiser and its inverse.
//
//   scale[t] = amax(row t) / 127, rounded to binary32, at least 2^-126
//   element  = x / scale rounded half to even, of the exact quotient
//
// The quantiser reads each row once: a wave (rows of up to 2048 elements) or a
// workgroup holds it in registers between the maximum and the elements.
// Bound by HBM: 2 (or 4) bytes read and 1 written per element.
//
// Nearest element: q = rint(x r), r the reciprocal unit's 1 / scale (1 ulp),
// is off by at most one, and only where x lies within 2^-15 scale of a border.
// d = x - q scale is exact in one fused multiply-add there (a multiple of the
// scale's last place no larger than the scale), so comparing 2 |d| with the
// scale finds the nearest, and the tie, without a division.
#include <algorithm>

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

// the row's scale from its largest magnitude's bits; NaN where that is no number
template <int DT>
__device__ __forceinline__ float scale_of(uint32_t top) {
  constexpr uint32_t inf = DT == NM_F32 ? 0x7F800000u : DT == NM_BF16 ? 0x7F80u : 0x7C00u;
  if (top >= inf) return __builtin_bit_cast(float, 0x7FC00000u);
  const float amax = DT == NM_F32 ? __builtin_bit_cast(float, top) : from_16<DT == NM_F32 ? NM_BF16 : DT>(top);
  return fmaxf(amax / 127.0f, 0x1p-126f);
}

// x / s to the nearest whole number, half to even (r: 1 / s within 1 ulp)
__device__ __forceinline__ float nearest(float x, float s, float r) {
  const float q = __builtin_rintf(x * r);
  const float d = __builtin_fmaf(-q, s, x);
  const float a = 2.0f * __builtin_fabsf(d);
  const bool odd = (int)q & 1;
  return a > s || (a == s && odd) ? q + __builtin_copysignf(1.0f, d) : q;
}

template <int DT>
__device__ __forceinline__ v2i codes_of(const Eight<DT>& e, float s, float r) {
  v2i c;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = nearest(e.value(4 * h + i), s, r);
    c[h] = (int)pack_rne_i8x4(q[0], q[1], q[2], q[3]);
  }
  return c;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t m) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  return m;
}

// TH threads a row, IT pieces of eight columns each in registers (TH = 64:
// four rows a workgroup); MORE: rows longer than that, read twice.
template <int DT, int TH, int IT, bool MORE>
__global__ void __launch_bounds__(256) i8_quantize_kernel(const uint8_t* X, int64_t ldx, int64_t rows, int64_t K,
                                                          int64_t Kp, int8_t* codes, float* scales) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int EB = DT == NM_F32 ? 4 : 2;
  constexpr int RW = 256 / TH;                          // rows of a workgroup
  __shared__ uint32_t part[4];
  const int th = threadIdx.x % TH;
  for (int64_t g = blockIdx.x; g * RW < rows; g += gridDim.x) {
    const int64_t row = g * RW + threadIdx.x / TH;
    if (RW > 1 && row >= rows) return;
    const uint8_t* x = X + row * ldx * EB;
    Eight<DT> e[IT];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int64_t k = 8 * (int64_t)(th + TH * i);
      e[i].clear();
      if (k < K) e[i].load(x, k, K);
    }
#pragma unroll
    for (int i = 0; i < IT; ++i) m = max(m, e[i].top());
    if constexpr (MORE) {
      for (int64_t k = 8 * (int64_t)(th + TH * IT); k < K; k += 8 * TH) {
        Eight<DT> f;
        f.load(x, k, K);
        m = max(m, f.top());
      }
    }
    m = wave_max(m);
    if constexpr (TH > 64) {
      if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
      __syncthreads();
      m = max(max(part[0], part[1]), max(part[2], part[3]));
      __syncthreads();                                  // (the next row's maximum comes after every read)
    }
    const float s = scale_of<DT>(m);
    const bool number = s == s;
    const float r = __builtin_amdgcn_rcpf(s);
    int8_t* c = codes + row * Kp;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int64_t k = 8 * (int64_t)(th + TH * i);
      if (k < Kp) *reinterpret_cast<v2i*>(c + k) = number ? codes_of<DT>(e[i], s, r) : v2i{0, 0};
    }
    if constexpr (MORE) {
      for (int64_t k = 8 * (int64_t)(th + TH * IT); k < Kp; k += 8 * TH) {
        Eight<DT> f;
        f.clear();
        if (k < K) f.load(x, k, K);
        *reinterpret_cast<v2i*>(c + k) = number ? codes_of<DT>(f, s, r) : v2i{0, 0};
      }
    }
    if (th == 0) scales[row] = s;
  }
#endif
}

template <int DT>
hipError_t launch_quantize_dt(const void* X, int64_t ldx, int64_t rows, int64_t K, int8_t* codes, float* scales,
                              hipStream_t s) {
  const int64_t Kp = i8_kp(K), pieces = Kp / 8;
  auto go = [&](auto kernel, int rw) {
    const int64_t n = (rows + rw - 1) / rw;
    hipLaunchKernelGGL(kernel, dim3((unsigned)std::min<int64_t>(n, 1 << 22)), dim3(256), 0, s,
                       static_cast<const uint8_t*>(X), ldx, rows, K, Kp, codes, scales);
    return hipGetLastError();
  };
  if (pieces <= 64) return go(i8_quantize_kernel<DT, 64, 1, false>, 4);
  if (pieces <= 128) return go(i8_quantize_kernel<DT, 64, 2, false>, 4);
  if (pieces <= 256) return go(i8_quantize_kernel<DT, 64, 4, false>, 4);
  if (pieces <= 512) return go(i8_quantize_kernel<DT, 256, 2, false>, 1);
  if (pieces <= 1024) return go(i8_quantize_kernel<DT, 256, 4, false>, 1);
  if (pieces <= 1536) return go(i8_quantize_kernel<DT, 256, 6, false>, 1);
  if (pieces <= 2048) return go(i8_quantize_kernel<DT, 256, 8, false>, 1);
  return go(i8_quantize_kernel<DT, 256, 8, true>, 1);
}

// eight elements a thread
template <int DT>
__global__ void __launch_bounds__(256) i8_dequantize_kernel(const int8_t* codes, const float* scales, int64_t rows,
                                                            int64_t K, int64_t Kp, void* Y, int64_t ldy) {
  const int64_t pr = (K + 7) / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * pr; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / pr, k = (i - r * pr) * 8;
    const v2i c = *reinterpret_cast<const v2i*>(codes + r * Kp + k);
    const float s = scales[r];
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = (float)((int)((uint32_t)c[e >> 2] << (24 - 8 * (e & 3))) >> 24) * s;
    const int n = (int)min(K - k, (int64_t)8);
    if (DT != NM_F32 && n == 8) {
      constexpr int D16 = DT == NM_F32 ? NM_F16 : DT;
      *reinterpret_cast<v4i_any*>(static_cast<uint16_t*>(Y) + r * ldy + k) =
          v4i_any{(int)pack_16x2<D16>(y[0], y[1]), (int)pack_16x2<D16>(y[2], y[3]), (int)pack_16x2<D16>(y[4], y[5]),
                  (int)pack_16x2<D16>(y[6], y[7])};
    } else {
      store4<DT>(Y, r * ldy + k, y, min(n, 4));
      if (n > 4) store4<DT>(Y, r * ldy + k + 4, y + 4, n - 4);
    }
  }
}

}  // namespace

hipError_t launch_i8_quantize(const void* X, int64_t ldx, int xdt, int64_t rows, int64_t K, int8_t* codes,
                              float* scales, hipStream_t s) {
  if (xdt == NM_F16) return launch_quantize_dt<NM_F16>(X, ldx, rows, K, codes, scales, s);
  if (xdt == NM_BF16) return launch_quantize_dt<NM_BF16>(X, ldx, rows, K, codes, scales, s);
  return launch_quantize_dt<NM_F32>(X, ldx, rows, K, codes, scales, s);
}

hipError_t launch_i8_dequantize(const int8_t* codes, const float* scales, int64_t rows, int64_t K, void* Y,
                                int64_t ldy, int ydt, hipStream_t s) {
  const dim3 grid(grid_1d(rows * ((K + 7) / 8), 256)), block(256);
  const int64_t Kp = i8_kp(K);
  if (ydt == NM_F16)
    hipLaunchKernelGGL((i8_dequantize_kernel<NM_F16>), grid, block, 0, s, codes, scales, rows, K, Kp, Y, ldy);
  else if (ydt == NM_BF16)
    hipLaunchKernelGGL((i8_dequantize_kernel<NM_BF16>), grid, block, 0, s, codes, scales, rows, K, Kp, Y, ldy);
  else
    hipLaunchKernelGGL((i8_dequantize_kernel<NM_F32>), grid, block, 0, s, codes, scales, rows, K, Kp, Y, ldy);
  return hipGetLastError();
}

}  // namespace nm
