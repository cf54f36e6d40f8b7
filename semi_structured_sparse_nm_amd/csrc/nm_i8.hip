// 8-bit rows: quantiser and its inverse.
//
//   scale[t] = amax(row t) x 1/127 in binary32, at least 2^-126
//   element  = x / scale rounded half to even, of the exact quotient
//
// The quantiser reads each row once: a wave (rows of up to 2048 elements) or a
// workgroup holds it in registers between the maximum and the elements.
// Bound by HBM: 2 (or 4) bytes read and 1 written per element.
#include <algorithm>

#include "nm_i8_device.hpp"

namespace nm {

namespace {

// TH threads a row, IT pieces of eight columns each in registers (TH = 64:
// four rows a workgroup); MORE: rows longer than that, read twice.
template <int DT, int TH, int IT, bool MORE>
__global__ void __launch_bounds__(TH < 256 ? 256 : TH)
    i8_quantize_kernel(const uint8_t* X, int64_t ldx, int64_t rows, int64_t K, int64_t Kp, int8_t* codes,
                       float* scales) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int EB = DT == NM_F32 ? 4 : 2;
  constexpr int RW = TH < 256 ? 256 / TH : 1;           // rows of a workgroup
  __shared__ uint32_t part[TH / 64];
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
#pragma unroll
      for (int w = 0; w < TH / 64; ++w) m = max(m, part[w]);
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
  auto go = [&](auto kernel, int rw, int threads = 256) {
    const int64_t n = (rows + rw - 1) / rw;
    hipLaunchKernelGGL(kernel, dim3((unsigned)std::min<int64_t>(n, 1 << 22)), dim3(threads), 0, s,
                       static_cast<const uint8_t*>(X), ldx, rows, K, Kp, codes, scales);
    return hipGetLastError();
  };
  // fewer rows than compute units: as many threads a row as it has pieces for
  // (16 rows of 11008: 7.0 us with 256 threads a row, 3.8 with 1024)
  if (rows <= 256 && pieces > 64 && pieces <= 2048) {
    if (pieces <= 256) return go(i8_quantize_kernel<DT, 256, 1, false>, 1);
    if (pieces <= 1024) return go(i8_quantize_kernel<DT, 1024, 1, false>, 1, 1024);
    return go(i8_quantize_kernel<DT, 1024, 2, false>, 1, 1024);
  }
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
