// Microscaled 4-bit format: quantiser and its inverse.
//
// Quantiser: one workgroup per unit of 32 rows x 256 columns.  Four lanes
// share a block of 32, eight elements each (one 16-byte load of 16-bit
// values, coalesced along the row); the block's largest magnitude meets by
// two lane exchanges, each lane writes its eight codes as one dword, and the
// unit's scales are gathered in LDS and leave as one 256-byte piece.  Bound by
// HBM: 2 (or 4) bytes read and 17 / 32 written per element (11008 x 4096 bf16:
// 20 us, 5.7 TB/s; back to bf16 28 us, 4.1 TB/s).
#include "nm_mx_device.hpp"

namespace nm {

namespace {

template <int DT>
__global__ void __launch_bounds__(256) mx_quantize_kernel(const uint8_t* X, int64_t ldx, int64_t rows, int64_t K,
                                                          int64_t nslab, uint8_t* codes, uint8_t* scales, bool vec) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int EB = DT == NM_F32 ? 4 : 2;
  constexpr int ND = 8 * EB / 4;                       // dwords of eight elements
  __shared__ uint8_t sc[256];
  const int64_t slab = blockIdx.x % nslab, grp = blockIdx.x / nslab;
  const int64_t k0 = slab * kMxSlab;
  sc[threadIdx.x] = 0;
  __syncthreads();
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int q = it * 256 + threadIdx.x;              // 32 pieces of eight per row
    const int rl = q >> 5, pc = q & 31;
    const int64_t r = grp * 32 + rl, k = k0 + 8 * pc;
    uint32_t x[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i) x[i] = 0;
    if (r < rows && k < K) {
      const uint8_t* p = X + (r * ldx + k) * EB;
      if (vec && k + 8 <= K) {
#pragma unroll
        for (int i = 0; i < ND / 4; ++i) {
          const v4i v = reinterpret_cast<const v4i*>(p)[i];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[4 * i + e] = (uint32_t)v[e];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (k + i < K) {
            if constexpr (EB == 4)
              x[i] = reinterpret_cast<const uint32_t*>(p)[i];
            else
              x[i >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
          }
      }
    }
    const uint32_t m = quad_max(mx_amax8<DT>(x));
    const uint32_t byte = mx_scale_byte(m);
    uint32_t c = mx_codes8<DT>(x, mx_scale_f32(byte));
    if (byte == 255u) c = 0;
    if (r < rows) {
      *reinterpret_cast<uint32_t*>(codes + r * (nslab * 128) + slab * 128 + 4 * pc) = c;
      const int b = pc >> 2;
      if ((pc & 3) == 0) sc[4 * (16 * (b & 3) + (rl & 15)) + 2 * (rl >> 4) + (b >> 2)] = (uint8_t)byte;
    }
  }
  __syncthreads();
  if (threadIdx.x < 64)
    reinterpret_cast<uint32_t*>(scales + (grp * nslab + slab) * 256)[threadIdx.x] =
        reinterpret_cast<const uint32_t*>(sc)[threadIdx.x];
#endif
}

// value of a 4-bit code times its scale
__device__ __forceinline__ float mx_value(uint32_t code, uint32_t byte) {
  // magnitudes times two: 0 1 2 3 4 6 8 12, one byte each
  const uint32_t m2 = (code & 4 ? 0x0C080604u >> (8 * (code & 3)) : 0x03020100u >> (8 * (code & 3))) & 0xFFu;
  if (byte == 255u) return __builtin_bit_cast(float, 0x7FC00000u);
  // m2 2^(byte - 128), in two exact factors: 2^-127 and 2^-128 are subnormal
  const float half = 0.5f * (float)m2;
  const float s = byte ? __builtin_bit_cast(float, byte << 23) : __builtin_bit_cast(float, 0x00400000u);
  const float y = half * s;
  return code & 8 ? -y : y;
}

template <int DT>
__global__ void __launch_bounds__(256) mx_dequantize_kernel(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                                            int64_t K, int64_t nslab, void* Y, int64_t ldy,
                                                            bool vec) {
  const int64_t pr = (K + 7) / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * pr; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / pr, k = (i - r * pr) * 8;
    const uint32_t c = *reinterpret_cast<const uint32_t*>(codes + r * (nslab * 128) + k / 2);
    const int b = (int)(k & 255) >> 5, rl = (int)(r & 31);
    const uint32_t byte =
        scales[((r >> 5) * nslab + (k >> 8)) * 256 + 4 * (16 * (b & 3) + (rl & 15)) + 2 * (rl >> 4) + (b >> 2)];
    float y[8];
  #pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = mx_value(c >> (4 * e) & 15u, byte);
    const int n = (int)min(K - k, (int64_t)8);
    if constexpr (DT != NM_F32) {
      if (vec && n == 8) {
        uint32_t o[4];
  #pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = pack_16x2<DT>(y[2 * e], y[2 * e + 1]);
        *reinterpret_cast<v4i*>(static_cast<uint16_t*>(Y) + r * ldy + k) =
            v4i{(int)o[0], (int)o[1], (int)o[2], (int)o[3]};
        continue;
      }
    }
    store4<DT>(Y, r * ldy + k, y, min(n, 4), vec);
    if (n > 4) store4<DT>(Y, r * ldy + k + 4, y + 4, n - 4, vec);
  }
}

}  // namespace

hipError_t launch_mx_quantize(const void* X, int64_t ldx, int xdt, int64_t rows, int64_t K, uint8_t* codes,
                              uint8_t* scales, hipStream_t s) {
  const int64_t nslab = mx_kp(K) / kMxSlab;
  const int eb = xdt == NM_F32 ? 4 : 2;
  const bool vec = (uintptr_t)X % 16 == 0 && ldx * eb % 16 == 0;
  const dim3 grid((unsigned)((rows + 31) / 32 * nslab)), block(256);
  const uint8_t* x = static_cast<const uint8_t*>(X);
  if (xdt == NM_F16)
    hipLaunchKernelGGL((mx_quantize_kernel<NM_F16>), grid, block, 0, s, x, ldx, rows, K, nslab, codes, scales, vec);
  else if (xdt == NM_BF16)
    hipLaunchKernelGGL((mx_quantize_kernel<NM_BF16>), grid, block, 0, s, x, ldx, rows, K, nslab, codes, scales, vec);
  else
    hipLaunchKernelGGL((mx_quantize_kernel<NM_F32>), grid, block, 0, s, x, ldx, rows, K, nslab, codes, scales, vec);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, void* Y,
                                int64_t ldy, int ydt, hipStream_t s) {
  const int64_t nslab = mx_kp(K) / kMxSlab;
  const bool vec = ydt == NM_F32 ? vec4_ok(Y, ldy, 4) : (uintptr_t)Y % 16 == 0 && ldy % 8 == 0;
  const int64_t n = rows * ((K + 7) / 8);
  const dim3 grid(grid_1d(n, 256)), block(256);
  if (ydt == NM_F16)
    hipLaunchKernelGGL((mx_dequantize_kernel<NM_F16>), grid, block, 0, s, codes, scales, rows, K, nslab, Y, ldy, vec);
  else if (ydt == NM_BF16)
    hipLaunchKernelGGL((mx_dequantize_kernel<NM_BF16>), grid, block, 0, s, codes, scales, rows, K, nslab, Y, ldy, vec);
  else
    hipLaunchKernelGGL((mx_dequantize_kernel<NM_F32>), grid, block, 0, s, codes, scales, rows, K, nslab, Y, ldy, vec);
  return hipGetLastError();
}

}  // namespace nm
