// Microscaled 4-bit format: quantiser and its inverse.
//
// Quantiser: one workgroup per unit of 32 rows x 256 columns.  Four lanes
// share a block of 32, eight elements each (one 16-byte load of 16-bit
// values, coalesced along the row); the block's largest magnitude meets by
// two lane exchanges, each lane writes its eight codes as one dword, and the
// unit's scales are gathered in LDS and leave as one 256-byte piece.  Bound by
// HBM: 2 (or 4) bytes read and 17 / 32 written per element (11008 x 4096 bf16:
// 20 us, 5.7 TB/s; back to bf16 21.5 us, 5.3 TB/s).
#include "nm_mx_device.hpp"

namespace nm {

namespace {

template <int DT, int TH>
__global__ void __launch_bounds__(TH) mx_quantize_kernel(const uint8_t* X, int64_t ldx, int64_t rows, int64_t K,
                                                          int64_t nslab, uint8_t* codes, uint8_t* scales) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int EB = DT == NM_F32 ? 4 : 2;
  constexpr int ND = 8 * EB / 4;                       // dwords of eight elements
  __shared__ __attribute__((aligned(16))) uint8_t sc[256];
  const int64_t slab = blockIdx.x % nslab, grp = blockIdx.x / nslab;
  const int64_t k0 = slab * kMxSlab;
  if (threadIdx.x < 256) sc[threadIdx.x] = 0;
  __syncthreads();
#pragma unroll
  for (int it = 0; it < 1024 / TH; ++it) {
    const int q = it * TH + (int)threadIdx.x;              // 32 pieces of eight per row
    const int rl = q >> 5, pc = q & 31;
    const int64_t r = grp * 32 + rl, k = k0 + 8 * pc;
    uint32_t x[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i) x[i] = 0;
    if (r < rows && k < K) {
      const uint8_t* p = X + (r * ldx + k) * EB;
      if constexpr (EB == 2) {
        const v4i v = load_piece(reinterpret_cast<const uint16_t*>(X) + r * ldx, k, K);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = (uint32_t)v[e];
      } else if (k + 8 <= K) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const v4i v = load16(p + 16 * i);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[4 * i + e] = (uint32_t)v[e];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (k + i < K) x[i] = reinterpret_cast<const uint32_t*>(p)[i];
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

// the quantiser's units and lanes, the other way
template <int DT, int TH>
__global__ void __launch_bounds__(TH) mx_dequantize_kernel(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                                            int64_t K, int64_t nslab, void* Y,
                                                            int64_t ldy) {
  const int64_t slab = blockIdx.x % nslab, grp = blockIdx.x / nslab;
  const uint8_t* sc = scales + (grp * nslab + slab) * 256;
#pragma unroll
  for (int it = 0; it < 1024 / TH; ++it) {
    const int q = it * TH + (int)threadIdx.x;
    const int rl = q >> 5, pc = q & 31, b = pc >> 2;
    const int64_t r = grp * 32 + rl, k = slab * kMxSlab + 8 * pc;
    if (r >= rows || k >= K) continue;
    const uint32_t c = *reinterpret_cast<const uint32_t*>(codes + r * (nslab * 128) + slab * 128 + 4 * pc);
    const uint32_t byte = sc[4 * (16 * (b & 3) + (rl & 15)) + 2 * (rl >> 4) + (b >> 2)];
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = mx_value(c >> (4 * e) & 15u, byte);
    const int n = (int)min(K - k, (int64_t)8);
    if constexpr (DT != NM_F32) {
      if (n == 8) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = pack_16x2<DT>(y[2 * e], y[2 * e + 1]);
        *reinterpret_cast<v4i_any*>(static_cast<uint16_t*>(Y) + r * ldy + k) =
            v4i_any{(int)o[0], (int)o[1], (int)o[2], (int)o[3]};
        continue;
      }
    }
    store4<DT>(Y, r * ldy + k, y, min(n, 4));
    if (n > 4) store4<DT>(Y, r * ldy + k + 4, y + 4, n - 4);
  }
}

}  // namespace

namespace {

// Threads of a workgroup: 256, four passes over the unit; 1024, one pass, where
// there are few units (197 x 768: 4.6 us, both ways, against 5.6 and 6.8).
bool few_units(int64_t units) { return units < 4 * device_cu_count(); }

template <int DT>
void quantize(const uint8_t* x, int64_t ldx, int64_t rows, int64_t K, int64_t nslab, uint8_t* codes, uint8_t* scales,
              hipStream_t s) {
  const unsigned units = (unsigned)((rows + 31) / 32 * nslab);
  if (few_units(units))
    hipLaunchKernelGGL((mx_quantize_kernel<DT, 1024>), dim3(units), dim3(1024), 0, s, x, ldx, rows, K, nslab, codes,
                       scales);
  else
    hipLaunchKernelGGL((mx_quantize_kernel<DT, 256>), dim3(units), dim3(256), 0, s, x, ldx, rows, K, nslab, codes,
                       scales);
}

template <int DT>
void dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, int64_t nslab, void* Y,
                int64_t ldy, hipStream_t s) {
  const unsigned units = (unsigned)((rows + 31) / 32 * nslab);
  if (few_units(units))
    hipLaunchKernelGGL((mx_dequantize_kernel<DT, 1024>), dim3(units), dim3(1024), 0, s, codes, scales, rows, K, nslab,
                       Y, ldy);
  else
    hipLaunchKernelGGL((mx_dequantize_kernel<DT, 256>), dim3(units), dim3(256), 0, s, codes, scales, rows, K, nslab, Y,
                       ldy);
}

}  // namespace

hipError_t launch_mx_quantize(const void* X, int64_t ldx, int xdt, int64_t rows, int64_t K, uint8_t* codes,
                              uint8_t* scales, hipStream_t s) {
  const int64_t nslab = mx_kp(K) / kMxSlab;
  const uint8_t* x = static_cast<const uint8_t*>(X);
  auto f = xdt == NM_F16 ? quantize<NM_F16> : xdt == NM_BF16 ? quantize<NM_BF16> : quantize<NM_F32>;
  f(x, ldx, rows, K, nslab, codes, scales, s);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, void* Y,
                                int64_t ldy, int ydt, hipStream_t s) {
  const int64_t nslab = mx_kp(K) / kMxSlab;
  auto f = ydt == NM_F16 ? dequantize<NM_F16> : ydt == NM_BF16 ? dequantize<NM_BF16> : dequantize<NM_F32>;
  f(codes, scales, rows, K, nslab, Y, ldy, s);
  return hipGetLastError();
}

}  // namespace nm
