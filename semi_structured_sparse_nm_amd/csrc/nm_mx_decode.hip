// Microscaled 4-bit product and gated block for few tokens: the weights'
// codes are streamed once from HBM for every tile of 16 NT tokens.
//
// A workgroup owns 16 weight rows (of both weights for the gated block); its
// waves take every NW-th slab of 256 columns, so a wave reads whole 128-byte
// lines of each row.  Up to 16 tokens that come as 16- or 32-bit values, in
// rows of any alignment, are quantised on the way (one launch in all): a wave
// reads its slab of a token pair in one 1 KB load, four lanes share a block as
// in the quantiser, and codes and scales pass through the wave's own LDS to the
// lanes of the scaled matrix instruction.  (Each lane reading the block it
// needs itself touches 64 pieces of 64 bytes a load: 20 us instead of 14 for
// 11008 x 4096, 16 tokens, on the same weights in every call; 15 on others.)
// More tokens come quantised, whole lines of eight tokens a load, and change
// to the instruction's order in the wave's LDS likewise (gated block of 11008 x
// 4096, 64 tokens: 24.4 us in that order from the caches, 17.6 so).  The waves'
// sums meet in LDS, added in wave order.
#include "nm_mx_device.hpp"
#include "nm_mx_lanes.hpp"

namespace nm {

namespace {

constexpr int kMxWaves = 8;

#if defined(__HIP_DEVICE_COMPILE__)
template <int OA, int OB>
__device__ __forceinline__ v4f mx_mul(v4i a, v4i b, v4f c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v8i{a[0], a[1], a[2], a[3], 0, 0, 0, 0},
                                                          v8i{b[0], b[1], b[2], b[3], 0, 0, 0, 0}, c, 4, 4, OA, sa,
                                                          OB, sb);
}
#endif

#if defined(__HIP_DEVICE_COMPILE__)
// ND dwords without their first `bytes` (zeros follow; 32: all of them)
template <int ND>
__device__ __forceinline__ void drop_front(uint32_t (&x)[ND], int bytes) {
#pragma unroll
  for (int w = 16; w >= 4; w /= 2)
#pragma unroll
    for (int i = 0; i < ND; ++i) {
      const uint32_t y = i + w / 4 < ND ? x[i + w / 4] : 0u;
      x[i] = bytes & w ? y : x[i];
    }
#pragma unroll
  for (int i = 0; i < ND; ++i) {
    const uint32_t hi = i + 1 < ND ? x[i + 1] : 0u;
    if (bytes & 2) x[i] = x[i] >> 16 | hi << 16;
    if (bytes & 32) x[i] = 0;
  }
}
#endif

// XDT: type of the activations quantised here (NT = 1), or -1: xcodes.  ANY:
// their rows start anywhere or end inside a 16-byte piece.  NW: waves the slabs
// are dealt to.
template <int XDT, bool GLU, int NT, int NW, bool ANY = false>
__global__ void __launch_bounds__(NW * 64) mx_decode_kernel(MxDecodeArgs a, int nslab, int groups) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NWT = GLU ? 2 : 1;                     // weights
  constexpr bool Q = XDT >= 0;
  constexpr int EB = XDT == NM_F32 ? 4 : 2;
  constexpr int ND = 2 * EB;                           // dwords of eight values
  static_assert(!Q || NT == 1, "activations are quantised here for one token tile");
  // a wave's slab of activations: 128 bytes of every token (16-byte piece c of
  // token t at c ^ (t % 8)), and where it is quantised here two scales a token
  // and lane group; then its sums
  constexpr int XBYTES = NT * 2048 + (Q ? 16 * 8 : 0), RBYTES = NWT * NT * 1024;
  __shared__ __attribute__((aligned(16))) uint8_t buf[NW][XBYTES > RBYTES ? XBYTES : RBYTES];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, lq = lane >> 4;
  // workgroups 8 apart (neighbours on their XCD) take the token groups of one row block
  const int b = blockIdx.x >> 3, q8 = __builtin_amdgcn_readfirstlane(b / groups);
  const int64_t rb = q8 * 8 + (blockIdx.x & 7);
  const int64_t t0 = (b - q8 * groups) * (16 * NT);
  if (rb * 16 >= a.R) return;
  const int64_t ldc = (int64_t)nslab * 128;

  const int64_t row = min(rb * 16 + li, a.R - 1);      // rows past R: the last one again, not stored
  const uint8_t* wc[NWT];
  const uint8_t* wsc[NWT];
#pragma unroll
  for (int w = 0; w < NWT; ++w) {
    wc[w] = a.codes[w] + row * ldc + 16 * lq;
    wsc[w] = a.scales[w] + (rb / 2) * (int64_t)nslab * 256 + 4 * lane;
  }
  const int wsh = 16 * (int)(rb & 1);                  // this 16-row half's two scales of each word

  // activations to quantise: lane 32 h + p takes values 8 p .. of the slab of
  // token 2 i + h.  Tokens past T repeat the last (what they give is not used);
  // columns past K are zeroed in registers
  const int hx = lane >> 5, px = lane & 31;
  const int tn = Q ? (int)min(a.T - t0, (int64_t)16) : 0;
  const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(Q ? static_cast<const uint8_t*>(a.X) + t0 * a.ldx * EB : a.xcodes), 0, 0x7fffffff,
      0x00020000);
  const int kbytes = (int)a.K * EB, pitch = (int)a.ldx * EB;
  uint8_t* const qw = buf[wave];
  // quantised activations: load h brings tokens 8 h .. 8 h + 7, lane l piece
  // l % 8 of token 8 h + l / 8; tokens past the last repeat it (not stored)
  const uint8_t* xc[2 * NT];
#pragma unroll
  for (int h = 0; h < 2 * NT; ++h)
    xc[h] = Q ? nullptr : a.xcodes + min(t0 + 8 * h + (lane >> 3), a.T - 1) * ldc + 16 * (lane & 7);
  const int put = (lane >> 3) * 128 + 16 * ((lane & 7) ^ (lane >> 3));

  v4f acc[NWT][NT];
#pragma unroll
  for (int w = 0; w < NWT; ++w)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[w][j] = v4f{0.f, 0.f, 0.f, 0.f};

  for (int s = wave; s < nslab; s += NW) {
    v4i fw[NWT][2];
    int sw[NWT];
#pragma unroll
    for (int w = 0; w < NWT; ++w) {
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) fw[w][kk] = *reinterpret_cast<const v4i*>(wc[w] + (int64_t)s * 128 + 64 * kk);
      sw[w] = (int)(*reinterpret_cast<const uint32_t*>(wsc[w] + (int64_t)s * 256) >> wsh);
    }
    v4i fx[NT][2];
    int sx[NT];
    if constexpr (Q) {
      const int so = __builtin_amdgcn_readfirstlane(s * 256 * EB);
      // two token pairs at a time, as many as there are tokens (four at a time
      // cost registers: 11.4 us instead of 10.6 for one token of the gated block)
      for (int i0 = 0; i0 < tn; i0 += 4) {
        uint32_t x[2][ND];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if constexpr (ANY) {
            const int t = i0 + 2 * u + hx;
            // a row's short last piece as its last eight values, shifted; all
            // lanes read inside their row
            const int64_t k = (int64_t)s * 256 + px * 8;
            const uint8_t* p =
                static_cast<const uint8_t*>(a.X) + (min(t0 + t, a.T - 1) * a.ldx + min(k, a.K - 8)) * EB;
#pragma unroll
            for (int i = 0; i < ND / 4; ++i) {
              const v4i v = load16(p + 16 * i);
#pragma unroll
              for (int e = 0; e < 4; ++e) x[u][4 * i + e] = (uint32_t)v[e];
            }
            if (s == nslab - 1) drop_front<ND>(x[u], k < a.K ? max((int)(k + 8 - a.K), 0) * EB : 32);
            if (t >= tn)
#pragma unroll
              for (int i = 0; i < ND; ++i) x[u][i] = 0;
            continue;
          }
#pragma unroll
          for (int i = 0; i < ND / 4; ++i) {
            const int off = mx_lane_offset<EB>(lane, i0 + 2 * u, i, tn, pitch, so, kbytes);
            const v4i v = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rx, off, so, 0));
#pragma unroll
            for (int e = 0; e < 4; ++e) x[u][4 * i + e] = (uint32_t)v[e];
          }
        }
        if (!ANY && so + 256 * EB > kbytes) {            // the row's last slab, short
#pragma unroll
          for (int i = 0; i < ND; ++i)
            if (!mx_lane_inside<EB>(lane, i / 4, so, kbytes)) x[0][i] = x[1][i] = 0;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int t = (i0 + 2 * u + hx) & 15;
          const uint32_t m = quad_max(mx_amax8<XDT>(x[u]));
          // (a NaN scale makes every product NaN whatever the codes)
          const uint32_t byte = mx_scale_byte(m);
          *reinterpret_cast<uint32_t*>(qw + t * 128 + 16 * ((px >> 2) ^ (t & 7)) + 4 * (px & 3)) =
              mx_codes8<XDT>(x[u], mx_scale_f32(byte));
          if ((px & 3) == 0) qw[16 * 128 + t * 8 + 2 * ((px >> 2) & 3) + (px >> 4)] = (uint8_t)byte;
        }
      }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const v4i v = *reinterpret_cast<const v4i*>(qw + li * 128 + 16 * ((4 * kk + lq) ^ (li & 7)));
        fx[0][kk] = li < tn ? v : v4i{0, 0, 0, 0};
      }
      sx[0] = li < tn ? (int)*reinterpret_cast<const uint16_t*>(qw + 16 * 128 + li * 8 + 2 * lq) : 0;
      __builtin_amdgcn_wave_barrier();
    } else {
      v4i x[2 * NT];
#pragma unroll
      for (int h = 0; h < 2 * NT; ++h) x[h] = *reinterpret_cast<const v4i*>(xc[h] + (int64_t)s * 128);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        // token tile t0 / 16 + j: half of the scale unit of its 32 tokens
        const int64_t tt = t0 / 16 + j;
        const int64_t unit = min(tt / 2, (a.T - 1) / 32);
        sx[j] = (int)(*reinterpret_cast<const uint32_t*>(a.xscales + (unit * nslab + s) * 256 + 4 * lane) >>
                      (16 * (int)(tt & 1)));
      }
#pragma unroll
      for (int h = 0; h < 2 * NT; ++h) *reinterpret_cast<v4i*>(qw + 1024 * h + put) = x[h];
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
          fx[j][kk] = *reinterpret_cast<const v4i*>(qw + 2048 * j + li * 128 + 16 * ((4 * kk + lq) ^ (li & 7)));
      __builtin_amdgcn_wave_barrier();
    }
#pragma unroll
    for (int w = 0; w < NWT; ++w)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        acc[w][j] = mx_mul<0, 0>(fw[w][0], fx[j][0], acc[w][j], sw[w], sx[j]);
        acc[w][j] = mx_mul<1, 1>(fw[w][1], fx[j][1], acc[w][j], sw[w], sx[j]);
      }
  }
  v4f(*const sum)[64] = reinterpret_cast<v4f(*)[64]>(qw);   // this wave's own reads of it are done
#pragma unroll
  for (int w = 0; w < NWT; ++w)
#pragma unroll
    for (int j = 0; j < NT; ++j) sum[w * NT + j][lane] = acc[w][j];
  __syncthreads();
  for (int q = threadIdx.x; q < 256 * NT; q += NW * 64) {
    const int rr = q & 15, tok = q >> 4;
    const int ln = 16 * (rr >> 2) + (tok & 15), v = rr & 3, j = tok >> 4;
    float y[NWT];
#pragma unroll
    for (int w = 0; w < NWT; ++w) {
      y[w] = 0.f;
#pragma unroll
      for (int p = 0; p < NW; ++p) y[w] += reinterpret_cast<const float*>(buf[p] + ((w * NT + j) * 64 + ln) * 16)[v];
    }
    const int64_t r = rb * 16 + rr, t = t0 + tok;
    if (r < a.R && t < a.T) {
      float o;
      if constexpr (GLU) {
        o = glu_act(a.act, y[0]) * y[NWT - 1];
      } else {
        o = y[0];
        if (a.bias) o += a.bias[r];
        if (a.act == NM_ACT_GELU) o = gelu_f32(o);
      }
      const int64_t at = t * a.ldy + r;
      if (a.ydt == NM_F32)
        static_cast<float*>(a.Y)[at] = o;
      else if (a.ydt == NM_F16)
        static_cast<uint16_t*>(a.Y)[at] = (uint16_t)pack_16x2<NM_F16>(o, 0.f);
      else
        static_cast<uint16_t*>(a.Y)[at] = (uint16_t)pack_16x2<NM_BF16>(o, 0.f);
    }
  }
#endif
}

template <bool GLU, int NW, int XDT>
void launch_quantising(const MxDecodeArgs& a, int nslab, dim3 grid, hipStream_t s) {
  constexpr int EB = XDT == NM_F32 ? 4 : 2;
  // 16-byte pieces within 32-bit offsets
  if ((uintptr_t)a.X % 16 == 0 && a.ldx * EB % 16 == 0 && a.K * EB % 16 == 0 && a.ldx * EB < (1 << 26))
    hipLaunchKernelGGL((mx_decode_kernel<XDT, GLU, 1, NW>), grid, dim3(NW * 64), 0, s, a, nslab, 1);
  else
    hipLaunchKernelGGL((mx_decode_kernel<XDT, GLU, 1, NW, true>), grid, dim3(NW * 64), 0, s, a, nslab, 1);
}

template <bool GLU, int NW>
hipError_t launch_one_tile(const MxDecodeArgs& a, int nslab, unsigned nrb, hipStream_t s) {
  const dim3 grid((nrb + 7) / 8 * 8);
  if (!a.X)
    hipLaunchKernelGGL((mx_decode_kernel<-1, GLU, 1, NW>), grid, dim3(NW * 64), 0, s, a, nslab, 1);
  else if (a.xdt == NM_F16)
    launch_quantising<GLU, NW, NM_F16>(a, nslab, grid, s);
  else if (a.xdt == NM_BF16)
    launch_quantising<GLU, NW, NM_BF16>(a, nslab, grid, s);
  else
    launch_quantising<GLU, NW, NM_F32>(a, nslab, grid, s);
  return hipGetLastError();
}

template <bool GLU>
hipError_t launch_decode(const MxDecodeArgs& a, hipStream_t s) {
  const int nslab = (int)(mx_kp(a.K) / kMxSlab);
  const unsigned nrb = (unsigned)((a.R + 15) / 16);
  constexpr int NW = kMxWaves;
  if (a.T <= 16) {
    // one workgroup or less a CU: sixteen waves keep more of the weight in
    // flight (4096 x 11008, one token: 8.8 us against 11.2 with eight)
    if (nrb <= (unsigned)device_cu_count() && nslab > NW) return launch_one_tile<GLU, 16>(a, nslab, nrb, s);
    return launch_one_tile<GLU, NW>(a, nslab, nrb, s);
  }
  const int nt = stream_tiles(nrb, a.T);
  const int groups = (int)((a.T + 16 * nt - 1) / (16 * nt));
  const dim3 grid((nrb + 7) / 8 * 8 * groups), block(NW * 64);
  if (nt == 1)
    hipLaunchKernelGGL((mx_decode_kernel<-1, GLU, 1, NW>), grid, block, 0, s, a, nslab, groups);
  else if (nt == 2)
    hipLaunchKernelGGL((mx_decode_kernel<-1, GLU, 2, NW>), grid, block, 0, s, a, nslab, groups);
  else
    hipLaunchKernelGGL((mx_decode_kernel<-1, GLU, 4, NW>), grid, block, 0, s, a, nslab, groups);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_decode(const MxDecodeArgs& a, hipStream_t s) {
  return a.glu ? launch_decode<true>(a, s) : launch_decode<false>(a, s);
}

}  // namespace nm
