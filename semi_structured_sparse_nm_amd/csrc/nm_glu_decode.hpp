// Gated block for few tokens: H = act(X Wg^T) (.) (X Wu^T), both packed
// weights streamed once from HBM for every tile of 16 NT tokens.
//
// With so few tokens the bound is the packed weights' bytes.  A workgroup
// owns one 16-row block of both weights; its NW waves take every NW-th
// 64-column block, so they read neighbouring blocks at a time, straight to
// registers (a fragment of a packed block is one contiguous run), U blocks
// of both weights in flight per wave.  2:4 windows go to the sparse matrix
// instruction as they are; other patterns are expanded in registers for the
// dense one.  The waves' sums meet in LDS, added in wave order.
//
// Activations come from the caches, 128 bytes of eight tokens a load, and
// change to the matrix instruction's order in the wave's own LDS.  (Loaded in
// that order, 16 bytes of each of 16 tokens for every quarter of a load, they
// pass the vector cache at a quarter of its rate, which bound the call: two
// 4:8 weights of 11008 x 4096, the same in every call, 16 tokens 22 us against
// 19 now, 32 tokens 33 and 23, 64 tokens 60 and 33; with weights that change
// between calls 16 tokens take 24.)  At 64 tokens one block in flight leaves the
// registers for two workgroups on a compute unit (two: 37 us, one workgroup).
//
// Expansion of 1 to 4 kept of 8: the kept values of a group are at most two
// registers, so each of its four dense registers is one byte permute of them.
// The permutes' selectors depend only on which columns are kept: a table in
// LDS, 16 bytes for each of the 256 sets of columns, read by the set's bits.
// (Shifting each value to its place takes about three times the vector
// instructions, which would bound the call: 4:8, 16 tokens, 11008 x 4096 31 us.)
#pragma once

#include "nm_expand.hpp"
#include "nm_ffn.hpp"

namespace nm {

namespace {

typedef _Float16 v16h_ __attribute__((ext_vector_type(16)));
typedef __bf16 v16bf_ __attribute__((ext_vector_type(16)));

template <int WT>
__device__ __forceinline__ v4f smfmac24(v4i a, v8i b, v4f c, int idx) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (WT == NM_F16)
    return __builtin_amdgcn_smfmac_f32_16x16x64_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v16h_, b), c, idx,
                                                    0, 0);
  else
    return __builtin_amdgcn_smfmac_f32_16x16x64_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v16bf_, b), c,
                                                     idx, 0, 0);
#else
  return c;
#endif
}

constexpr int kGluWaves = 8;

// One lane's part of one packed block (64 dense columns).
template <int WT, int N, int M>
struct GluFrag {
  typedef Run<WT, N, M> RunT;
  static constexpr bool SPARSE = N == 2 && M == 4;
  static constexpr bool TABLE = M == 8 && N <= 4;
  uint32_t vd[RunT::VD];
  uint64_t mb;
  __device__ __forceinline__ void load(const uint8_t* values, const uint8_t* meta, int64_t blk, int li, int lg) {
    const uint8_t* v = values + blk * (16 * RunT::C_B) + li * RunT::C_B + lg * RunT::VB;
#pragma unroll
    for (int i = 0; i < RunT::VD; ++i) vd[i] = reinterpret_cast<const uint32_t*>(v)[i];
    mb = 0;
    if constexpr (N != M) {
      const uint8_t* m = meta + blk * (16 * RunT::MRB) + li * RunT::MRB;
      if constexpr (SPARSE) {
        mb = *reinterpret_cast<const uint16_t*>(m + 2 * lg);
      } else {
        int dw, sh;
        RunT::meta_window(lg, dw, sh);
        const uint32_t* mw = reinterpret_cast<const uint32_t*>(m);
        mb = mw[dw];
        if (RunT::MRB >= 8) mb |= (uint64_t)mw[dw + 1] << 32;
        mb >>= sh;
        // 7:8 (42 bits a lane): lane group 3 starts at bit 30 of its dword
        // and needs a third one (every group's third dword is in the row)
        if constexpr (RunT::MBL > 36) {
          static_assert(RunT::MRB >= 24, "three dwords from every window's first");
          if (sh) mb |= (uint64_t)mw[dw + 2] << (64 - sh);
        }
      }
    }
  }
  // group q (of the lane's two) of eight columns, expanded
  __device__ __forceinline__ v4i group(int q, const v4i* table) const {
#if defined(__HIP_DEVICE_COMPILE__)
    uint32_t set = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) set |= 1u << ((uint32_t)(mb >> (3 * (q * N + j))) & 7u);
    // the group's kept values: halves q N .. + N - 1 of the run
    uint32_t lo, hi = 0;
    if constexpr (N == 4) {
      lo = vd[2 * q];
      hi = vd[2 * q + 1];
    } else if constexpr (N == 3) {
      lo = q ? (uint32_t)__builtin_amdgcn_alignbit(vd[2], vd[1], 16) : vd[0];
      hi = q ? vd[2] >> 16 : vd[1];
    } else if constexpr (N == 2) {
      lo = vd[q];
    } else {
      lo = vd[0] >> (16 * q);
    }
    const v4i sel = table[set];
    v4i o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (int)__builtin_amdgcn_perm(hi, lo, (uint32_t)sel[i]);
    return o;
#else
    return v4i{};
#endif
  }
  // x: the lane's 16 activations, as the two 16-byte pieces the product wants
  __device__ __forceinline__ v4f mul(v4i x0, v4i x1, v4f c, const v4i* table) const {
    if constexpr (TABLE) {
#if defined(__HIP_DEVICE_COMPILE__)
      c = mfma_dense<WT>(group(0, table), x0, c);
      return mfma_dense<WT>(group(1, table), x1, c);
#else
      return c;
#endif
    } else if constexpr (SPARSE) {
      const v4i a = {(int)vd[0], (int)vd[1], (int)vd[2], (int)vd[3]};
      return smfmac24<WT>(a, v8i{x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]}, c, (int)mb);
    } else {
#if defined(__HIP_DEVICE_COMPILE__)
      c = mfma_dense<WT>(expand_step<WT, N, M, 0>(vd, mb), x0, c);
      return mfma_dense<WT>(expand_step<WT, N, M, 1>(vd, mb), x1, c);
#else
      return c;
#endif
    }
  }
  // first column of each piece within the block: the sparse instruction's
  // second operand holds k = 8 lg .. and 32 + 8 lg .., the dense steps the
  // halves of the lane's run of 16
  __device__ static int kpiece(int p, int lg) { return SPARSE ? 32 * p + 8 * lg : 16 * lg + 8 * p; }
};

// SHORT: K is no multiple of eight (groups of four only).
template <int WT, int N, int M, int NT, bool SHORT>
__global__ void __launch_bounds__(kGluWaves * 64) glu_decode_kernel(GluArgs a, int groups) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NW = kGluWaves;
  constexpr int U = NT == 1 ? 4 : NT == 2 ? 2 : 1;
  typedef GluFrag<WT, N, M> Frag;
  // a wave's activations of one block, then its sums
  __shared__ __attribute__((aligned(16))) v4f red[NW][2 * NT][64];
  __shared__ __attribute__((aligned(16))) v4i table[Frag::TABLE ? 256 : 1];
  if constexpr (Frag::TABLE) {
    // column c of set s: bytes 2 k, 2 k + 1 of the kept values where it is
    // the set's k-th (from 0), else zeros (selector 12)
    for (int q = threadIdx.x; q < 1024; q += NW * 64) {
      const int s = q >> 2, c = 2 * (q & 3);
      uint32_t sel = 0;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int k = __builtin_popcount(s & ((1 << (c + e)) - 1));
        const uint32_t b = (s >> (c + e) & 1) && k < 4 ? (uint32_t)((2 * k + 1) << 8 | 2 * k) : 0x0C0Cu;
        sel |= b << (16 * e);
      }
      reinterpret_cast<uint32_t*>(table)[q] = sel;
    }
    __syncthreads();
  }
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, lg = lane >> 4;
  // workgroups 8 apart (neighbours on their XCD) take the token groups of one row block
  const int b = blockIdx.x >> 3, q8 = __builtin_amdgcn_readfirstlane(b / groups);
  const int64_t rb = q8 * 8 + (blockIdx.x & 7);
  const int64_t t0 = (b - q8 * groups) * (16 * NT);
  if (rb >= a.g.nRB) return;
  const int nKB = (int)a.g.nKB;
  const int K = (int)a.g.K;

  // activations: load h of token tile j brings rows 8 h .. 8 h + 7 of it, lane l
  // piece l % 8 (eight columns) of row 8 h + l / 8; tokens past the last
  // repeat it (their results are not stored)
  // A row's last piece may hold fewer than eight columns: it is read as the
  // row's last eight and shifted, so nothing past the row is read.
  const int piece = lane & 7;
  const int short_by = SHORT ? 8 - (K & 7) : 0;        // columns its last piece lacks
  const uint16_t* xr[NT][2];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      xr[j][h] = static_cast<const uint16_t*>(a.X) + min(t0 + 16 * j + 8 * h + (lane >> 3), a.T - 1) * a.ldx + 8 * piece;
  uint8_t* const xs = reinterpret_cast<uint8_t*>(&red[wave][0][0]);
  const int put = (lane >> 3) * 128 + 16 * (piece ^ (lane >> 3));
  const int get0 = li * 128 + 16 * ((Frag::kpiece(0, lg) >> 3) ^ (li & 7));
  const int get1 = li * 128 + 16 * ((Frag::kpiece(1, lg) >> 3) ^ (li & 7));
  v4f ag[NT], au[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) ag[j] = au[j] = v4f{0.f, 0.f, 0.f, 0.f};

  for (int b0 = wave; b0 < nKB; b0 += NW * U) {
    Frag fg[U], fu[U];
    v4i x[U][NT][2];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int kb = min(b0 + NW * i, nKB - 1);        // past the end: a block read again, not used
      fg[i].load(a.values[0], a.meta[0], rb * nKB + kb, li, lg);
      fu[i].load(a.values[1], a.meta[1], rb * nKB + kb, li, lg);
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = kb * 64 + 8 * piece;
          x[i][j][h] = v4i{0, 0, 0, 0};
          if (k < K) x[i][j][h] = load16(xr[j][h] + kb * 64 - (SHORT && k + 8 > K ? short_by : 0));
        }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (b0 + NW * i < nKB) {
        if (SHORT && b0 + NW * i == nKB - 1) {
          const bool last = (b0 + NW * i) * 64 + 8 * piece + 8 > K;
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) x[i][j][h] = last ? shift_out(x[i][j][h], short_by) : x[i][j][h];
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) *reinterpret_cast<v4i*>(xs + 2048 * j + 1024 * h + put) = x[i][j][h];
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const v4i x0 = *reinterpret_cast<const v4i*>(xs + 2048 * j + get0);
          const v4i x1 = *reinterpret_cast<const v4i*>(xs + 2048 * j + get1);
          ag[j] = fg[i].mul(x0, x1, ag[j], table);
          au[j] = fu[i].mul(x0, x1, au[j], table);
        }
        __builtin_amdgcn_wave_barrier();
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    red[wave][2 * j][lane] = ag[j];
    red[wave][2 * j + 1][lane] = au[j];
  }
  __syncthreads();
  for (int q = threadIdx.x; q < 256 * NT; q += NW * 64) {
    const int row = q & 15, tok = q >> 4;              // token tok % 16 of tile tok / 16
    const int ln = 16 * (row >> 2) + (tok & 15), v = row & 3, j = tok >> 4;
    float g = 0.f, u = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      g += reinterpret_cast<const float*>(&red[w][2 * j][ln])[v];
      u += reinterpret_cast<const float*>(&red[w][2 * j + 1][ln])[v];
    }
    const int64_t r = rb * 16 + row, t = t0 + tok;
    if (r < a.g.R && t < a.T) {
      const float h = glu_act(a.act, g) * u;
      static_cast<uint16_t*>(a.H)[t * a.ldh + r] = (uint16_t)pack_16x2<WT>(h, 0.f);
      if (a.P[0] && a.p32) {
        static_cast<float*>(a.P[0])[t * a.ldp + r] = g;
        static_cast<float*>(a.P[1])[t * a.ldp + r] = u;
      } else if (a.P[0]) {
        static_cast<uint16_t*>(a.P[0])[t * a.ldp + r] = (uint16_t)pack_16x2<WT>(g, 0.f);
        static_cast<uint16_t*>(a.P[1])[t * a.ldp + r] = (uint16_t)pack_16x2<WT>(u, 0.f);
      }
    }
  }
#endif
}

template <int WT, int N, int M, bool SHORT>
hipError_t launch_glu_decode_rows(const GluArgs& a, hipStream_t s) {
  const int nt = stream_tiles(a.g.nRB, a.T);
  const int groups = (int)((a.T + 16 * nt - 1) / (16 * nt));
  const dim3 grid((unsigned)((a.g.nRB + 7) / 8 * 8 * groups)), block(kGluWaves * 64);
  if (nt == 1)
    hipLaunchKernelGGL((glu_decode_kernel<WT, N, M, 1, SHORT>), grid, block, 0, s, a, groups);
  else if (nt == 2)
    hipLaunchKernelGGL((glu_decode_kernel<WT, N, M, 2, SHORT>), grid, block, 0, s, a, groups);
  else
    hipLaunchKernelGGL((glu_decode_kernel<WT, N, M, 4, SHORT>), grid, block, 0, s, a, groups);
  return hipGetLastError();
}

template <int WT, int N, int M>
hipError_t launch_glu_decode_nm(const GluArgs& a, hipStream_t s) {
  if constexpr (M == 4)
    if (a.g.K % 8) return launch_glu_decode_rows<WT, N, M, true>(a, s);
  return launch_glu_decode_rows<WT, N, M, false>(a, s);
}

template <int WT>
hipError_t launch_glu_decode_wt(const GluArgs& a, hipStream_t s) {
  switch (a.g.M * 16 + a.g.N) {
    case 4 * 16 + 1: return launch_glu_decode_nm<WT, 1, 4>(a, s);
    case 4 * 16 + 2: return launch_glu_decode_nm<WT, 2, 4>(a, s);
    case 4 * 16 + 3: return launch_glu_decode_nm<WT, 3, 4>(a, s);
    case 4 * 16 + 4: return launch_glu_decode_nm<WT, 4, 4>(a, s);
    case 8 * 16 + 1: return launch_glu_decode_nm<WT, 1, 8>(a, s);
    case 8 * 16 + 2: return launch_glu_decode_nm<WT, 2, 8>(a, s);
    case 8 * 16 + 3: return launch_glu_decode_nm<WT, 3, 8>(a, s);
    case 8 * 16 + 4: return launch_glu_decode_nm<WT, 4, 8>(a, s);
    case 8 * 16 + 5: return launch_glu_decode_nm<WT, 5, 8>(a, s);
    case 8 * 16 + 6: return launch_glu_decode_nm<WT, 6, 8>(a, s);
    case 8 * 16 + 7: return launch_glu_decode_nm<WT, 7, 8>(a, s);
    case 8 * 16 + 8: return launch_glu_decode_nm<WT, 8, 8>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

}  // namespace nm
