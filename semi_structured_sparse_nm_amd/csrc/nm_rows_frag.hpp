// One lane's part of a packed block as an operand of the matrix instructions,
// for the products of grouped rows.
#pragma once

#include "nm_expand.hpp"
#include "nm_glu_decode.hpp"
#include "nm_rows.hpp"

namespace nm {

namespace {

#if defined(__HIP_DEVICE_COMPILE__)
template <int WT>
using acc_of = typename std::conditional<WT == NM_I8, v4i, v4f>::type;

// One lane's positions in a packed block row of MRB bytes: MBL bits from bit lg
// MBL on, brought by one load of ML dwords from the byte they begin in (a load of
// its own for every dword would cost the vector memory path as much as 1 KB of
// values), or, where that would leave the row, from the row's last ML dwords.
template <int MBL, int MRB>
struct Positions {
  static constexpr int MD = (MBL + 31) / 32;           // dwords they fill
  static constexpr int ML = (MBL + (MBL % 8 == 0 ? 0 : MBL % 4 == 0 ? 4 : 6) + 31) / 32;
  static_assert(4 * ML <= MRB, "inside the row");
  uint32_t w[ML];
  struct __attribute__((packed, aligned(1))) Words {
    uint32_t w[ML];
  };
  __device__ static __forceinline__ int first(int lg) { return min(lg * MBL >> 3, MRB - 4 * ML); }
  // m: the block's positions (the same in all lanes)
  __device__ __forceinline__ void load(const uint8_t* m, int li, int lg) {
    const Words v = *reinterpret_cast<const Words*>(m + (uint32_t)(li * MRB + first(lg)));
#pragma unroll
    for (int i = 0; i < ML; ++i) w[i] = v.w[i];
  }
  // from bit 0 of b
  __device__ __forceinline__ void align(int lg, uint32_t (&b)[MD]) const {
    const int sh = lg * MBL - 8 * first(lg);           // below 32
#pragma unroll
    for (int i = 0; i < MD; ++i) b[i] = i + 1 < ML ? __builtin_amdgcn_alignbit(w[i + 1], w[i], sh) : w[i] >> sh;
  }
};
template <int MRB>
struct Positions<0, MRB> {
  static constexpr int MD = 1;
  __device__ __forceinline__ void load(const uint8_t*, int, int) {}
  __device__ __forceinline__ void align(int, uint32_t (&)[1]) const {}
};

// The set of kept columns, a bit each, of eight columns whose positions begin at
// bit 0 of pos: one group of 8, or two of 4.
template <int N, int M>
__device__ __forceinline__ uint32_t kept_set(uint32_t pos) {
  constexpr int W = M == 4 ? 2 : 3;
  uint32_t set = 0;
#pragma unroll
  for (int j = 0; j < 8 * N / M; ++j) set |= (j < N ? 1u : 16u) << (pos >> (W * j) & (M - 1));
  return set;
}

// One lane's part of one packed block of 8-bit weights (128 dense columns, a
// run of 32 a lane): load brings it as it is stored, so that nothing waits for it
// there; ready gives the operands of the block's product, a0 and a1 the dense ones
// of its two steps, or (2:4) the packed values and, in a1[0], their positions, with
// the table as fill_table leaves it.  Eight columns hold at most
// two registers of kept values, so each of their two dense registers is one byte
// permute of them, by the table of selectors.
template <int N, int M>
struct I8Frag {
  static constexpr bool SPARSE = N == 2 && M == 4;
  static constexpr int KEPT = 8 * N / M;               // of eight columns
  static constexpr bool TABLE = !SPARSE && N < M && (M == 8 || N == 3);
  static constexpr int W = N == M ? 0 : M == 4 ? 2 : 3;
  static constexpr int VB = 32 * N / M, VD = VB / 4;   // bytes, dwords of the run's values
  static constexpr int MBL = VB * W;                   // bits of its positions
  static constexpr int MRB = (4 * MBL + 31) / 32 * 4;  // bytes of a block row's positions
  static constexpr int VBLK = 64 * VB, MBLK = 16 * MRB;   // bytes of a block
  typedef Positions<MBL, MRB> Pos;
  static constexpr int MD = Pos::MD;
  uint32_t vd[VD];
  Pos pos;
  // v, m: the block's values and positions (the same in all lanes)
  __device__ __forceinline__ void load(const uint8_t* v, const uint8_t* m, int li, int lg) {
    const uint32_t at = (uint32_t)(li * (4 * VB) + lg * VB);
#pragma unroll
    for (int i = 0; i < VD; ++i) vd[i] = *reinterpret_cast<const uint32_t*>(v + at + 4 * i);
    pos.load(m, li, lg);
  }
  // bits b .. b + 23 and more of the positions mb, b known when compiled
  __device__ static __forceinline__ uint32_t positions(const uint32_t* mb, int b) {
    const int d = b >> 5, sh = b & 31;
    return d + 1 < MD ? __builtin_amdgcn_alignbit(mb[d + 1], mb[d], sh) : mb[d] >> sh;
  }
  // the run's bytes b .. b + 3 (zeros behind the run)
  __device__ __forceinline__ uint32_t bytes(int b) const {
    const int d = b >> 2, sh = b & 3;
    return d >= VD ? 0u : __builtin_amdgcn_alignbyte(d + 1 < VD ? vd[d + 1] : 0u, vd[d], sh);
  }
  // columns 8 q .. + 7 of the lane's 32, expanded
  __device__ __forceinline__ v2i group(const uint32_t* mb, int q, const v2i* table) const {
    const v2i sel = table[kept_set<N, M>(positions(mb, KEPT * W * q))];
    const uint32_t lo = bytes(KEPT * q), hi = KEPT > 4 ? bytes(KEPT * q + 4) : 0u;
    return v2i{(int)__builtin_amdgcn_perm(hi, lo, (uint32_t)sel[0]),
               (int)__builtin_amdgcn_perm(hi, lo, (uint32_t)sel[1])};
  }
  __device__ __forceinline__ void ready(int lg, v4i& a0, v4i& a1, const v2i* table) const {
    uint32_t mb[MD];
    pos.align(lg, mb);
    if constexpr (TABLE) {
      const v2i g0 = group(mb, 0, table), g1 = group(mb, 1, table), g2 = group(mb, 2, table), g3 = group(mb, 3, table);
      a0 = v4i{g0[0], g0[1], g1[0], g1[1]};
      a1 = v4i{g2[0], g2[1], g3[0], g3[1]};
    } else if constexpr (SPARSE) {
      a0 = v4i{(int)vd[0], (int)vd[1], (int)vd[2], (int)vd[3]};
      a1[0] = (int)mb[0];
    } else {
      const uint64_t bits = MD > 1 ? (uint64_t)mb[MD - 1] << 32 | mb[0] : mb[0];
      a0 = expand_step<NM_I8, N, M, 0>(vd, bits);
      a1 = expand_step<NM_I8, N, M, 1>(vd, bits);
    }
  }
  // the two 16-byte pieces (of a row's eight in the block) the product wants
  __device__ static int kpiece(int p, int lg) { return SPARSE ? 4 * p + lg : 2 * lg + p; }
};

// The same of 16-bit weights (64 columns, a run of 16 a lane).  Dense register i of
// eight columns holds columns 2 i and 2 i + 1: with at most four values kept they
// are among the same two registers for every i; with six or seven, column c's is
// one of values c - 2 .. c, so that i's are in two neighbouring registers known
// when compiled.  (Of 5:8 they may be in three: its values are shifted to their
// places one by one, which takes about twice the instructions.)
template <int WT, int N, int M>
struct RowsFrag {
  typedef Run<WT, N, M> RunT;
  typedef v4i Entry;
  static constexpr bool SPARSE = N == 2 && M == 4;
  static constexpr int KEPT = 8 * N / M;               // of eight columns
  static constexpr bool TABLE = !SPARSE && N < M && ((M == 8 && N != 5) || N == 3);
  static constexpr int SLAB = 64;                      // columns of a block
  static constexpr int MBL = RunT::MBL, MRB = RunT::MRB;
  static constexpr int VBLK = 16 * RunT::C_B, MBLK = 16 * MRB;
  typedef Positions<SPARSE ? 0 : MBL, MRB> Pos;
  static constexpr int MD = Pos::MD;
  uint32_t vd[RunT::VD];
  uint32_t idx;                                        // 2:4
  Pos pos;                                             // others
  __device__ __forceinline__ void load(const uint8_t* v, const uint8_t* m, int li, int lg) {
    const uint32_t at = (uint32_t)(li * RunT::C_B + lg * RunT::VB);
#pragma unroll
    for (int i = 0; i < RunT::VD; ++i) vd[i] = *reinterpret_cast<const uint32_t*>(v + at + 4 * i);
    if constexpr (SPARSE) idx = *reinterpret_cast<const uint16_t*>(m + (uint32_t)(li * MRB + 2 * lg));
    else pos.load(m, li, lg);
  }
  // the two 16-byte pieces (of a row's eight in the block) the product wants
  __device__ static int kpiece(int p, int lg) { return SPARSE ? 4 * p + lg : 2 * lg + p; }
  // columns 8 q .. + 7 of the lane's 16, expanded
  __device__ __forceinline__ v4i group(uint64_t mb, int q, const v4i* table) const {
    constexpr int W = M == 4 ? 2 : 3;
    const v4i sel = table[kept_set<N, M>((uint32_t)(mb >> (KEPT * W * q)))];
    // the kept values: halves KEPT q .. of the run
    uint32_t e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int h = KEPT * q + 2 * i, d = h >> 1;
      const uint32_t lo = d < RunT::VD ? vd[d] : 0u, hi = d + 1 < RunT::VD ? vd[d + 1] : 0u;
      e[i] = 2 * i >= KEPT ? 0u : h & 1 ? (uint32_t)__builtin_amdgcn_alignbit(hi, lo, 16) : lo;
    }
    v4i o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = first_source(i);
      o[i] = (int)__builtin_amdgcn_perm(e[b + 1], e[b], (uint32_t)sel[i]);
    }
    return o;
  }
  // register of the kept values from which dense register i's two sources begin
  __host__ __device__ static constexpr int first_source(int i) { return KEPT <= 4 || i < 1 ? 0 : i - 1; }
  __device__ __forceinline__ void ready(int lg, v4i& a0, v4i& a1, const v4i* table) const {
    if constexpr (SPARSE) {
      a0 = v4i{(int)vd[0], (int)vd[1], (int)vd[2], (int)vd[3]};
      a1[0] = (int)idx;
    } else {
      uint32_t w[MD];
      pos.align(lg, w);
      const uint64_t mb = MD > 1 ? (uint64_t)w[MD - 1] << 32 | w[0] : w[0];
      if constexpr (TABLE) {
        a0 = group(mb, 0, table);
        a1 = group(mb, 1, table);
      } else {
        a0 = expand_step<WT, N, M, 0>(vd, mb);
        a1 = expand_step<WT, N, M, 1>(vd, mb);
      }
    }
  }
};
template <int N, int M>
struct RowsFrag<NM_I8, N, M> : I8Frag<N, M> {
  typedef v2i Entry;
  static constexpr int SLAB = 128;
};

// x0, x1: the lane's 32 bytes of activations, as the pieces kpiece names
template <int WT, bool SPARSE>
__device__ __forceinline__ acc_of<WT> rows_mul(v4i a0, v4i a1, v4i x0, v4i x1, acc_of<WT> c) {
  if constexpr (SPARSE) {
    const v8i x = __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7);
    if constexpr (WT == NM_I8) return __builtin_amdgcn_smfmac_i32_16x16x128_i8(a0, x, c, a1[0], 0, 0);
    else return smfmac24<WT>(a0, x, c, a1[0]);
  } else {
    return mfma_dense<WT>(a1, x1, mfma_dense<WT>(a0, x0, c));
  }
}

// The selectors of every set of kept columns, by all threads: a column's bytes are
// those of the set's k-th kept value where it is the set's k-th (from 0), else
// zeros (selector 12).
template <class Frag, int XB>
__device__ __forceinline__ void fill_table(typename Frag::Entry* table) {
  if constexpr (Frag::TABLE) {
    constexpr int ND = 2 * XB;                          // dwords of eight columns
    for (int q = threadIdx.x; q < 256 * ND; q += blockDim.x) {
      const int s = q / ND, i = q % ND, c = 4 / XB * i;
      int base = 0;                                     // the first source's first value
      if constexpr (XB == 2) base = 2 * Frag::first_source(i);
      uint32_t sel = 0;
#pragma unroll
      for (int e = 0; e < 4 / XB; ++e) {
        const int k = __builtin_popcount(s & ((1 << (c + e)) - 1)) - base;
        const bool in = (s >> (c + e) & 1) && k >= 0 && k < 8 / XB;
        const uint32_t b = XB == 2 ? (in ? (uint32_t)((2 * k + 1) << 8 | 2 * k) : 0x0C0Cu) : (in ? (uint32_t)k : 0x0Cu);
        sel |= b << (8 * XB * e);
      }
      reinterpret_cast<uint32_t*>(table)[q] = sel;
    }
    __syncthreads();
  }
}
#endif

}  // namespace

}  // namespace nm
