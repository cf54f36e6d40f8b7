// Where the lanes of a wave read the activations that the 4-bit few-token
// product quantises itself.  Plain integers, for the kernel and the host alike:
// a test goes through every load's lanes on the CPU.
#pragma once

#if defined(__HIP__)
#define NM_LANES __host__ __device__ __forceinline__
#else
#define NM_LANES inline
#endif

namespace nm {

// A load brings a 16-byte piece of two tokens: lane 32 h + p reads piece `part`
// of the eight values p of token t = first + h in the slab of 256 columns that
// starts `slab` bytes into a row.  Its offset from that slab of token 0, for
// `tokens` rows of `row` bytes, `pitch` bytes apart, EB bytes a value.  Tokens
// past the last repeat it and columns past the row repeat the slab's first:
// every lane reads inside its operand (a load with no lane inside would
// complete ahead of older ones, and a wait that counts loads pass too early).
template <int EB>
NM_LANES bool mx_lane_inside(int lane, int part, int slab, int row) {
  return slab + (lane & 31) * 8 * EB + 16 * part < row;
}
template <int EB>
NM_LANES int mx_lane_offset(int lane, int first, int part, int tokens, int pitch, int slab, int row) {
  const int t = first + (lane >> 5);
  return (t < tokens ? t : tokens - 1) * pitch +
         (mx_lane_inside<EB>(lane, part, slab, row) ? (lane & 31) * 8 * EB + 16 * part : 0);
}

}  // namespace nm
