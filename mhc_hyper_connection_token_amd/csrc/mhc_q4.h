// mhc_q4.h -- 4-bit groups on the device (include/mhc.h, "4-bit groups").
//
// The 16 bytes of a block of 32 columns are four dwords: dword d holds columns 4 d .. + 3 in the
// low halves of its bytes and columns 16 + 4 d .. + 3 in the high ones.  Two neighbouring dwords
// thus hold two octets of columns: dwords 0 and 1 octet 0 (columns 0 .. 7) and, in the high
// halves, octet 2; dwords 2 and 3 octets 1 and 3.  A matrix instruction takes an octet of every
// lane group; which ones is chosen so that what it sums lies in one group of columns.
#pragma once
#include "mhc_f8.h"

namespace mhc {

typedef int intx2 __attribute__((ext_vector_type(2)));

constexpr int kQ4Block = 32;  // columns of 16 bytes of codes; divides every group

inline int q4_shift(int group) { return group == 32 ? 0 : group == 64 ? 1 : 2; }

// A group's scale from its two bytes.
__device__ __forceinline__ float q4_scale(unsigned short bits, int f16) {
  _Float16 h;
  __builtin_memcpy(&h, &bits, 2);
  return f16 ? (float)h : __uint_as_float((unsigned)bits << 16);
}

// The codes of a dword's low halves and of its high ones.
__device__ __forceinline__ int q4_low(int c) { return c & 0x0f0f0f0f; }
__device__ __forceinline__ int q4_high(int c) { return (c >> 4) & 0x0f0f0f0f; }

// An octet of two neighbouring dwords: of their low halves, or of their high ones.
__device__ __forceinline__ intx2 q4_octet(int a, int b, int high) {
  return intx2{(a >> (4 * high)) & 0x0f0f0f0f, (b >> (4 * high)) & 0x0f0f0f0f};
}

// ... as bf16, exact: a byte 0 .. 15 read as e4m3 is that multiple of its smallest step,
// 2^-9 (its subnormals and first normal numbers are evenly spaced), so the conversion with
// scale 2^9 gives the integer, two to an instruction.
__device__ __forceinline__ bf16x8 q4_to_bf16(intx2 c) { return f8_to_bf16(c[0], c[1], 512.f); }

// ... and two of four codes as fp32, the same way: the lower two or the upper two.
template <bool UPPER>
__device__ __forceinline__ floatx2 q4_to_f32(int c) {
  return __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c, 512.f, UPPER);
}

}  // namespace mhc
