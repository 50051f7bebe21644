// mhc_q4.h -- 4-bit groups on the device (include/mhc.h, "4-bit groups").
//
// The 64 bytes of a row's 128 columns are sixteen dwords, dword 4 g + b an octet: columns
// 32 b + 8 g .. + 7, the first four in the low halves of its bytes.  Sixteen bytes from
// 16 g on are thus one octet of each of the four blocks of 32 columns, and the four lanes
// (g = 0 .. 3) of a matrix instruction's column that load them hold with their dword b all
// of block b: what one instruction sums lies in one block, and so in one group.
#pragma once
#include "mhc_f8.h"

namespace mhc {

constexpr int kQ4Block = 32;  // columns a matrix instruction sums; divides every group

inline int q4_shift(int group) { return group == 32 ? 0 : group == 64 ? 1 : 2; }

// A group's scale from its two bytes.
__device__ __forceinline__ float q4_scale(unsigned short bits, int f16) {
  _Float16 h;
  __builtin_memcpy(&h, &bits, 2);
  return f16 ? (float)h : __uint_as_float((unsigned)bits << 16);
}

// The codes of an octet, four to a dword.
__device__ __forceinline__ int q4_low(int c) { return c & 0x0f0f0f0f; }
__device__ __forceinline__ int q4_high(int c) { return (c >> 4) & 0x0f0f0f0f; }

// ... as bf16, exact: a byte 0 .. 15 read as e4m3 is that multiple of its smallest step,
// 2^-9 (its subnormals and first normal numbers are evenly spaced), so the conversion with
// scale 2^9 gives the integer, two to an instruction.
__device__ __forceinline__ bf16x8 q4_to_bf16(int c) {
  return f8_to_bf16(q4_low(c), q4_high(c), 512.f);
}

}  // namespace mhc
