// mhc_f8.h -- the 8-bit block format on the device: e4m3 codes with one
// power-of-two scale per block of 128 (include/mhc.h, "8-bit blocks").
//
// A block's scale is 2^e with e the least integer for which amax <= 448 * 2^e.
// A power of two moves exponents only: the relative rounding of a code does not
// depend on it, a decoded value has four significant bits and is exact in bf16
// and fp32, and the conversion of a code to bf16 applies it on the way.
#pragma once
#include <hip/hip_bf16.h>

#include "mhc_device.h"

namespace mhc {

constexpr int kF8Block = 128;

typedef int intx4 __attribute__((ext_vector_type(4)));
typedef float floatx2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef unsigned uintx2 __attribute__((ext_vector_type(2)));

// |v| as bits, 0 where v is infinite or NaN: such entries do not set a scale.
__device__ __forceinline__ unsigned f8_size(float v) {
  const unsigned a = __float_as_uint(v) & 0x7fffffffu;
  return a < 0x7f800000u ? a : 0u;
}

// The scale byte of a block whose largest size is `a` (bits): with a = 1.M * 2^p,
// a <= 448 * 2^e = 1.75 * 2^(e+8) holds from e = p - 8 where 1.M <= 1.75, else
// from p - 7.  Adding 2^21 - 1 carries into the exponent exactly when M passes
// 1.75.  e is at least -126, so that 2^-e is a normal number; 2^0 for a block
// without a finite nonzero entry.
__device__ __forceinline__ unsigned f8_scale_byte(unsigned a) {
  const int b = (int)((a + 0x1fffffu) >> 23) - 8;
  return a == 0u ? 127u : (unsigned)(b > 1 ? b : 1);
}
__device__ __forceinline__ float f8_inverse(unsigned byte) {  // 2^-e
  return __uint_as_float((254u - byte) << 23);
}
__device__ __forceinline__ float f8_scale(unsigned byte) {  // 2^e
  return __uint_as_float(byte << 23);
}

// Four entries to four codes, round to nearest even.  A finite scaled entry is
// at most 448, so the conversion never saturates one; it turns an infinity or a
// NaN into the NaN code (the format has no infinity).
__device__ __forceinline__ unsigned f8_pack(float a, float b, float c, float d, float inv) {
  int q = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
  q = __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, q, true);
  return (unsigned)q;
}
__device__ __forceinline__ float4 f8_unpack(unsigned q, float scale) {
  const floatx2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)q, false);
  const floatx2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)q, true);
  return make_float4(lo[0] * scale, lo[1] * scale, hi[0] * scale, hi[1] * scale);
}

// Eight codes (two dwords) to bf16, times the block scale.
__device__ __forceinline__ bf16x8 f8_to_bf16(int lo, int hi, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// 16 bytes from global memory to LDS without a register: lane i's bytes land at
// base + 16 * i (base the same for the whole wave).
__device__ __forceinline__ void load_to_lds(const unsigned char* src, unsigned char* base) {
  __builtin_amdgcn_global_load_lds(
      (const __attribute__((address_space(1))) void*)src,
      (__attribute__((address_space(3))) void*)base, 16, 0, 0);
}

// A byte a lane, into the low byte of dword i of base.
__device__ __forceinline__ void load_byte_to_lds(const unsigned char* src, unsigned char* base) {
  __builtin_amdgcn_global_load_lds(
      (const __attribute__((address_space(1))) void*)src,
      (__attribute__((address_space(3))) void*)base, 1, 0, 0);
}

// Maximum over the 32 lanes of a half-wave; every lane ends with it.
template <int CTRL>
__device__ __forceinline__ unsigned dpp_umax(unsigned v) {
  const unsigned o = (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
  return v > o ? v : o;
}
__device__ __forceinline__ unsigned umax_half(unsigned v) {
  v = dpp_umax<0xB1>(v);   // lane ^ 1
  v = dpp_umax<0x4E>(v);   // lane ^ 2
  v = dpp_umax<0x141>(v);  // the other quad of the half-row
  v = dpp_umax<0x128>(v);  // lane ^ 8
  auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return r[0] > r[1] ? r[0] : r[1];
}

// Four consecutive entries of a matrix row, as fp32.
template <typename E>
__device__ __forceinline__ float4 load_quad(const E* p);
template <>
__device__ __forceinline__ float4 load_quad<float>(const float* p) {
  return nt_load4(p);
}
template <>
__device__ __forceinline__ float4 load_quad<__hip_bfloat16>(const __hip_bfloat16* p) {
  const uintx2 v = __builtin_nontemporal_load(reinterpret_cast<const uintx2*>(p));
  return make_float4(__uint_as_float(v[0] << 16), __uint_as_float(v[0] & 0xffff0000u),
                     __uint_as_float(v[1] << 16), __uint_as_float(v[1] & 0xffff0000u));
}

// acc + a.b, the four products in order.
__device__ __forceinline__ float dot4(float4 a, float4 b, float acc) {
  acc = fmaf(a.x, b.x, acc);
  acc = fmaf(a.y, b.y, acc);
  acc = fmaf(a.z, b.z, acc);
  return fmaf(a.w, b.w, acc);
}

}  // namespace mhc
