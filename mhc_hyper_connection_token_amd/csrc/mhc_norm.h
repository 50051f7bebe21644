// mhc_norm.h -- device pieces shared by the norms around a branch and their
// gradients: operands whose type is known at run time, the gate, block sums.
#pragma once
#include "mhc_f8.h"
#include "mhc_kernels.h"

namespace mhc {

typedef unsigned uintx4 __attribute__((ext_vector_type(4)));

// Four entries of a row as they lie in memory: fp32, bf16, or e4m3 codes with their
// scale byte.  The type is the same for a whole launch, so the branch is uniform, and
// nothing in it waits for the load: the values are made where they are used.
enum Kind { kF32 = 0, kBF16 = 1, kF8 = 2 };

__device__ __forceinline__ uintx4 load_raw(const void* p, const unsigned char* s, int kind,
                                           size_t row, int HQ, int KB, int q) {
  uintx4 v{0u, 0u, 0u, 0u};
  if (kind == kF32) {
    v = __builtin_nontemporal_load(static_cast<const uintx4*>(p) + row * HQ + q);
  } else if (kind == kBF16) {
    const uintx2 h = __builtin_nontemporal_load(static_cast<const uintx2*>(p) + row * HQ + q);
    v[0] = h[0];
    v[1] = h[1];
  } else {
    v[0] = __builtin_nontemporal_load(static_cast<const unsigned*>(p) + row * KB * 32 + q);
    v[1] = s[row * KB + (q >> 5)];
  }
  return v;
}
__device__ __forceinline__ float4 raw_values(uintx4 v, int kind) {
  if (kind == kF8) return f8_unpack(v[0], f8_scale(v[1]));
  const bool h = kind == kBF16;
  return make_float4(__uint_as_float(h ? v[0] << 16 : v[0]),
                     __uint_as_float(h ? v[0] & 0xffff0000u : v[1]),
                     __uint_as_float(h ? v[1] << 16 : v[2]),
                     __uint_as_float(h ? v[1] & 0xffff0000u : v[3]));
}

// The factor a(g) of a gate and its slope a'(g).  With t = exp(-|g|) and d = 1/(1+t),
// sigmoid(g) and sigmoid(-g) are d and t*d in either order, so neither cancels.
template <bool SLOPE>
__device__ __forceinline__ void gate_one(float g, int act, float& a, float& s) {
  if (act == 0) {
    a = g;
    if (SLOPE) s = 1.f;
    return;
  }
  const float t = expf(-fabsf(g));
  const float d = __builtin_amdgcn_rcpf(1.f + t);
  const float p = g >= 0.f ? d : t * d;
  a = act == 1 ? p : g * p;
  if (SLOPE) {
    const float m = g >= 0.f ? t * d : d;  // 1 - p
    s = act == 1 ? p * m : fmaf(g * p, m, p);
  }
}
template <bool SLOPE>
__device__ __forceinline__ void gate_quad(float4 g, int act, float4& a, float4& s) {
  gate_one<SLOPE>(g.x, act, a.x, s.x);
  gate_one<SLOPE>(g.y, act, a.y, s.y);
  gate_one<SLOPE>(g.z, act, a.z, s.z);
  gate_one<SLOPE>(g.w, act, a.w, s.w);
}

__device__ __forceinline__ float4 mul4(float4 a, float4 b) {
  return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}
__device__ __forceinline__ float4 scale4(float4 a, float b) {
  return make_float4(a.x * b, a.y * b, a.z * b, a.w * b);
}
__device__ __forceinline__ float4 fma4(float4 a, float4 b, float4 c) {
  return make_float4(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y), fmaf(a.z, b.z, c.z),
                     fmaf(a.w, b.w, c.w));
}
__device__ __forceinline__ float4 zero4() { return make_float4(0.f, 0.f, 0.f, 0.f); }

__device__ __forceinline__ float wave_total(float v) {  // sum_wave, in every lane
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(sum_wave(v))));
}

// Four values to bf16, round to nearest even.
__device__ __forceinline__ uintx2 bf16_quad(float4 v) {
  const __hip_bfloat162 lo = __float22bfloat162_rn(make_float2(v.x, v.y));
  const __hip_bfloat162 hi = __float22bfloat162_rn(make_float2(v.z, v.w));
  unsigned u[2];
  __builtin_memcpy(&u[0], &lo, 4);
  __builtin_memcpy(&u[1], &hi, 4);
  return uintx2{u[0], u[1]};
}

}  // namespace mhc
