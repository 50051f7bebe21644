// mhc_norm.h -- device pieces shared by the norms around a branch and their
// gradients: operands whose type is known at run time, the gate, block sums.
#pragma once
#include "mhc_f8.h"
#include "mhc_kernels.h"

namespace mhc {

// Four entries of a row as they lie in memory: fp32, bf16, or e4m3 codes with their scale
// byte.  (The type is a template's: loads of one that is known at run time end up behind
// branches, each of which waits for the loads before it.)
enum Kind { kF32 = 0, kBF16 = 1, kF8 = 2 };

template <int KIND>
struct Raw;
template <>
struct Raw<kF32> {
  floatx4 v;
};
template <>
struct Raw<kBF16> {
  uintx2 v;
};
template <>
struct Raw<kF8> {
  unsigned v, scale;
};

// Quad q of row `row` of [rows][4 * HQ]; s and KB: the scale bytes of 8-bit blocks.
template <int KIND>
__device__ __forceinline__ Raw<KIND> load_raw(const void* p, const unsigned char* s, size_t row,
                                              int HQ, int KB, int q) {
  Raw<KIND> r;
  if constexpr (KIND == kF32) {
    r.v = __builtin_nontemporal_load(static_cast<const floatx4*>(p) + row * HQ + q);
  } else if constexpr (KIND == kBF16) {
    r.v = __builtin_nontemporal_load(static_cast<const uintx2*>(p) + row * HQ + q);
  } else {
    r.v = __builtin_nontemporal_load(static_cast<const unsigned*>(p) + row * KB * 32 + q);
    r.scale = s[row * KB + (q >> 5)];
  }
  return r;
}
__device__ __forceinline__ float4 raw_values(Raw<kF32> r) {
  return make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
}
__device__ __forceinline__ float4 raw_values(Raw<kBF16> r) {
  return make_float4(__uint_as_float(r.v[0] << 16), __uint_as_float(r.v[0] & 0xffff0000u),
                     __uint_as_float(r.v[1] << 16), __uint_as_float(r.v[1] & 0xffff0000u));
}
__device__ __forceinline__ float4 raw_values(Raw<kF8> r) {
  return f8_unpack(r.v, f8_scale(r.scale));
}

// A gate: none, or one of the kinds.
enum Gate { kNoGate = 0, kGateF32 = 1, kGateBF16 = 2 };
template <int GATE>
constexpr int gate_kind() {
  return GATE == kGateBF16 ? kBF16 : kF32;
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
__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
__device__ __forceinline__ float4 zero4() { return make_float4(0.f, 0.f, 0.f, 0.f); }

// What the memory-side cache can hold of the outputs until the next kernel reads them; past
// its size stores that stay in it only displace (measured at the post mix's gradient).
constexpr size_t kCacheBytes = size_t(256) << 20;
__device__ __forceinline__ void store_out(float* p, float4 v, int stream) {
  if (stream)
    nt_store4(p, v);
  else
    *reinterpret_cast<float4*>(p) = v;
}

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
