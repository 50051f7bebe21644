// mhc_q4.hip -- 4-bit groups (include/mhc.h): weights to codes with a scale and, where asked
// for, a zero point per group, and back.  Done once per weight.
//
// A thread holds four neighbouring columns; a group's G/4 threads are neighbouring lanes
// and exchange its extremes.  The code dword of an octet of columns (mhc_q4.h) is put together
// by the lane of its low halves; the high ones are four lanes on.
#include "mhc_norm.h"
#include "mhc_q4.h"

namespace mhc {

namespace {
__device__ __forceinline__ float finite_or_zero(float v) {
  return (__float_as_uint(v) & 0x7f800000u) == 0x7f800000u ? 0.f : v;
}
__device__ __forceinline__ float to_bf16(float v) {  // the value, rounded to nearest even
  return __bfloat162float(__float2bfloat16(v));
}
}  // namespace

template <int G, int KIND>
__global__ __launch_bounds__(256) void q4_encode_kernel(const void* __restrict__ w, int N,
                                                        int K, int KG,
                                                        unsigned char* __restrict__ codes,
                                                        __hip_bfloat16* __restrict__ scales,
                                                        unsigned char* __restrict__ zeros) {
  const int PQ = (K + 127) / 128 * 32;  // quads of a row, up to whole groups
  const size_t total = (size_t)N * PQ;
  // whole waves stay in the loop: the exchange below needs every lane of a group
  for (size_t at = (size_t)blockIdx.x * 256 + threadIdx.x; at - (threadIdx.x & 63) < total;
       at += (size_t)gridDim.x * 256) {
    const bool in = at < total;
    const size_t n = in ? at / PQ : 0;
    const int q = in ? (int)(at - n * PQ) : 0;
    const bool real = in && q * 4 < K;
    float4 v = zero4();
    if (real) v = raw_values(load_raw<KIND>(w, nullptr, n, K / 4, 0, q));
    const float x[4] = {v.x, v.y, v.z, v.w};
    float lo = 0.f, hi = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo = fminf(lo, finite_or_zero(x[i]));
      hi = fmaxf(hi, finite_or_zero(x[i]));
    }
#pragma unroll
    for (int m = 1; m < G / 4; m *= 2) {
      lo = fminf(lo, __shfl_xor(lo, m));
      hi = fmaxf(hi, __shfl_xor(hi, m));
    }
    // a group whose scale is below the smallest normal number takes that number: its
    // entries are far below one step then and get the zero point
    float d = to_bf16(zeros ? hi / 15.f - lo / 15.f : fmaxf(hi, -lo) / 7.f);
    if (d < 1.17549435e-38f) d = 1.17549435e-38f;
    const float z = zeros ? fminf(rintf(-lo / d), 15.f) : 8.f;
    const float least = zeros ? 0.f : 1.f;
    unsigned mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // NaN takes the zero point, an infinity the end of the range
      const float c = x[i] == x[i] ? fminf(fmaxf(rintf(x[i] / d) + z, least), 15.f) : z;
      mine |= (unsigned)c << (8 * i);
    }
    const unsigned high = __shfl_xor(mine, 4);
    if (real && !(q & 4))
      reinterpret_cast<unsigned*>(codes)[n * (K / 8) + (q >> 3) * 4 + (q & 3)] =
          mine | (high << 4);
    if (real && q % (G / 4) == 0) {
      scales[n * KG + q / (G / 4)] = __float2bfloat16(d);
      if (zeros) zeros[n * KG + q / (G / 4)] = (unsigned char)z;
    }
  }
}

__global__ __launch_bounds__(256) void q4_decode_kernel(const unsigned char* __restrict__ codes,
                                                        const unsigned short* __restrict__ scales,
                                                        int f16,
                                                        const unsigned char* __restrict__ zeros,
                                                        int N, int K, int KG, int gshift,
                                                        float* __restrict__ out) {
  const int KO = K / 8;  // octets of a row
  const size_t total = (size_t)N * KO;
  for (size_t at = (size_t)blockIdx.x * 256 + threadIdx.x; at < total;
       at += (size_t)gridDim.x * 256) {
    const size_t n = at / KO;
    const int o = (int)(at - n * KO);
    const unsigned c = reinterpret_cast<const unsigned*>(codes)[at];
    const size_t k = n * KG + (o >> (2 + gshift));
    const float d = q4_scale(scales[k], f16), z = zeros ? (float)zeros[k] : 8.f;
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = ((float)((c >> (8 * i)) & 15) - z) * d;
      v[4 + i] = ((float)((c >> (8 * i + 4)) & 15) - z) * d;
    }
    float4* p = reinterpret_cast<float4*>(out + n * K + (o >> 2) * 32 + (o & 3) * 4);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[4] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

namespace {
unsigned blocks_for(size_t threads) {
  const size_t n = (threads + 255) / 256;
  return (unsigned)(n < 65536 ? n : 65536);
}
}  // namespace

namespace {
template <int G>
void launch_q4_encode_g(const void* w, bool bf16, int N, int K, unsigned char* codes,
                        __hip_bfloat16* scales, unsigned char* zeros, hipStream_t st) {
  const int KG = (K + G - 1) / G;
  const dim3 grid(blocks_for((size_t)N * ((K + 127) / 128 * 32)));
  if (bf16)
    hipLaunchKernelGGL((q4_encode_kernel<G, kBF16>), grid, dim3(256), 0, st, w, N, K, KG, codes,
                       scales, zeros);
  else
    hipLaunchKernelGGL((q4_encode_kernel<G, kF32>), grid, dim3(256), 0, st, w, N, K, KG, codes,
                       scales, zeros);
}
}  // namespace

hipError_t launch_q4_encode(const void* w, bool bf16, int N, int K, int group,
                            unsigned char* codes, void* scales, unsigned char* zeros,
                            hipStream_t st) {
  __hip_bfloat16* s = static_cast<__hip_bfloat16*>(scales);
  if (group == 32)
    launch_q4_encode_g<32>(w, bf16, N, K, codes, s, zeros, st);
  else if (group == 64)
    launch_q4_encode_g<64>(w, bf16, N, K, codes, s, zeros, st);
  else
    launch_q4_encode_g<128>(w, bf16, N, K, codes, s, zeros, st);
  return hipGetLastError();
}

hipError_t launch_q4_decode(const unsigned char* codes, const void* scales, bool f16,
                            const unsigned char* zeros, int N, int K, int group, float* out,
                            hipStream_t st) {
  hipLaunchKernelGGL(q4_decode_kernel, dim3(blocks_for((size_t)N * (K / 8))), dim3(256), 0, st,
                     codes, static_cast<const unsigned short*>(scales), (int)f16, zeros, N, K,
                     (K + group - 1) / group, q4_shift(group), out);
  return hipGetLastError();
}

}  // namespace mhc
