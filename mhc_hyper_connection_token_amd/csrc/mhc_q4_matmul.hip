// mhc_q4_matmul.hip -- out[m,n] = sum_k a[m,k] w[n,k] with 4-bit groups (mhc_q4.h):
//   out[m,n] = sum_g scale[n,g] * (sum_{k in g} a[m,k] code[n,k] - zero[n,g] sum_{k in g} a[m,k])
// so that the matrix instructions multiply the codes themselves, which are exact in any type,
// and a scale is applied once to a group's sum, in fp32.
//   fp32 activations: three bf16 planes that add up to the value, each a product of its own;
//   bf16 activations: as they are;  both on v_mfma_f32_16x16x32_bf16, summed in fp32;
//   int8 codes with a scale per 32 columns: v_mfma_i32_16x16x32_i8, exact per block of 32.
// The sums of a, which the zero points multiply, come from the same instruction with a
// column operand of ones: they lie where the products lie.
#include "mhc_q4.h"

#include "mhc_kernels.h"

namespace mhc {

typedef int intx2 __attribute__((ext_vector_type(2)));

namespace {

enum Act { kActF32 = 0, kActBF16 = 1, kActQ8 = 2 };

// Eight neighbouring activations of one row.
template <int A>
struct Octet;
template <>
struct Octet<kActF32> {
  floatx4 v[2];
};
template <>
struct Octet<kActBF16> {
  intx4 v;
};
template <>
struct Octet<kActQ8> {
  intx2 v;
};
template <int A>
constexpr int act_size() {
  return A == kActF32 ? 4 : A == kActBF16 ? 2 : 1;
}

template <int A>
__device__ __forceinline__ Octet<A> load_octet(const unsigned char* p, bool in) {
  Octet<A> o;
  __builtin_memset(&o, 0, sizeof(o));
  if (in) o = *reinterpret_cast<const Octet<A>*>(p);
  return o;
}

// The top eight significant bits of eight fp32 values as bf16, and what they leave.
__device__ __forceinline__ bf16x8 take_plane(floatx4 (&v)[2]) {
  unsigned u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned lo = __float_as_uint(v[i >> 1][2 * (i & 1)]);
    const unsigned hi = __float_as_uint(v[i >> 1][2 * (i & 1) + 1]);
    u[i] = __builtin_amdgcn_perm(hi, lo, 0x07060302);
    v[i >> 1][2 * (i & 1)] -= __uint_as_float(lo & 0xffff0000u);
    v[i >> 1][2 * (i & 1) + 1] -= __uint_as_float(hi & 0xffff0000u);
  }
  bf16x8 r;
  __builtin_memcpy(&r, u, 16);
  return r;
}

template <int A>
constexpr int planes() {
  return A == kActF32 ? 3 : 1;
}

struct Q4Args {
  const unsigned char* a;
  const float* ad;  // scales of int8 activations, [M][K/32]
  const unsigned char* codes;
  const unsigned short* scales;
  const unsigned char* zeros;
  void* out;
  int M, N, K, KG, f16, bf16_out;
};

}  // namespace

// 16*MT rows of a and 16*NF columns n a block; its W waves take chunks of U times 128
// columns of the depth in turn, and their sums are added in wave order through LDS.
template <int A, int GS, int MT, int NF, int W, int U>
__global__ __launch_bounds__(64 * W) void q4_matmul_kernel(Q4Args p) {
  constexpr int PL = planes<A>(), GB = 1 << GS;  // blocks of 32 a group
  __shared__ floatx4 part[W][MT * NF][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16 * NF, m0 = blockIdx.y * 16 * MT;
  const int KB = p.K / kQ4Block, SB = (p.K + 127) / 128;
  // rows past the end read the last row; their results are not stored
  const unsigned char *crow[NF], *arow[MT];
  size_t srow[NF];
#pragma unroll
  for (int j = 0; j < NF; ++j) {
    const size_t n = min(n0 + 16 * j + r, p.N - 1);
    crow[j] = p.codes + n * SB * 64 + 16 * g;
    srow[j] = n * p.KG;
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
    arow[i] = p.a + (min(m0 + 16 * i + r, p.M - 1) * (size_t)p.K + 8 * g) * act_size<A>();
  floatx4 acc[MT][NF];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  for (int s0 = wave * U; s0 < SB; s0 += W * U) {
    intx4 cv[U][NF];
    float sv[U][NF][4 / GB], zv[U][NF][4 / GB];
    Octet<A> av[U][MT][4];
    float dv[A == kActQ8 ? U : 1][MT][4][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = min(s0 + u, SB - 1);
#pragma unroll
      for (int j = 0; j < NF; ++j) {
        cv[u][j] = *reinterpret_cast<const intx4*>(crow[j] + (size_t)s * 64);
#pragma unroll
        for (int b = 0; b < 4; b += GB) {
          const size_t k = srow[j] + min((4 * s + b) >> GS, p.KG - 1);
          sv[u][j][b / GB] = q4_scale(p.scales[k], p.f16);
          zv[u][j][b / GB] = p.zeros ? (float)p.zeros[k] : 8.f;
        }
      }
      // a block past the end: zeros
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int k = 4 * (s0 + u) + b;
          av[u][i][b] = load_octet<A>(arow[i] + (size_t)k * kQ4Block * act_size<A>(), k < KB);
          if constexpr (A == kActQ8)
#pragma unroll
            for (int v = 0; v < 4; ++v)
              dv[u][i][b][v] =
                  p.ad[(size_t)min(m0 + 16 * i + 4 * g + v, p.M - 1) * KB + min(k, KB - 1)];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      floatx4 sum[MT][NF], ones[MT];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (b % GB == 0) {
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            ones[i] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < NF; ++j) sum[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
          }
        }
        if constexpr (A == kActQ8) {
          const long one = 0x0101010101010101L;
          long cx[NF];
#pragma unroll
          for (int j = 0; j < NF; ++j)
            cx[j] = (long)(unsigned)q4_low(cv[u][j][b]) | ((long)q4_high(cv[u][j][b]) << 32);
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            long ax;
            __builtin_memcpy(&ax, &av[u][i][b].v, 8);
            const intx4 none{0, 0, 0, 0};
            const intx4 q = __builtin_amdgcn_mfma_i32_16x16x32_i8(ax, one, none, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < NF; ++j) {
              const intx4 t = __builtin_amdgcn_mfma_i32_16x16x32_i8(ax, cx[j], none, 0, 0, 0);
              const int z = (int)zv[u][j][b / GB];
#pragma unroll
              for (int v = 0; v < 4; ++v)
                sum[i][j][v] = fmaf((float)(t[v] - z * q[v]), dv[u][i][b][v], sum[i][j][v]);
            }
          }
        } else {
          bf16x8 cx[NF], one;
#pragma unroll
          for (int v = 0; v < 8; ++v) one[v] = (__bf16)1.0f;
#pragma unroll
          for (int j = 0; j < NF; ++j) cx[j] = q4_to_bf16(cv[u][j][b]);
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int l = 0; l < PL; ++l) {
              bf16x8 ax;
              if constexpr (A == kActF32)
                ax = take_plane(av[u][i][b].v);
              else
                __builtin_memcpy(&ax, &av[u][i][b].v, 16);
              ones[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ax, one, ones[i], 0, 0, 0);
#pragma unroll
              for (int j = 0; j < NF; ++j)
                sum[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ax, cx[j], sum[i][j], 0, 0, 0);
            }
        }
        if (b % GB == GB - 1) {
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NF; ++j)
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                const float t = A == kActQ8 ? sum[i][j][v]
                                            : fmaf(-zv[u][j][b / GB], ones[i][v], sum[i][j][v]);
                acc[i][j][v] = fmaf(sv[u][j][b / GB], t, acc[i][j][v]);
              }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) part[wave][i * NF + j][lane] = acc[i][j];
  __syncthreads();
  for (int i = threadIdx.x; i < MT * NF * 64; i += 64 * W) {
    const int l = i & 63, f = i >> 6;
    floatx4 s = part[0][f][l];
#pragma unroll
    for (int w = 1; w < W; ++w) s += part[w][f][l];
    const int n = n0 + 16 * (f % NF) + (l & 15);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int m = m0 + 16 * (f / NF) + 4 * (l >> 4) + v;
      if (m < p.M && n < p.N) {
        const size_t at = (size_t)m * p.N + n;
        if (p.bf16_out)
          static_cast<__hip_bfloat16*>(p.out)[at] = __float2bfloat16(s[v]);
        else
          static_cast<float*>(p.out)[at] = s[v];
      }
    }
  }
}

namespace {
template <int A, int GS, int MT, int NF, int W, int U>
void launch_q4_at(const Q4Args& p, hipStream_t st) {
  hipLaunchKernelGGL((q4_matmul_kernel<A, GS, MT, NF, W, U>),
                     dim3((p.N + 16 * NF - 1) / (16 * NF), (p.M + 16 * MT - 1) / (16 * MT)),
                     dim3(64 * W), 0, st, p);
}
template <int A, int GS>
void launch_q4_g(const Q4Args& p, hipStream_t st) {
  if (p.M > 16)
    launch_q4_at<A, GS, 2, 2, 8, 1>(p, st);
  else if (p.N >= 8192)
    launch_q4_at<A, GS, 1, 2, 8, 1>(p, st);
  else
    launch_q4_at<A, GS, 1, 1, 8, 2>(p, st);
}
template <int A>
void launch_q4_a(const Q4Args& p, int group, hipStream_t st) {
  if (group == 32)
    launch_q4_g<A, 0>(p, st);
  else if (group == 64)
    launch_q4_g<A, 1>(p, st);
  else
    launch_q4_g<A, 2>(p, st);
}
}  // namespace

hipError_t launch_q4_matmul(const Q4Matmul& q, int M, int N, int K, int group, hipStream_t st) {
  const Q4Args p{static_cast<const unsigned char*>(q.a),
                 q.a_scales,
                 q.codes,
                 static_cast<const unsigned short*>(q.scales),
                 q.zeros,
                 q.out,
                 M,
                 N,
                 K,
                 (K + group - 1) / group,
                 q.f16_scales,
                 q.bf16_out};
  if (q.a_kind == kActF32)
    launch_q4_a<kActF32>(p, group, st);
  else if (q.a_kind == kActBF16)
    launch_q4_a<kActBF16>(p, group, st);
  else
    launch_q4_a<kActQ8>(p, group, st);
  return hipGetLastError();
}

}  // namespace mhc
