// mhc_norm_bwd.hip -- the gradients of the norms around a branch (mhc_norm.hip).
//
// branch_norm, with n = y r:  dn = dz nw;  dy = r (dn - n mean_i(dn n));  dnw = sum_t dz n.
// site_post_norm, with G = dL/dx', u = a(gate) nw f and e = sum_k post_k G_k:
//   dx[j] = sum_k comb[j,k] G_k            dcomb[j,k] = sum_i x_j G_k
//   dpost[k] = alpha r sum_i G_k u         df = alpha r (a nw e - f r^2 sum_i(e u) / H)
//   dnw = sum_t alpha r a f e              dgate = alpha r a' nw f e  (per token or summed)
// r stands in front of every sum over the row, so the row is read once: its sums are
// formed as it streams, e and f (dz and y) stay in registers, and the rest follows once
// the block has added the sums up.  A block takes tokens blockIdx.x, + gridDim.x, ... and
// keeps its part of the sums over tokens in registers; a second launch adds the
// parts up, in an order fixed by the shape.  HBM-bound.
#include "mhc_norm.h"

namespace mhc {

namespace {
// Parts of a sum over tokens: blocks of the first launch.
int parts_of(int T, int most) { return T < most ? T : most; }
constexpr int kParts = 1024;
}  // namespace

// Sums of several values over the block, in wave order, in every thread; `at` alternates
// between two buffers, so that one barrier a token is enough.
template <int N, int NW>
__device__ __forceinline__ void block_sums(float (&v)[N], float (&buf)[NW][N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_total(v[i]);
  if constexpr (NW > 1) {
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) buf[threadIdx.x >> 6][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = buf[0][i];
#pragma unroll
      for (int w = 1; w < NW; ++w) v[i] += buf[w][i];
    }
  }
}

template <int NW, int Q>
__global__ __launch_bounds__(64 * NW) void branch_norm_bwd_kernel(NormBwd p, int T, int HQ,
                                                                   int KB, float eps,
                                                                   float* __restrict__ part) {
  constexpr int NT = 64 * NW;
  __shared__ float buf[2][NW][2];
  const int y_kind = p.y_scales ? kF8 : kF32;
  const float inv_h = 1.f / (float)(4 * HQ);
  float4 w[Q], dw[Q];
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int q = threadIdx.x + NT * i;
    w[i] = q < HQ ? reinterpret_cast<const float4*>(p.nw)[q] : zero4();
    dw[i] = zero4();
  }
  int at = 0;
  for (size_t t = blockIdx.x; t < (size_t)T; t += gridDim.x, at ^= 1) {
    uintx4 zr[Q], yr[Q];
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const int q = threadIdx.x + NT * i;
      zr[i] = yr[i] = uintx4{0u, 0u, 0u, 0u};
      if (q < HQ) {
        zr[i] = load_raw(p.dz, nullptr, p.dz_kind, t, HQ, KB, q);
        yr[i] = load_raw(p.y, p.y_scales, y_kind, t, HQ, KB, q);
      }
    }
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const float4 y = raw_values(yr[i], y_kind), dz = raw_values(zr[i], p.dz_kind);
      sum[0] = sq4(y, sum[0]);
      sum[1] = dot4(mul4(dz, w[i]), y, sum[1]);
    }
    block_sums<2, NW>(sum, buf[at]);
    const float r = rms_inverse(sum[0], 4 * HQ, eps);
    const float c = -(sum[1] * r) * r * inv_h * r;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const int q = threadIdx.x + NT * i;
      const float4 y = raw_values(yr[i], y_kind), dz = raw_values(zr[i], p.dz_kind);
      if (q < HQ)
        reinterpret_cast<float4*>(p.dy)[t * HQ + q] =
            fma4(make_float4(c, c, c, c), y, scale4(mul4(dz, w[i]), r));
      dw[i] = fma4(dz, scale4(y, r), dw[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int q = threadIdx.x + NT * i;
    if (q < HQ) reinterpret_cast<float4*>(part)[(size_t)blockIdx.x * HQ + q] = dw[i];
  }
}

// out[i] = sum of n rows part[k][i]: a block takes 16 quads, 16 threads of a wave's four
// rows at a time.
template <int RG>
__global__ __launch_bounds__(16 * RG) void sum_rows_kernel(const float* __restrict__ part, int n,
                                                           int HQ, float* __restrict__ out,
                                                           float* __restrict__ out2,
                                                           size_t stride2) {
  __shared__ float4 acc[RG][16];
  const int c = threadIdx.x & 15, g = threadIdx.x >> 4, q = blockIdx.x * 16 + c;
  const float4* src = reinterpret_cast<const float4*>(part + (blockIdx.y ? stride2 : 0));
  float4 s = zero4();
  if (q < HQ)
    for (int k = g; k < n; k += RG) {
      const float4 v = src[(size_t)k * HQ + q];
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
  acc[g][c] = s;
  __syncthreads();
#pragma unroll
  for (int m = RG / 2; m > 0; m >>= 1) {
    if (g < m) {
      const float4 o = acc[g + m][c];
      s.x += o.x;
      s.y += o.y;
      s.z += o.z;
      s.w += o.w;
      acc[g][c] = s;
    }
    __syncthreads();
  }
  if (g == 0 && q < HQ) reinterpret_cast<float4*>(blockIdx.y ? out2 : out)[q] = s;
}

// GATE: 0 none, 1 one row for all tokens (its gradient summed over them), 2 one a token.
template <int S, int NW, int Q>
__global__ __launch_bounds__(64 * NW) void post_norm_bwd_kernel(PostNormBwd p, int T, int HQ,
                                                                int KB, float eps,
                                                                float* __restrict__ part,
                                                                size_t gate_part) {
  constexpr int NT = 64 * NW, NS = S * S + S;
  __shared__ float tail[2][NW][2];
  __shared__ float mix[2][NW][NS];
  const int x_kind = p.x_scales ? kF8 : kF32;
  const float inv_h = 1.f / (float)(4 * HQ);
  float4 dw[Q], dg[Q];
#pragma unroll
  for (int i = 0; i < Q; ++i) dw[i] = dg[i] = zero4();
  int at = 0;
  for (size_t t = blockIdx.x; t < (size_t)T; t += gridDim.x, at ^= 1) {
    float pk[S], ck[S][S];
#pragma unroll
    for (int k = 0; k < S; ++k) pk[k] = p.post[t * S + k];
#pragma unroll
    for (int j = 0; j < S; ++j)
#pragma unroll
      for (int k = 0; k < S; ++k) ck[j][k] = p.comb[t * S * S + j * S + k];
    float sum[NS], ends[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NS; ++i) sum[i] = 0.f;
    float4 e[Q];
    uintx4 fr[Q], gr[Q];
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const int q = threadIdx.x + NT * i;
      fr[i] = gr[i] = uintx4{0u, 0u, 0u, 0u};
      e[i] = zero4();
      if (q >= HQ) continue;
      float4 gv[S];
      uintx4 xr[S];
#pragma unroll
      for (int k = 0; k < S; ++k) gv[k] = nt_load4(p.g + ((t * S + k) * HQ + q) * 4);
      fr[i] = load_raw(p.f, p.f_scales, p.f_kind, t, HQ, KB, q);
      if (p.gate) gr[i] = load_raw(p.gate, nullptr, p.gate_kind, p.gate_rows ? t : 0, HQ, 0, q);
#pragma unroll
      for (int j = 0; j < S; ++j) xr[j] = load_raw(p.x, p.x_scales, x_kind, t * S + j, HQ, KB, q);
      const float4 f = raw_values(fr[i], p.f_kind);
      float4 u = mul4(f, reinterpret_cast<const float4*>(p.nw)[q]);
      if (p.gate) {
        float4 a, s;
        gate_quad<false>(raw_values(gr[i], p.gate_kind), p.gate_act, a, s);
        u = mul4(u, a);
      }
      e[i] = collapse4<S>(pk, gv, S);
      ends[0] = sq4(f, ends[0]);
      ends[1] = dot4(e[i], u, ends[1]);
#pragma unroll
      for (int j = 0; j < S; ++j) {
        reinterpret_cast<float4*>(p.dx)[(t * S + j) * HQ + q] = collapse4<S>(ck[j], gv, S);
        const float4 x = raw_values(xr[j], x_kind);
#pragma unroll
        for (int k = 0; k < S; ++k) sum[j * S + k] = dot4(x, gv[k], sum[j * S + k]);
        sum[S * S + j] = dot4(u, gv[j], sum[S * S + j]);
      }
    }
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const float v = sum_wave(sum[i]);
      if ((threadIdx.x & 63) == 0) mix[at][wave][i] = v;
    }
    if (NW == 1) __syncthreads();
    block_sums<2, NW>(ends, tail[at]);
    const float r = rms_inverse(ends[0], 4 * HQ, eps), ar = p.alpha * r;
    for (int i = threadIdx.x; i < NS; i += NT) {
      float v = mix[at][0][i];
#pragma unroll
      for (int w = 1; w < NW; ++w) v += mix[at][w][i];
      if (i < S * S)
        p.dcomb[t * S * S + i] = v;
      else
        p.dpost[t * S + i - S * S] = ar * v;
    }
    const float c = -(ends[1] * r) * r * inv_h * ar;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const int q = threadIdx.x + NT * i;
      if (q >= HQ) continue;
      const float4 f = raw_values(fr[i], p.f_kind);
      const float4 w = reinterpret_cast<const float4*>(p.nw)[q];
      const float4 b = scale4(e[i], ar);  // alpha r e
      float4 bw = mul4(b, w), ba = b;
      if (p.gate) {
        float4 a, s;
        gate_quad<true>(raw_values(gr[i], p.gate_kind), p.gate_act, a, s);
        const float4 d = mul4(mul4(bw, f), s);
        if (p.gate_rows)
          reinterpret_cast<float4*>(p.dgate)[t * HQ + q] = d;
        else
          dg[i] = make_float4(dg[i].x + d.x, dg[i].y + d.y, dg[i].z + d.z, dg[i].w + d.w);
        ba = mul4(ba, a);
        bw = mul4(bw, a);
      }
      reinterpret_cast<float4*>(p.df)[t * HQ + q] = fma4(make_float4(c, c, c, c), f, bw);
      dw[i] = fma4(ba, f, dw[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int q = threadIdx.x + NT * i;
    if (q >= HQ) continue;
    reinterpret_cast<float4*>(part)[(size_t)blockIdx.x * HQ + q] = dw[i];
    if (p.gate && !p.gate_rows)
      reinterpret_cast<float4*>(part + gate_part)[(size_t)blockIdx.x * HQ + q] = dg[i];
  }
}

size_t norm_bwd_work_bytes(int T, int H, int sums) {
  return (size_t)parts_of(T, kParts) * H * 4 * sums;
}

namespace {
void sum_rows(const float* part, int n, int HQ, float* out, float* out2, size_t stride2,
              hipStream_t st) {
  const dim3 grid((HQ + 15) / 16, out2 ? 2 : 1);  // n = 0 gives zeros
  hipLaunchKernelGGL(sum_rows_kernel<64>, grid, dim3(1024), 0, st, part, n, HQ, out, out2,
                     stride2);
}
}  // namespace

hipError_t launch_norm_bwd(const NormBwd& p, int T, int H, float eps, void* work,
                           hipStream_t st) {
  const int HQ = H / 4, KB = (H + kF8Block - 1) / kF8Block, n = parts_of(T, kParts);
  float* part = static_cast<float*>(work);
  if (n == 0) {
    sum_rows(part, 0, HQ, p.dnw, nullptr, 0, st);
    return hipGetLastError();
  }
#define MHC_NORM(W, Q)                                                                       \
  hipLaunchKernelGGL((branch_norm_bwd_kernel<W, Q>), dim3((unsigned)n), dim3(64 * W), 0, st, \
                     p, T, HQ, KB, eps, part)
  if (HQ <= 64)
    MHC_NORM(1, 1);
  else if (HQ <= 1024)
    MHC_NORM(4, 4);
  else if (HQ <= 2048)
    MHC_NORM(8, 4);
  else
    MHC_NORM(16, 4);
#undef MHC_NORM
  sum_rows(part, n, HQ, p.dnw, nullptr, 0, st);
  return hipGetLastError();
}

namespace {
template <int S>
void launch_post_norm_bwd_s(const PostNormBwd& p, int T, int HQ, int KB, float eps, float* part,
                            int n, size_t gate_part, hipStream_t st) {
#define MHC_NORM(W, Q)                                                                        \
  hipLaunchKernelGGL((post_norm_bwd_kernel<S, W, Q>), dim3((unsigned)n), dim3(64 * W), 0, st, \
                     p, T, HQ, KB, eps, part, gate_part)
  if (HQ <= 64)
    MHC_NORM(1, 1);
  else if (HQ <= 1024)
    MHC_NORM(8, 2);
  else if (HQ <= 2048)
    MHC_NORM(8, 4);
  else
    MHC_NORM(16, 4);
#undef MHC_NORM
}
}  // namespace

hipError_t launch_post_norm_bwd(const PostNormBwd& p, int T, int S, int H, float eps, void* work,
                                hipStream_t st) {
  const int HQ = H / 4, KB = (H + kF8Block - 1) / kF8Block, n = parts_of(T, kParts);
  float* part = static_cast<float*>(work);
  const size_t gate_part = (size_t)n * H;
  if (n > 0) switch (S) {
#define MHC_S(SS)                                                                  \
  case SS:                                                                         \
    launch_post_norm_bwd_s<SS>(p, T, HQ, KB, eps, part, n, gate_part, st);          \
    break;
    MHC_S(1) MHC_S(2) MHC_S(3) MHC_S(4) MHC_S(5) MHC_S(6) MHC_S(7) MHC_S(8)
#undef MHC_S
    default:
      return hipErrorInvalidValue;
  }
  sum_rows(part, n, HQ, p.dnw, p.gate && !p.gate_rows ? p.dgate : nullptr, gate_part, st);
  return hipGetLastError();
}

}  // namespace mhc
