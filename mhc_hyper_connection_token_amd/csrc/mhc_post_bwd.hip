// mhc_post_bwd.hip -- the gradient of the post mix.  With g = dL/dx' [T,S,H]:
//   dx[t,j,i]    = sum_k comb[t,j,k] g[t,k,i]
//   df[t,i]      = sum_k post[t,k] g[t,k,i]
//   dpost[t,k]   = sum_i g[t,k,i] f[t,i]
//   dcomb[t,j,k] = sum_i x[t,j,i] g[t,k,i]
// One block per token, one pass: a thread owns hidden quads, holds the S
// quads of g, writes the S + 1 output quads and adds S*S + S products to its
// sums, which the block adds up in a fixed order at the end.  x and f are fp32
// or 8-bit checkpoints (one dword per quad, one scale byte per 32 lanes).
// HBM-bound: 4*(2*S*H + H) bytes per token plus x and f once.
#include "mhc_f8.h"
#include "mhc_kernels.h"

namespace mhc {

// Quad q of row `row` of an fp32 matrix [rows][H], or of its 8-bit form.
template <bool F8>
__device__ __forceinline__ float4 kept_quad(const void* p, const unsigned char* s, size_t row,
                                            int HQ, int KB, int q) {
  if constexpr (F8) {
    const unsigned c = __builtin_nontemporal_load(static_cast<const unsigned*>(p) +
                                                  row * KB * 32 + q);
    return f8_unpack(c, f8_scale(s[row * KB + (q >> 5)]));
  } else {
    return nt_load4(static_cast<const float*>(p) + (row * HQ + q) * 4);
  }
}

template <bool STREAM>
__device__ __forceinline__ void store_out(float* p, float4 v) {
  if constexpr (STREAM)
    nt_store4(p, v);
  else
    *reinterpret_cast<float4*>(p) = v;
}

template <int S, bool XF8, bool FF8, int NT, bool STREAM>
__global__ __launch_bounds__(NT) void post_bwd_kernel(
    const float* __restrict__ g, const void* __restrict__ x,
    const unsigned char* __restrict__ xs, const void* __restrict__ f,
    const unsigned char* __restrict__ fs, const float* __restrict__ post,
    const float* __restrict__ comb, int H, int KB, float* __restrict__ dx,
    float* __restrict__ df, float* __restrict__ dpost, float* __restrict__ dcomb) {
  constexpr int NW = NT / 64, NS = S * S + S;
  __shared__ float part[NW][NS];
  const size_t t = blockIdx.x;
  const int HQ = H >> 2;
  float pk[S], ck[S][S];
#pragma unroll
  for (int k = 0; k < S; ++k) pk[k] = post[t * S + k];
#pragma unroll
  for (int j = 0; j < S; ++j)
#pragma unroll
    for (int k = 0; k < S; ++k) ck[j][k] = comb[t * S * S + j * S + k];
  float sum[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) sum[i] = 0.f;
  for (int q = threadIdx.x; q < HQ; q += NT) {
    float4 gv[S];
#pragma unroll
    for (int k = 0; k < S; ++k) gv[k] = nt_load4(g + ((t * S + k) * HQ + q) * 4);
    const float4 fv = kept_quad<FF8>(f, fs, t, HQ, KB, q);
    float4 xv[S];
#pragma unroll
    for (int j = 0; j < S; ++j) xv[j] = kept_quad<XF8>(x, xs, t * S + j, HQ, KB, q);
    store_out<STREAM>(df + (t * HQ + q) * 4, collapse4<S>(pk, gv, S));
#pragma unroll
    for (int j = 0; j < S; ++j) {
      store_out<STREAM>(dx + ((t * S + j) * HQ + q) * 4, collapse4<S>(ck[j], gv, S));
#pragma unroll
      for (int k = 0; k < S; ++k) sum[j * S + k] = dot4(xv[j], gv[k], sum[j * S + k]);
      sum[S * S + j] = dot4(fv, gv[j], sum[S * S + j]);
    }
  }
  const int wave = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const float v = sum_wave(sum[i]);
    if ((threadIdx.x & 63) == 0) part[wave][i] = v;
  }
  __syncthreads();
  if (threadIdx.x < NS) {
    float v = part[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < NW; ++w) v += part[w][threadIdx.x];
    if (threadIdx.x < S * S)
      dcomb[t * S * S + threadIdx.x] = v;
    else
      dpost[t * S + threadIdx.x - S * S] = v;
  }
}

namespace {
// What the memory-side cache can hold of the outputs until the next kernel reads
// them.  Stores that stay in it: 92 against 112 us at 1024 tokens of 8 x 7168 (264 MB
// written); past its size they only displace: 124 against 117 at 4096 tokens of
// 4 x 4096 (335 MB), call after call.
constexpr size_t kCacheBytes = size_t(256) << 20;

template <int S, bool XF8, bool FF8>
void launch(const PostBwd& p, int T, int H, hipStream_t st) {
  constexpr int NT = S <= 4 ? 512 : 256;  // 8 x 7168: 256 is 10 % faster, 4 x 4096: 2 % slower
  const int KB = (H + kF8Block - 1) / kF8Block;
  if ((size_t)T * (S + 1) * H * 4 <= kCacheBytes)
    hipLaunchKernelGGL((post_bwd_kernel<S, XF8, FF8, NT, false>), dim3((unsigned)T), dim3(NT), 0,
                       st, p.g, p.x, p.x_scales, p.f, p.f_scales, p.post, p.comb, H, KB, p.dx,
                       p.df, p.dpost, p.dcomb);
  else
    hipLaunchKernelGGL((post_bwd_kernel<S, XF8, FF8, NT, true>), dim3((unsigned)T), dim3(NT), 0,
                       st, p.g, p.x, p.x_scales, p.f, p.f_scales, p.post, p.comb, H, KB, p.dx,
                       p.df, p.dpost, p.dcomb);
}
template <int S>
void launch_s(const PostBwd& p, int T, int H, hipStream_t st) {
  if (p.x_scales)
    p.f_scales ? launch<S, true, true>(p, T, H, st) : launch<S, true, false>(p, T, H, st);
  else
    p.f_scales ? launch<S, false, true>(p, T, H, st) : launch<S, false, false>(p, T, H, st);
}
}  // namespace

hipError_t launch_post_bwd(const PostBwd& p, int T, int S, int H, hipStream_t st) {
  switch (S) {
#define MHC_S(SS)             \
  case SS:                    \
    launch_s<SS>(p, T, H, st); \
    break;
    MHC_S(1) MHC_S(2) MHC_S(3) MHC_S(4) MHC_S(5) MHC_S(6) MHC_S(7) MHC_S(8)
#undef MHC_S
    default:
      return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace mhc
