// mhc_norm_bwd.h -- the kernel of the post mix's gradient with the norm behind the branch
// (mhc_norm_bwd.hip has the formulas), launched from a source for each pair of stream counts
// (it has many forms).
#pragma once
#include "mhc_norm.h"

namespace mhc {

constexpr int kOneWaveHidden = 1024;  // rows up to this are one wave's

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

template <int S, int X, int F, int GATE, int NW, int Q>
__global__ __launch_bounds__(64 * NW) void post_norm_bwd_kernel(PostNormBwd p, int T, int HQ,
                                                                int KB, float eps,
                                                                float* __restrict__ part,
                                                                float* __restrict__ gate_part) {
  constexpr int NT = 64 * NW, NS = S * S + S;
  __shared__ float tail[2][NW][2];
  __shared__ float mix[2][NW][NS];
  const float inv_h = 1.f / (float)(4 * HQ);
  float4 dw[Q], dg[Q];
#pragma unroll
  for (int i = 0; i < Q; ++i) dw[i] = dg[i] = zero4();
  // What of the next token is asked for while this one's sums are added up: the first quad of
  // each thread, past the row's end its last one.  us for none, one and two of them: 4096 tokens
  // of 4 x 4096 157, 147 and 151 with an 8-bit state and a bf16 gate, in fp32 186, 171 and 173
  // with a gate, 176, 170 and 164 without; 1024 of 4 x 7168 in fp32 82, 81 and 105 without (two
  // quads are kept in scratch there: 130 registers of some forms), 100, 122 and 144 with a gate a
  // token; 8192 of 4 x 512 59, 56 and 60.
  float4 gn[S];
  Raw<X> xn[S];
  Raw<F> fn;
  Raw<gate_kind<GATE>()> an;
  auto fetch = [&](size_t t) {
    const int q = min((int)threadIdx.x, HQ - 1);
#pragma unroll
    for (int k = 0; k < S; ++k) gn[k] = nt_load4(p.g + ((t * S + k) * HQ + q) * 4);
    fn = load_raw<F>(p.f, p.f_scales, t, HQ, KB, q);
    if constexpr (GATE != kNoGate)
      an = load_raw<gate_kind<GATE>()>(p.gate, nullptr, p.gate_rows ? t : 0, HQ, 0, q);
#pragma unroll
    for (int j = 0; j < S; ++j) xn[j] = load_raw<X>(p.x, p.x_scales, t * S + j, HQ, KB, q);
  };
  fetch(blockIdx.x);
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
    Raw<F> fr[Q];
    Raw<gate_kind<GATE>()> gr[Q];
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const int q = threadIdx.x + NT * i;
      if (q >= HQ) continue;
      float4 gv[S];
      Raw<X> xr[S];
      if (i == 0) {
        fr[0] = fn;
        if constexpr (GATE != kNoGate) gr[0] = an;
#pragma unroll
        for (int k = 0; k < S; ++k) {
          gv[k] = gn[k];
          xr[k] = xn[k];
        }
      } else {
#pragma unroll
        for (int k = 0; k < S; ++k) gv[k] = nt_load4(p.g + ((t * S + k) * HQ + q) * 4);
        fr[i] = load_raw<F>(p.f, p.f_scales, t, HQ, KB, q);
        if constexpr (GATE != kNoGate)
          gr[i] = load_raw<gate_kind<GATE>()>(p.gate, nullptr, p.gate_rows ? t : 0, HQ, 0, q);
#pragma unroll
        for (int j = 0; j < S; ++j) xr[j] = load_raw<X>(p.x, p.x_scales, t * S + j, HQ, KB, q);
      }
      const float4 f = raw_values(fr[i]);
      float4 u = mul4(f, reinterpret_cast<const float4*>(p.nw)[q]);
      if constexpr (GATE != kNoGate) {
        float4 a, s;
        gate_quad<false>(raw_values(gr[i]), p.gate_act, a, s);
        u = mul4(u, a);
      }
      e[i] = collapse4<S>(pk, gv, S);
      ends[0] = sq4(f, ends[0]);
      ends[1] = dot4(e[i], u, ends[1]);
#pragma unroll
      for (int j = 0; j < S; ++j) {
        store_out(p.dx + ((t * S + j) * HQ + q) * 4, collapse4<S>(ck[j], gv, S), p.stream);
        const float4 x = raw_values(xr[j]);
#pragma unroll
        for (int k = 0; k < S; ++k) sum[j * S + k] = dot4(x, gv[k], sum[j * S + k]);
        sum[S * S + j] = dot4(u, gv[j], sum[S * S + j]);
      }
    }
    if (t + gridDim.x < (size_t)T) fetch(t + gridDim.x);
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
      const float4 f = raw_values(fr[i]);
      const float4 w = reinterpret_cast<const float4*>(p.nw)[q];
      const float4 b = scale4(e[i], ar);  // alpha r e
      float4 bw = mul4(b, w), ba = b;
      if constexpr (GATE != kNoGate) {
        float4 a, s;
        gate_quad<true>(raw_values(gr[i]), p.gate_act, a, s);
        const float4 d = mul4(mul4(bw, f), s);
        if (p.gate_rows)
          store_out(p.dgate + (t * HQ + q) * 4, d, p.stream);
        else
          dg[i] = add4(dg[i], d);
        ba = mul4(ba, a);
        bw = mul4(bw, a);
      }
      store_out(p.df + (t * HQ + q) * 4, fma4(make_float4(c, c, c, c), f, bw), p.stream);
      dw[i] = fma4(ba, f, dw[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int q = threadIdx.x + NT * i;
    if (q >= HQ) continue;
    reinterpret_cast<float4*>(part)[(size_t)blockIdx.x * HQ + q] = dw[i];
    if (GATE != kNoGate && !p.gate_rows)
      reinterpret_cast<float4*>(gate_part)[(size_t)blockIdx.x * HQ + q] = dg[i];
  }
}

template <int S, int X, int F, int GATE>
void launch_post_norm_bwd_g(const PostNormBwd& p, int T, int HQ, int KB, float eps, float* part,
                            int n, float* gate_part, hipStream_t st) {
#define MHC_NORM(W, Q) \
  post_norm_bwd_kernel<S, X, F, GATE, W, Q><<<n, 64 * W, 0, st>>>(p, T, HQ, KB, eps, part, gate_part)
  // (Rows past 4096 still take more registers than there are in 14 of 18 forms at four streams,
  // 2 to 50 of them, and in 5 at eight, 2 to 42; 1024 tokens of 4 x 7168 in fp32 with a gate a
  // token 123 us, without a gate, which fits, 81.)
  if (HQ * 4 <= kOneWaveHidden)
    MHC_NORM(1, 4);
  else if constexpr (S > 4)  // the sums of many streams leave 512 threads too few registers:
    HQ <= 1024 ? MHC_NORM(4, 4) : MHC_NORM(4, 8);  // 1024 tokens of 8 x 7168 181 -> 151 us
  else
    HQ <= 1024 ? MHC_NORM(8, 2) : MHC_NORM(8, 4);
#undef MHC_NORM
}
template <int S, int X, int F>
void launch_post_norm_bwd_f(const PostNormBwd& p, int T, int HQ, int KB, float eps, float* part,
                            int n, float* gate_part, hipStream_t st) {
  if (!p.gate)
    launch_post_norm_bwd_g<S, X, F, kNoGate>(p, T, HQ, KB, eps, part, n, gate_part, st);
  else if (p.gate_kind == kF32)
    launch_post_norm_bwd_g<S, X, F, kGateF32>(p, T, HQ, KB, eps, part, n, gate_part, st);
  else
    launch_post_norm_bwd_g<S, X, F, kGateBF16>(p, T, HQ, KB, eps, part, n, gate_part, st);
}
template <int S>
void launch_post_norm_bwd_s(const PostNormBwd& p, int T, int HQ, int KB, float eps, float* part,
                            int n, float* gate_part, hipStream_t st) {
#define MHC_F(F)                                                                               \
  p.x_scales ? launch_post_norm_bwd_f<S, kF8, F>(p, T, HQ, KB, eps, part, n, gate_part, st)    \
             : launch_post_norm_bwd_f<S, kF32, F>(p, T, HQ, KB, eps, part, n, gate_part, st)
  if (p.f_kind == kF32)
    MHC_F(kF32);
  else if (p.f_kind == kBF16)
    MHC_F(kBF16);
  else
    MHC_F(kF8);
#undef MHC_F
}

// Streams 2k + 1 and 2k + 2, a source file each pair.
void launch_post_norm_bwd_12(const PostNormBwd& p, int T, int S, int HQ, int KB, float eps,
                             float* part, int n, float* gate_part, hipStream_t st);
void launch_post_norm_bwd_34(const PostNormBwd& p, int T, int S, int HQ, int KB, float eps,
                             float* part, int n, float* gate_part, hipStream_t st);
void launch_post_norm_bwd_56(const PostNormBwd& p, int T, int S, int HQ, int KB, float eps,
                             float* part, int n, float* gate_part, hipStream_t st);
void launch_post_norm_bwd_78(const PostNormBwd& p, int T, int S, int HQ, int KB, float eps,
                             float* part, int n, float* gate_part, hipStream_t st);

}  // namespace mhc
