// mhc_pre_bwd.hip -- the gradient of the pre chain (include/mhc.h,
// mhc_site_pre_bwd), recomputed from the site's input x, which is fp32 or an
// 8-bit checkpoint.  Per token, with n = S*H:
//   raw = W x, ss = |x|^2, r = 1/sqrt(ss/n + eps), m = r raw, z = scale m + base
//   dpre_c  = (given) + sum_i dy_i x_c,i
//   dz      = dpre p(1-p), dpost q(1 - q/2), and exp(z) times the gradient that
//             the Sinkhorn rounds hand back: a pass c' = c/s, s = sum c + eps,
//             has dc = (dc' - sum dc' c') / s over the same row or column
//   u_r     = r scale dz_r,   alpha = -(sum_r scale dz_r m_r) r^2 / n
//   dx_c    = dx_in_c + pre_c dy + sum_r u_r W_r,c + alpha x_c
//   dW      = sum_t u_t x_t^T,  dbase = sum_t dz,  dscale_g = sum_t sum_g dz m
// Four launches: the dots (raw, ss, dy.x) split over the hidden axis; the gates
// forward and backward, one wave per four tokens (one where S > 4); the stream
// that writes dx and adds up dW, a wave owning 64 columns over a range of
// tokens; and the sums over the ranges and tokens.  x and dy are read twice
// (neither fits on chip while a token's dots are open); everything else once.
#include "mhc_f8.h"
#include "mhc_kernels.h"

namespace mhc {

namespace {

constexpr int rows_of(int S) { return (2 + S) * S; }
constexpr int row_tiles(int S) { return (rows_of(S) + 15) / 16; }

// Quad q of row `row` of x as fp32.
template <bool F8>
__device__ __forceinline__ float4 x_quad(const void* p, const unsigned char* s, size_t row,
                                         int HQ, int KB, int q) {
  if constexpr (F8) {
    const unsigned c = static_cast<const unsigned*>(p)[row * KB * 32 + q];
    return f8_unpack(c, f8_scale(s[row * KB + (q >> 5)]));
  } else {
    return static_cast<const float4*>(p)[row * HQ + q];
  }
}
__device__ __forceinline__ float fma4(float4 a, float4 b, float acc) {
  acc = fmaf(a.x, b.x, acc);
  acc = fmaf(a.y, b.y, acc);
  acc = fmaf(a.z, b.z, acc);
  return fmaf(a.w, b.w, acc);
}
// Sum over the four 16-lane rows of a wave, lane by lane.
__device__ __forceinline__ float sum_rows(float v) { return swap32_sum(swap16_sum(v)); }

}  // namespace

// ---------------------------------------------------------------- dots
// part[G][T][R + 1 + S]: the R dots, the sum of squares, the S products with dy.
// A block takes 16 tokens and one of G ranges of hidden quads (all streams of
// it); its waves take every fourth step of four quads.
template <int S, bool F8>
__global__ __launch_bounds__(256) void pre_bwd_dots_kernel(
    const void* __restrict__ x, const unsigned char* __restrict__ xs,
    const float* __restrict__ w, const float* __restrict__ dy, int T, int H, int KB, int G,
    int steps, float* __restrict__ part) {
  constexpr int R = rows_of(S), NRT = row_tiles(S), V = R + 1 + S;
  __shared__ float sums[4][16][NRT * 16 + 1 + S];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane & 15, g = lane >> 4;
  const int tb = blockIdx.x / G, gi = blockIdx.x - tb * G, HQ = H >> 2;
  const size_t n4 = (size_t)S * HQ;
  const size_t t = min(tb * 16 + r16, T - 1);
  const float4* w4 = reinterpret_cast<const float4*>(w);
  const float4* dy4 = reinterpret_cast<const float4*>(dy) + t * HQ;
  floatx4 acc[NRT];
  float ss = 0.f, dp[S];
#pragma unroll
  for (int i = 0; i < NRT; ++i) acc[i] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < S; ++c) dp[c] = 0.f;
  const int s_end = min((gi + 1) * steps, (HQ + 3) / 4);
  for (int st = gi * steps + wave; st < s_end; st += 4) {
    const int q = st * 4 + g;
    const bool in = q < HQ;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 d = in ? dy4[q] : zero;
#pragma unroll
    for (int c = 0; c < S; ++c) {
      const float4 xv = in ? x_quad<F8>(x, xs, t * S + c, HQ, KB, q) : zero;
      ss = fma4(xv, xv, ss);
      dp[c] = fma4(d, xv, dp[c]);
#pragma unroll
      for (int i = 0; i < NRT; ++i) {
        const size_t row = min(16 * i + r16, R - 1);
        const float4 wv = in ? w4[row * n4 + (size_t)c * HQ + q] : zero;
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(wv.x, xv.x, acc[i], 0, 0, 0);
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(wv.y, xv.y, acc[i], 0, 0, 0);
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(wv.z, xv.z, acc[i], 0, 0, 0);
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(wv.w, xv.w, acc[i], 0, 0, 0);
      }
    }
  }
  float* mine = sums[wave][r16];
#pragma unroll
  for (int i = 0; i < NRT; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) mine[16 * i + 4 * g + v] = acc[i][v];
  ss = sum_rows(ss);
  if (g == 0) mine[NRT * 16] = ss;
#pragma unroll
  for (int c = 0; c < S; ++c) {
    const float v = sum_rows(dp[c]);
    if (g == 0) mine[NRT * 16 + 1 + c] = v;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * V; i += 256) {
    const int k = i / V, v = i - k * V, at = v < R ? v : v - R + NRT * 16;
    if (tb * 16 + k < T)
      part[((size_t)gi * T + tb * 16 + k) * V + v] =
          (sums[0][k][at] + sums[1][k][at]) + (sums[2][k][at] + sums[3][k][at]);
  }
}

// ---------------------------------------------------------------- gates
// u [T][16*NRT] (zero past R), side [T][S + 1] = the pre gates and alpha,
// red [R + 3][T] = dz and, per scale, the sum of dz * m.
// hist (LDS): the matrix before every pass, 64 entries each.
template <int S>
__global__ __launch_bounds__(64) void pre_bwd_gates_kernel(
    const float* __restrict__ part, int G, int T, int n, const float* __restrict__ scale,
    const float* __restrict__ base, int iters, float eps, const float* __restrict__ dpre,
    const float* __restrict__ dpost, const float* __restrict__ dcomb, float* __restrict__ u_out,
    float* __restrict__ side, float* __restrict__ red) {
  constexpr int L = S <= 4 ? 4 : 8, NU = L == 4 ? 4 : 1;
  constexpr int R = rows_of(S), NRT = row_tiles(S), V = R + 1 + S;
  __shared__ float raw[NU][V], dzs[NU][R];
  extern __shared__ float hist[];
  const int lane = threadIdx.x, t0 = blockIdx.x * NU;
  for (int i = lane; i < NU * V; i += 64) {
    const int k = i / V, v = i - k * V;
    float s = 0.f;
    if (t0 + k < T)
      for (int gi = 0; gi < G; ++gi) s += part[((size_t)gi * T + t0 + k) * V + v];
    raw[k][v] = s;
  }
  __syncthreads();
  {
    const int k = L == 4 ? lane >> 3 : 0, gt = L == 4 ? lane & 7 : lane;
    const size_t t = t0 + k;
    if (k < NU && t < (size_t)T && gt < 2 * S) {
      const float rinv = rms_inverse(raw[k][R], n, eps), m = raw[k][gt] * rinv;
      if (gt < S) {
        const float p = sigmoid_exact_ends(fmaf(scale[0], m, base[gt]));
        const float d = raw[k][R + 1 + gt] + (dpre ? dpre[t * S + gt] : 0.f);
        side[t * (S + 1) + gt] = p;
        dzs[k][gt] = d * p * (1.0f - p);
      } else {
        const float p = sigmoid_exact_ends(fmaf(scale[1], m, base[gt]));
        dzs[k][gt] = dpost[t * S + gt - S] * 2.0f * p * (1.0f - p);
      }
    }
  }
  {
    int j, k, tu;
    sinkhorn_lane_entry<L>(lane, tu, j, k);
    const bool valid = j < S && k < S && tu < NU && t0 + tu < T;
    const int r = 2 * S + j * S + k;
    float c = 0.f, d = 0.f;
    if (valid) {
      const float rinv = rms_inverse(raw[tu][R], n, eps);
      c = expf(fmaf(scale[2], raw[tu][r] * rinv, base[r]));
      d = dcomb[((size_t)(t0 + tu) * S + j) * S + k];
    }
    // padded entries divide by one: they stay zero whatever eps is
    const float pad = valid ? eps : 1.0f;
    for (int it = 0; it < iters; ++it) {
      hist[(2 * it) * 64 + lane] = c;
      c *= __builtin_amdgcn_rcpf(row_sum<L>(c) + pad);
      hist[(2 * it + 1) * 64 + lane] = c;
      c *= __builtin_amdgcn_rcpf(col_sum<L>(c) + pad);
    }
    for (int it = iters - 1; it >= 0; --it) {
      float before = hist[(2 * it + 1) * 64 + lane];
      d = (d - col_sum<L>(d * c)) * __builtin_amdgcn_rcpf(col_sum<L>(before) + pad);
      d = valid ? d : 0.f;
      c = before;
      before = hist[(2 * it) * 64 + lane];
      d = (d - row_sum<L>(d * c)) * __builtin_amdgcn_rcpf(row_sum<L>(before) + pad);
      d = valid ? d : 0.f;
      c = before;
    }
    if (valid) dzs[tu][r] = d * c;
  }
  __syncthreads();
  for (int k = 0; k < NU && t0 + k < T; ++k) {
    const size_t t = t0 + k;
    const float rinv = rms_inverse(raw[k][R], n, eps);
    float gm[3] = {0.f, 0.f, 0.f};
    for (int r = lane; r < 16 * NRT; r += 64) {
      float uv = 0.f;
      if (r < R) {
        const int grp = r < S ? 0 : r < 2 * S ? 1 : 2;
        const float dz = dzs[k][r], p = dz * (raw[k][r] * rinv);
        gm[0] += grp == 0 ? p : 0.f;
        gm[1] += grp == 1 ? p : 0.f;
        gm[2] += grp == 2 ? p : 0.f;
        uv = scale[grp] * dz * rinv;
        red[(size_t)r * T + t] = dz;
      }
      u_out[t * (16 * NRT) + r] = uv;
    }
    float dot = 0.f;
    for (int q = 0; q < 3; ++q) {
      gm[q] = sum_wave(gm[q]);
      dot = fmaf(scale[q], gm[q], dot);
    }
    if (lane == 0) {
      side[t * (S + 1) + S] = -dot * rinv * rinv / (float)n;
      for (int q = 0; q < 3; ++q) red[(size_t)(R + q) * T + t] = gm[q];
    }
  }
}

// ---------------------------------------------------------------- stream
// A wave owns 64 columns (lane: quad r16 of 16) and walks a range of tokens 16
// at a time; lane group g holds tokens 4g .. 4g+3 of them, four columns each.
//   dx: D[token][column] = u W on v_mfma_f32_16x16x4_f32, started from the
//       vector sum dx_in + pre dy + alpha x; W stays in registers.
//   dW: D[row][column] += u^T x over four tokens (one per lane group), with x
//       as it was loaded: both products use the layout of the loads.
template <int S, bool F8>
__global__ __launch_bounds__(256) void pre_bwd_stream_kernel(
    const void* __restrict__ x, const unsigned char* __restrict__ xs,
    const float* __restrict__ w, const float* __restrict__ dy, const float* __restrict__ u,
    const float* __restrict__ side, const float* dx_in, int T, int H, int KB, int SB, int chunk,
    float* dx, float* __restrict__ dw_part) {
  constexpr int R = rows_of(S), NRT = row_tiles(S), KS = (R + 3) / 4, RP = 16 * NRT;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane & 15, g = lane >> 4;
  const int ci = blockIdx.x / SB, HQ = H >> 2, n4 = S * HQ;
  const int cq = ((blockIdx.x - ci * SB) * 4 + wave) * 16 + r16;
  const bool in = cq < n4;
  const int cs = in ? cq / HQ : 0, q = in ? cq - cs * HQ : 0;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const float4* w4 = reinterpret_cast<const float4*>(w);
  float4 wv[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s)
    wv[s] = in && 4 * s + g < R ? w4[(size_t)(4 * s + g) * n4 + cq] : zero;
  floatx4 dw[NRT][4];
#pragma unroll
  for (int i = 0; i < NRT; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) dw[i][k] = floatx4{0.f, 0.f, 0.f, 0.f};
  const int t_end = min((ci + 1) * chunk, T);
  for (int t0 = ci * chunk; t0 < t_end; t0 += 16) {
    float4 xv[4];
    floatx4 acc[4];
    float ut[4][NRT];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + 4 * g + i;
      const bool live = t < t_end;
      const size_t tt = live ? t : t_end - 1;
      xv[i] = live && in ? x_quad<F8>(x, xs, tt * S + cs, HQ, KB, q) : zero;
      const float4 d = live && in ? reinterpret_cast<const float4*>(dy)[tt * HQ + q] : zero;
      const float4 o =
          live && in && dx_in ? reinterpret_cast<const float4*>(dx_in)[tt * n4 + cq] : zero;
      const float p = side[tt * (S + 1) + cs], al = side[tt * (S + 1) + S];
      acc[0][i] = fmaf(al, xv[i].x, fmaf(p, d.x, o.x));
      acc[1][i] = fmaf(al, xv[i].y, fmaf(p, d.y, o.y));
      acc[2][i] = fmaf(al, xv[i].z, fmaf(p, d.z, o.z));
      acc[3][i] = fmaf(al, xv[i].w, fmaf(p, d.w, o.w));
#pragma unroll
      for (int k = 0; k < NRT; ++k) ut[i][k] = live ? u[tt * RP + 16 * k + r16] : 0.f;
    }
    const size_t ta = min(t0 + r16, t_end - 1);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const float ua = u[ta * RP + 4 * s + g];
      acc[0] = __builtin_amdgcn_mfma_f32_16x16x4f32(ua, wv[s].x, acc[0], 0, 0, 0);
      acc[1] = __builtin_amdgcn_mfma_f32_16x16x4f32(ua, wv[s].y, acc[1], 0, 0, 0);
      acc[2] = __builtin_amdgcn_mfma_f32_16x16x4f32(ua, wv[s].z, acc[2], 0, 0, 0);
      acc[3] = __builtin_amdgcn_mfma_f32_16x16x4f32(ua, wv[s].w, acc[3], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < NRT; ++k) {
        dw[k][0] = __builtin_amdgcn_mfma_f32_16x16x4f32(ut[i][k], xv[i].x, dw[k][0], 0, 0, 0);
        dw[k][1] = __builtin_amdgcn_mfma_f32_16x16x4f32(ut[i][k], xv[i].y, dw[k][1], 0, 0, 0);
        dw[k][2] = __builtin_amdgcn_mfma_f32_16x16x4f32(ut[i][k], xv[i].z, dw[k][2], 0, 0, 0);
        dw[k][3] = __builtin_amdgcn_mfma_f32_16x16x4f32(ut[i][k], xv[i].w, dw[k][3], 0, 0, 0);
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + 4 * g + i;
      if (t < t_end && in)
        reinterpret_cast<float4*>(dx)[(size_t)t * n4 + cq] =
            make_float4(acc[0][i], acc[1][i], acc[2][i], acc[3][i]);
    }
  }
  if (!in) return;
  float4* o4 = reinterpret_cast<float4*>(dw_part) + (size_t)ci * R * n4 + cq;
#pragma unroll
  for (int k = 0; k < NRT; ++k)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int r = 16 * k + 4 * g + v;
      if (r < R)
        o4[(size_t)r * n4] = make_float4(dw[k][0][v], dw[k][1][v], dw[k][2][v], dw[k][3][v]);
    }
}

// ---------------------------------------------------------------- sums
// The first rblocks blocks add red [R + 3][T] over tokens (one row each), the
// rest add the chunks of dW in order, a quad per thread.
__global__ __launch_bounds__(256) void pre_bwd_sums_kernel(const float* __restrict__ red, int T,
                                                           int R, const float* __restrict__ part,
                                                           int chunks, long quads,
                                                           float* __restrict__ dw,
                                                           float* __restrict__ dscale,
                                                           float* __restrict__ dbase) {
  const int row = blockIdx.x;
  if (row < R + 3) {
    __shared__ float sums[4];
    float s = 0.f;
    for (int t = threadIdx.x; t < T; t += 256) s += red[(size_t)row * T + t];
    s = sum_wave(s);
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
      const float v = (sums[0] + sums[1]) + (sums[2] + sums[3]);
      if (row < R)
        dbase[row] = v;
      else
        dscale[row - R] = v;
    }
    return;
  }
  const long i = (long)(row - R - 3) * 256 + threadIdx.x;
  if (i >= quads) return;
  const float4* p = reinterpret_cast<const float4*>(part) + i;
  float4 s = chunks > 0 ? p[0] : make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = 1; c < chunks; ++c) {
    const float4 v = p[c * quads];
    s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
  }
  reinterpret_cast<float4*>(dw)[i] = s;
}

namespace {

// The split of a call's work: G hidden ranges of `steps` steps (of 16 columns)
// for the dots, `chunks` token ranges of `chunk` for the stream, about 2048 waves
// each (8 per compute unit) where the shape has that many.
struct Plan {
  int G, steps, SB, chunk, chunks;
  size_t part, u, side, red, dw, floats;  // offsets and total, in floats
};
size_t round4(size_t v) { return (v + 63) / 64 * 64; }

Plan plan(int T, int S, int H) {
  Plan p;
  const int R = rows_of(S), HQ = H / 4, TB = (T + 15) / 16;
  const int hs = (HQ + 3) / 4;
  int g = 512 / TB;
  const int gmax = (hs + 15) / 16;
  g = g < 1 ? 1 : g > gmax ? gmax : g;
  p.steps = (hs + g - 1) / g;
  p.G = (hs + p.steps - 1) / p.steps;
  const int strips = (S * HQ + 15) / 16;
  p.SB = (strips + 3) / 4;
  int c = 512 / p.SB;
  const int cmax = (T + 63) / 64;
  c = c < 1 ? 1 : c > cmax ? cmax : c;
  p.chunk = ((T + c - 1) / c + 15) / 16 * 16;
  p.chunks = (T + p.chunk - 1) / p.chunk;
  size_t at = 0;
  p.part = at;
  at += round4((size_t)p.G * T * (R + 1 + S));
  p.u = at;
  at += round4((size_t)T * 16 * ((R + 15) / 16));
  p.side = at;
  at += round4((size_t)T * (S + 1));
  p.red = at;
  at += round4((size_t)T * (R + 3));
  p.dw = at;
  if (p.chunks > 1) at += round4((size_t)p.chunks * R * S * H);
  p.floats = at;
  return p;
}

template <int S, bool F8>
void run(const PreBwd& a, int T, int H, int iters, float eps, float* work, hipStream_t st) {
  constexpr int R = rows_of(S), NU = S <= 4 ? 4 : 1;
  const int KB = (H + kF8Block - 1) / kF8Block, n = S * H;
  if (T == 0) {  // sums of no tokens
    const long quads = (long)R * n / 4;
    hipLaunchKernelGGL(pre_bwd_sums_kernel, dim3((unsigned)(R + 3 + (quads + 255) / 256)),
                       dim3(256), 0, st, nullptr, 0, R, nullptr, 0, quads, a.dfn_w, a.dscale,
                       a.dbase);
    return;
  }
  const Plan p = plan(T, S, H);
  float *part = work + p.part, *u = work + p.u, *side = work + p.side, *red = work + p.red;
  float* dw = p.chunks > 1 ? work + p.dw : a.dfn_w;
  hipLaunchKernelGGL((pre_bwd_dots_kernel<S, F8>), dim3((unsigned)((T + 15) / 16 * p.G)),
                     dim3(256), 0, st, a.x, a.x_scales, a.fn_w, a.dy, T, H, KB, p.G, p.steps,
                     part);
  hipLaunchKernelGGL((pre_bwd_gates_kernel<S>), dim3((unsigned)((T + NU - 1) / NU)), dim3(64),
                     (size_t)iters * 2 * 64 * sizeof(float), st, part, p.G, T, n, a.scale,
                     a.base, iters, eps, a.dpre, a.dpost, a.dcomb, u, side, red);
  hipLaunchKernelGGL((pre_bwd_stream_kernel<S, F8>), dim3((unsigned)(p.SB * p.chunks)),
                     dim3(256), 0, st, a.x, a.x_scales, a.fn_w, a.dy, u, side, a.dx_in, T, H, KB,
                     p.SB, p.chunk, a.dx, dw);
  const long quads = p.chunks > 1 ? (long)R * n / 4 : 0;
  hipLaunchKernelGGL(pre_bwd_sums_kernel, dim3((unsigned)(R + 3 + (quads + 255) / 256)),
                     dim3(256), 0, st, red, T, R, dw, p.chunks, quads, a.dfn_w, a.dscale,
                     a.dbase);
}
template <int S>
void run_s(const PreBwd& a, int T, int H, int iters, float eps, float* work, hipStream_t st) {
  a.x_scales ? run<S, true>(a, T, H, iters, eps, work, st)
             : run<S, false>(a, T, H, iters, eps, work, st);
}

}  // namespace

size_t pre_bwd_work_bytes(int T, int S, int H) {
  return T > 0 ? plan(T, S, H).floats * sizeof(float) : 0;
}

// The history of the rounds lies in 64 KiB of LDS beside the staged dots.
int pre_bwd_max_iters() { return 120; }

hipError_t launch_pre_bwd(const PreBwd& a, int T, int S, int H, int iters, float eps, void* work,
                          hipStream_t st) {
  float* wk = static_cast<float*>(work);
  switch (S) {
#define MHC_S(SS)                           \
  case SS:                                  \
    run_s<SS>(a, T, H, iters, eps, wk, st); \
    break;
    MHC_S(1) MHC_S(2) MHC_S(3) MHC_S(4) MHC_S(5) MHC_S(6) MHC_S(7) MHC_S(8)
#undef MHC_S
    default:
      return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace mhc
