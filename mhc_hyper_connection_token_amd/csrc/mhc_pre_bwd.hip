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

__device__ __forceinline__ float fma4(float4 a, float4 b, float acc) {
  acc = fmaf(a.x, b.x, acc);
  acc = fmaf(a.y, b.y, acc);
  acc = fmaf(a.z, b.z, acc);
  return fmaf(a.w, b.w, acc);
}
}  // namespace

// ---------------------------------------------------------------- weight planes
// An fp32 value as three bf16 of eight bits each, high to low: v = p0 + p1 + p2
// exactly (v cut at 8 bits, the rest cut at 8 bits, and what is left).
__device__ __forceinline__ void planes(float v, float& p0, float& p1, float& p2) {
  p0 = __uint_as_float(__float_as_uint(v) & 0xffff0000u);
  const float rest = v - p0;
  p1 = __uint_as_float(__float_as_uint(rest) & 0xffff0000u);
  p2 = rest - p1;
}
// The bf16 in the upper halves of two floats, as one dword.
__device__ __forceinline__ unsigned upper_halves(float lo, float hi) {
  return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}
// Eight fp32 values to their planes, one matrix operand each.
__device__ __forceinline__ void planes8(float4 a, float4 b, bf16x8 out[3]) {
  const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float p[3][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) planes(v[i], p[0][i], p[1][i], p[2][i]);
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    union {
      unsigned u[4];
      bf16x8 v;
    } o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.u[i] = upper_halves(p[k][2 * i], p[k][2 * i + 1]);
    out[k] = o.v;
  }
}

// The dots' order of a slice of 64 hidden columns: step ks = 2j + s of four,
// lane half h, holds columns 32j + 16h + 8s .. +7.  The 16 codes of chunk 2j + h
// of a row, one load of a lane, serve steps 2j and 2j + 1.
__device__ __forceinline__ int dots_column(int ks, int h) {
  return 32 * (ks >> 1) + 16 * h + 8 * (ks & 1);
}

// W [R][S*H] as row operands of the dots: for stream c, slice, step, plane and
// row tile of 32, 64 lanes of eight bf16 (row = lane % 32), zeros past R and H.
__global__ __launch_bounds__(256) void pre_bwd_planes_kernel(const float* __restrict__ w, int R,
                                                             int NRT, int S, int H, int HS,
                                                             long total,
                                                             bf16x8* __restrict__ out) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  const int lane = (int)(i & 63);
  const long f = i >> 6;
  const int rt = (int)(f % NRT);
  const long step = f / NRT;  // (c * HS + slice) * 4 + ks
  const int ks = (int)(step & 3), cs = (int)(step >> 2), c = cs / HS, slice = cs - c * HS;
  const int row = 32 * rt + (lane & 31), col = 64 * slice + dots_column(ks, lane >> 5);
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* p = w + ((size_t)row * S + c) * H + col;
  const float4 a = row < R && col < H ? *reinterpret_cast<const float4*>(p) : zero;
  const float4 b = row < R && col + 4 < H ? *reinterpret_cast<const float4*>(p + 4) : zero;
  bf16x8 o[3];
  planes8(a, b, o);
#pragma unroll
  for (int k = 0; k < 3; ++k) out[((step * 3 + k) * NRT + rt) * 64 + lane] = o[k];
}

// ---------------------------------------------------------------- dots
// part[G][T][R + 1 + S]: the R dots, the sum of squares, the S products with dy.
// A wave takes 32*TT tokens and `steps` slices of 64 hidden columns in all S
// streams; the four waves of a block take neighbouring ranges and are added up
// in LDS, the G blocks of a token group by the gates kernel.
// The dots run on v_mfma_f32_32x32x16_bf16 with W in three planes.  A decoded
// code is exact in bf16, so three products give fp32 dots; an fp32 x is cut into
// planes as well and takes six (the three left out are below 2^-24).  Against
// v_mfma_f32_16x16x4_f32 this is 16/3 (or 16/6) of the rate.
template <int S, bool F8, int TT>
__global__ __launch_bounds__(256, 2) void pre_bwd_dots_kernel(
    const void* __restrict__ x, const unsigned char* __restrict__ xs,
    const bf16x8* __restrict__ wp, const float* __restrict__ dy, int T, int H, int KB, int G,
    int HS, int steps, float* __restrict__ part) {
  constexpr int R = rows_of(S), NRT = (R + 31) / 32, V = R + 1 + S, VP = 32 * NRT + 1 + S;
  constexpr int UC = S <= 4 ? S : 1;  // unrolled further, the streams' loads spill
  __shared__ float sums[4][32 * TT][VP];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 31, h = lane >> 5;
  const int tb = blockIdx.x / G, gi = blockIdx.x - tb * G, HQ = H >> 2;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  size_t t[TT];
#pragma unroll
  for (int k = 0; k < TT; ++k) t[k] = min((tb * TT + k) * 32 + r, T - 1);
  floatx16 acc[TT][NRT];
  float ss[TT], dp[TT][S];
#pragma unroll
  for (int k = 0; k < TT; ++k) {
    ss[k] = 0.f;
#pragma unroll
    for (int c = 0; c < S; ++c) dp[k][c] = 0.f;
#pragma unroll
    for (int i = 0; i < NRT; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[k][i][v] = 0.f;
  }
  const int s0 = (gi * 4 + wave) * steps, s1 = min(s0 + steps, HS);
  for (int sl = s0; sl < s1; ++sl) {
    float4 d[TT][4][2];
#pragma unroll
    for (int k = 0; k < TT; ++k)
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const int q = 16 * sl + dots_column(ks, h) / 4;
        const float4* p = reinterpret_cast<const float4*>(dy) + t[k] * HQ;
        d[k][ks][0] = q < HQ ? p[q] : zero;
        d[k][ks][1] = q + 1 < HQ ? p[q + 1] : zero;
      }
#pragma unroll UC
    for (int c = 0; c < S; ++c) {
      float dc[TT];
#pragma unroll
      for (int k = 0; k < TT; ++k) dc[k] = 0.f;
      const bf16x8* wc = wp + (size_t)(c * HS + sl) * 4 * 3 * NRT * 64 + lane;
      intx4 code[TT][2];
      float scale[TT];
      if constexpr (F8) {
#pragma unroll
        for (int k = 0; k < TT; ++k) {
          const size_t row = t[k] * S + c;
          const intx4* p = static_cast<const intx4*>(x) + row * KB * 8 + 4 * sl + h;
          code[k][0] = p[0];
          code[k][1] = p[2];
          scale[k] = f8_scale(xs[row * KB + (sl >> 1)]);
        }
      }
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        bf16x8 wv[3][NRT];
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
          for (int i = 0; i < NRT; ++i) wv[p][i] = wc[((ks * 3 + p) * NRT + i) * 64];
#pragma unroll
        for (int k = 0; k < TT; ++k) {
          float4 xa, xb;
          bf16x8 xp[3];
          if constexpr (F8) {
            const intx4 q = code[k][ks >> 1];
            xp[0] = f8_to_bf16(q[2 * (ks & 1)], q[2 * (ks & 1) + 1], scale[k]);
            union {
              bf16x8 v;
              unsigned u[4];
            } o;
            o.v = xp[0];
            xa = make_float4(__uint_as_float(o.u[0] << 16), __uint_as_float(o.u[0] & 0xffff0000u),
                             __uint_as_float(o.u[1] << 16), __uint_as_float(o.u[1] & 0xffff0000u));
            xb = make_float4(__uint_as_float(o.u[2] << 16), __uint_as_float(o.u[2] & 0xffff0000u),
                             __uint_as_float(o.u[3] << 16), __uint_as_float(o.u[3] & 0xffff0000u));
          } else {
            const int q = 16 * sl + dots_column(ks, h) / 4;
            const float4* p = static_cast<const float4*>(x) + (t[k] * S + c) * HQ;
            xa = q < HQ ? p[q] : zero;
            xb = q + 1 < HQ ? p[q + 1] : zero;
            planes8(xa, xb, xp);
          }
          ss[k] = fma4(xb, xb, fma4(xa, xa, ss[k]));
          dc[k] = fma4(d[k][ks][1], xb, fma4(d[k][ks][0], xa, dc[k]));
#pragma unroll
          for (int i = 0; i < NRT; ++i) {
#pragma unroll
            for (int p = 0; p < 3; ++p)
#pragma unroll
              for (int m = 0; m < (F8 ? 1 : 3 - p); ++m)
                acc[k][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wv[p][i], xp[m], acc[k][i],
                                                                    0, 0, 0);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < TT; ++k)
#pragma unroll
        for (int i = 0; i < S; ++i) dp[k][i] += i == c ? dc[k] : 0.f;
    }
  }
#pragma unroll
  for (int k = 0; k < TT; ++k) {
    float* mine = sums[wave][32 * k + r];
#pragma unroll
    for (int i = 0; i < NRT; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) mine[32 * i + 8 * (v >> 2) + 4 * h + (v & 3)] = acc[k][i][v];
    const float s = swap32_sum(ss[k]);
    if (h == 0) mine[32 * NRT] = s;
#pragma unroll
    for (int c = 0; c < S; ++c) {
      const float v = swap32_sum(dp[k][c]);
      if (h == 0) mine[32 * NRT + 1 + c] = v;
    }
  }
  __syncthreads();
  const int first = tb * 32 * TT;
  for (int i = threadIdx.x; i < 32 * TT * V; i += 256) {
    const int k = i / V, v = i - k * V, at = v < R ? v : v - R + 32 * NRT;
    if (first + k < T)
      part[((size_t)gi * T + first + k) * V + v] =
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
  // what one step of 16 tokens reads; the next step's is on its way while this
  // one is computed
  struct Step {
    unsigned code[4], byte[4];
    float4 x[4], d[4], o[4];
    float p[4], al[4], ut[4][NRT], ua[KS];
  };
  auto load = [&](int t0, Step& n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const size_t t = min(t0 + 4 * g + i, t_end - 1);
      if constexpr (F8) {
        const size_t row = t * S + cs;
        n.code[i] = static_cast<const unsigned*>(x)[row * KB * 32 + q];
        n.byte[i] = xs[row * KB + (q >> 5)];
      } else {
        n.x[i] = static_cast<const float4*>(x)[(t * S + cs) * HQ + q];
      }
      n.d[i] = reinterpret_cast<const float4*>(dy)[t * HQ + q];
      n.o[i] = dx_in ? reinterpret_cast<const float4*>(dx_in)[t * n4 + (in ? cq : 0)] : zero;
      n.p[i] = side[t * (S + 1) + cs];
      n.al[i] = side[t * (S + 1) + S];
#pragma unroll
      for (int k = 0; k < NRT; ++k) n.ut[i][k] = u[t * RP + 16 * k + r16];
    }
    const size_t ta = min(t0 + r16, t_end - 1);
#pragma unroll
    for (int s = 0; s < KS; ++s) n.ua[s] = u[ta * RP + 4 * s + g];
  };
  Step next;
  load(ci * chunk, next);
  for (int t0 = ci * chunk; t0 < t_end; t0 += 16) {
    Step now = next;
    if (t0 + 16 < t_end) load(t0 + 16, next);
    floatx4 acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool live = t0 + 4 * g + i < t_end;
      if constexpr (F8) now.x[i] = f8_unpack(now.code[i], f8_scale(now.byte[i]));
      const float4 xv = now.x[i], d = now.d[i], o = now.o[i];
      acc[0][i] = fmaf(now.al[i], xv.x, fmaf(now.p[i], d.x, o.x));
      acc[1][i] = fmaf(now.al[i], xv.y, fmaf(now.p[i], d.y, o.y));
      acc[2][i] = fmaf(now.al[i], xv.z, fmaf(now.p[i], d.z, o.z));
      acc[3][i] = fmaf(now.al[i], xv.w, fmaf(now.p[i], d.w, o.w));
      // a token past the end (the last one again) adds nothing to dW
      if (!live) {
        now.x[i] = zero;
#pragma unroll
        for (int k = 0; k < NRT; ++k) now.ut[i][k] = 0.f;
      }
    }
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      acc[0] = __builtin_amdgcn_mfma_f32_16x16x4f32(now.ua[s], wv[s].x, acc[0], 0, 0, 0);
      acc[1] = __builtin_amdgcn_mfma_f32_16x16x4f32(now.ua[s], wv[s].y, acc[1], 0, 0, 0);
      acc[2] = __builtin_amdgcn_mfma_f32_16x16x4f32(now.ua[s], wv[s].z, acc[2], 0, 0, 0);
      acc[3] = __builtin_amdgcn_mfma_f32_16x16x4f32(now.ua[s], wv[s].w, acc[3], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < NRT; ++k) {
        const float a = now.ut[i][k];
        dw[k][0] = __builtin_amdgcn_mfma_f32_16x16x4f32(a, now.x[i].x, dw[k][0], 0, 0, 0);
        dw[k][1] = __builtin_amdgcn_mfma_f32_16x16x4f32(a, now.x[i].y, dw[k][1], 0, 0, 0);
        dw[k][2] = __builtin_amdgcn_mfma_f32_16x16x4f32(a, now.x[i].z, dw[k][2], 0, 0, 0);
        dw[k][3] = __builtin_amdgcn_mfma_f32_16x16x4f32(a, now.x[i].w, dw[k][3], 0, 0, 0);
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

// The split of a call's work: token groups of 32*TT tokens times G ranges of the
// hidden axis for the dots (4 waves, `steps` slices each), `chunks` token ranges
// of `chunk` for the stream, about 2048 waves each (8 per compute unit) where the
// shape has that many.
struct Plan {
  int TT, G, HS, steps, SB, chunk, chunks;
  size_t planes, part, u, side, red, dw, floats;  // offsets and total, in floats
};
size_t round64(size_t v) { return (v + 63) / 64 * 64; }
int div_up(int a, int b) { return (a + b - 1) / b; }

Plan plan(int T, int S, int H, bool f8) {
  Plan p;
  const int R = rows_of(S);
  p.TT = f8 && S <= 4 && T >= 1024 ? 2 : 1;
  p.HS = div_up(H, 64);
  const int groups = div_up(T, 32 * p.TT);
  const int want = div_up(512, groups);
  p.steps = div_up(p.HS, 4 * want);
  p.G = div_up(p.HS, 4 * p.steps);
  p.SB = div_up(S * (H / 4), 64);
  int c = 512 / p.SB;
  const int cmax = div_up(T, 64);
  c = c < 1 ? 1 : c > cmax ? cmax : c;
  p.chunk = div_up(div_up(T, c), 16) * 16;
  p.chunks = div_up(T, p.chunk);
  size_t at = 0;
  p.planes = at;  // 64 lanes of 16 bytes for each step, plane and row tile
  at += (size_t)S * p.HS * 4 * 3 * div_up(R, 32) * 64 * 4;
  p.part = at;
  at += round64((size_t)p.G * T * (R + 1 + S));
  p.u = at;
  at += round64((size_t)T * 16 * div_up(R, 16));
  p.side = at;
  at += round64((size_t)T * (S + 1));
  p.red = at;
  at += round64((size_t)T * (R + 3));
  p.dw = at;
  if (p.chunks > 1) at += round64((size_t)p.chunks * R * S * H);
  p.floats = at;
  return p;
}

template <int S, bool F8, int TT>
void dots(const PreBwd& a, const Plan& p, int T, int H, int KB, float* work, hipStream_t st) {
  hipLaunchKernelGGL((pre_bwd_dots_kernel<S, F8, TT>),
                     dim3((unsigned)(div_up(T, 32 * TT) * p.G)), dim3(256), 0, st, a.x,
                     a.x_scales, reinterpret_cast<const bf16x8*>(work + p.planes), a.dy, T, H,
                     KB, p.G, p.HS, p.steps, work + p.part);
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
  const Plan p = plan(T, S, H, F8);
  float *part = work + p.part, *u = work + p.u, *side = work + p.side, *red = work + p.red;
  float* dw = p.chunks > 1 ? work + p.dw : a.dfn_w;
  constexpr int NRT = (R + 31) / 32;
  const long frags = (long)S * p.HS * 4 * NRT * 64;
  hipLaunchKernelGGL(pre_bwd_planes_kernel, dim3((unsigned)((frags + 255) / 256)), dim3(256), 0,
                     st, a.fn_w, R, NRT, S, H, p.HS, frags,
                     reinterpret_cast<bf16x8*>(work + p.planes));
  if constexpr (F8 && S <= 4) {
    if (p.TT == 2)
      dots<S, F8, 2>(a, p, T, H, KB, work, st);
    else
      dots<S, F8, 1>(a, p, T, H, KB, work, st);
  } else {
    dots<S, F8, 1>(a, p, T, H, KB, work, st);
  }
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
  if (T < 1) return 0;
  const size_t a = plan(T, S, H, false).floats, b = plan(T, S, H, true).floats;
  return (a > b ? a : b) * sizeof(float);
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
