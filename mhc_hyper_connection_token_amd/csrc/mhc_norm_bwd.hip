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
// parts up, in an order fixed by the shape.  HBM-bound: branch_norm_bwd of 1001 x 7168 in fp32
// 22 us (3.9 TB/s, the parts not counted), 4096 x 4096 in fp32 37 (5.4), from an 8-bit y and
// a bf16 gradient 30 (3.9); site_post_norm_bwd of 4096 tokens of 4 x 4096 with an 8-bit state, a
// bf16 branch and gate 146 us (5.5), in fp32 171 (5.5), 1024 of 8 x 7168 149 (4.1: the sums of
// eight streams take the registers that would hide the loads).
#include "mhc_norm_bwd.h"

namespace mhc {

namespace {
// Parts of a sum over tokens, blocks of the first launch: eight waves for each unit.  More
// parts are more to write and to read again: 1001 tokens of 7168 22 us with 256 of eight
// waves, 25 with 512, 33 with 1024; 8192 of 256 16 us with 1024 of one wave, 17
// with 2048, 22 with 256.
// A few short rows are one block's: it writes the sums themselves, without the second launch.
int parts_of(int T, int H) {
  if (H <= kOneWaveHidden && T <= 4) return T < 1 ? T : 1;
  const int most = H <= kOneWaveHidden ? 1024 : 256;
  return T < most ? T : most;
}
}  // namespace

template <int NW, int Q, int DZ, int Y>
__global__ __launch_bounds__(64 * NW) void branch_norm_bwd_kernel(NormBwd p, int T, int HQ,
                                                                   int KB, float eps,
                                                                   float* __restrict__ part) {
  constexpr int NT = 64 * NW;
  __shared__ float buf[2][NW][2];
  const float inv_h = 1.f / (float)(4 * HQ);
  float4 w[Q], dw[Q];
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int q = threadIdx.x + NT * i;
    w[i] = q < HQ ? reinterpret_cast<const float4*>(p.nw)[q] : zero4();
    dw[i] = zero4();
  }
  Raw<DZ> zn[Q];
  Raw<Y> yn[Q];  // the next token's, asked for while this one's sums are added up
  auto fetch = [&](size_t t) {
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const int q = min((int)threadIdx.x + NT * i, HQ - 1);
      zn[i] = load_raw<DZ>(p.dz, nullptr, t, HQ, KB, q);
      yn[i] = load_raw<Y>(p.y, p.y_scales, t, HQ, KB, q);
    }
  };
  fetch(blockIdx.x);
  int at = 0;
  for (size_t t = blockIdx.x; t < (size_t)T; t += gridDim.x, at ^= 1) {
    float4 y[Q], dz[Q];
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const bool in = (int)threadIdx.x + NT * i < HQ;
      y[i] = in ? raw_values(yn[i]) : zero4();
      dz[i] = in ? raw_values(zn[i]) : zero4();
      sum[0] = sq4(y[i], sum[0]);
      sum[1] = dot4(mul4(dz[i], w[i]), y[i], sum[1]);
    }
    if (t + gridDim.x < (size_t)T) fetch(t + gridDim.x);
    block_sums<2, NW>(sum, buf[at]);
    const float r = rms_inverse(sum[0], 4 * HQ, eps);
    const float c = -(sum[1] * r) * r * inv_h * r;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const int q = threadIdx.x + NT * i;
      if (q < HQ)
        store_out(p.dy + (t * HQ + q) * 4,
                  fma4(make_float4(c, c, c, c), y[i], scale4(mul4(dz[i], w[i]), r)), p.stream);
      dw[i] = fma4(dz[i], scale4(y[i], r), dw[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int q = threadIdx.x + NT * i;
    if (q < HQ) reinterpret_cast<float4*>(part)[(size_t)blockIdx.x * HQ + q] = dw[i];
  }
}

// out[i] = sum of n rows part[k][i]: a block takes 16 quads, thread (g, c) the rows g, g + RG,
// ... of quad c, eight at a time on their way.
template <int RG>
__global__ __launch_bounds__(16 * RG) void sum_rows_kernel(const float* __restrict__ part, int n,
                                                           int HQ, float* __restrict__ out,
                                                           const float* __restrict__ part2,
                                                           float* __restrict__ out2) {
  __shared__ float4 acc[RG][16];
  const int c = threadIdx.x & 15, g = threadIdx.x >> 4, q = blockIdx.x * 16 + c;
  const float4* src = reinterpret_cast<const float4*>(blockIdx.y ? part2 : part);
  float4 s = zero4();
  if (q < HQ)
    for (int k = g; k < n; k += 8 * RG) {
      float4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        v[u] = k + u * RG < n ? src[(size_t)(k + u * RG) * HQ + q] : zero4();
#pragma unroll
      for (int u = 0; u < 8; ++u) s = add4(s, v[u]);
    }
  acc[g][c] = s;
  __syncthreads();
#pragma unroll
  for (int m = RG / 2; m > 0; m >>= 1) {
    if (g < m) {
      s = add4(s, acc[g + m][c]);
      acc[g][c] = s;
    }
    __syncthreads();
  }
  if (g == 0 && q < HQ) reinterpret_cast<float4*>(blockIdx.y ? out2 : out)[q] = s;
}

size_t norm_bwd_work_bytes(int T, int H, int sums) {
  const int n = parts_of(T, H);
  return n > 1 ? (size_t)n * H * 4 * sums : 0;
}

namespace {
// The sums of part into out, and of part2 into out2 where that is given.
void sum_rows(const float* part, int n, int HQ, float* out, const float* part2, float* out2,
              hipStream_t st) {
  const dim3 grid((HQ + 15) / 16, out2 ? 2 : 1);  // n = 0 gives zeros
  if (n > 32)
    hipLaunchKernelGGL(sum_rows_kernel<64>, grid, dim3(1024), 0, st, part, n, HQ, out, part2,
                       out2);
  else
    hipLaunchKernelGGL(sum_rows_kernel<16>, grid, dim3(256), 0, st, part, n, HQ, out, part2,
                       out2);
}
}  // namespace

namespace {
template <int DZ, int Y>
void launch_norm_bwd_k(const NormBwd& p, int T, int HQ, int KB, float eps, float* part, int n,
                       hipStream_t st) {
#define MHC_NORM(W, Q)                                                                   \
  hipLaunchKernelGGL((branch_norm_bwd_kernel<W, Q, DZ, Y>), dim3((unsigned)n), dim3(64 * W), 0, \
                     st, p, T, HQ, KB, eps, part)
  if (HQ * 4 <= kOneWaveHidden)
    MHC_NORM(1, 4);
  else if (HQ <= 1024)
    MHC_NORM(8, 2);
  else
    MHC_NORM(8, 4);
#undef MHC_NORM
}
}  // namespace

hipError_t launch_norm_bwd(const NormBwd& call, int T, int H, float eps, void* work,
                           hipStream_t st) {
  NormBwd p = call;
  p.stream = (size_t)T * H * 4 > kCacheBytes;
  const int HQ = H / 4, KB = (H + kF8Block - 1) / kF8Block, n = parts_of(T, H);
  float* part = n == 1 ? p.dnw : static_cast<float*>(work);
  if (n > 0) {
    if (p.dz_kind == kF32)
      p.y_scales ? launch_norm_bwd_k<kF32, kF8>(p, T, HQ, KB, eps, part, n, st)
                 : launch_norm_bwd_k<kF32, kF32>(p, T, HQ, KB, eps, part, n, st);
    else
      p.y_scales ? launch_norm_bwd_k<kBF16, kF8>(p, T, HQ, KB, eps, part, n, st)
                 : launch_norm_bwd_k<kBF16, kF32>(p, T, HQ, KB, eps, part, n, st);
  }
  if (n != 1) sum_rows(part, n, HQ, p.dnw, nullptr, nullptr, st);
  return hipGetLastError();
}

hipError_t launch_post_norm_bwd(const PostNormBwd& call, int T, int S, int H, float eps,
                                void* work, hipStream_t st) {
  PostNormBwd p = call;
  p.stream = (size_t)T * (S + 1) * H * 4 > kCacheBytes;
  const int HQ = H / 4, KB = (H + kF8Block - 1) / kF8Block, n = parts_of(T, H);
  float* part = n == 1 ? p.dnw : static_cast<float*>(work);
  float* gate_part = n == 1 ? p.dgate : part + (size_t)n * H;
  if (n > 0) {
    const auto launch = S <= 2   ? launch_post_norm_bwd_12
                        : S <= 4 ? launch_post_norm_bwd_34
                        : S <= 6 ? launch_post_norm_bwd_56
                                 : launch_post_norm_bwd_78;
    launch(p, T, S, HQ, KB, eps, part, n, gate_part, st);
  }
  if (n != 1)
    sum_rows(part, n, HQ, p.dnw, gate_part, p.gate && !p.gate_rows ? p.dgate : nullptr, st);
  return hipGetLastError();
}

}  // namespace mhc
