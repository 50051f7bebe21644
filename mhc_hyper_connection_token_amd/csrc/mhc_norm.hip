// mhc_norm.hip -- the norm before a branch, and the post mix with the norm behind it:
//   branch_norm     z[t,i] = y[t,i] * r_t * nw[i],  r_t = 1/sqrt(mean_i y[t,i]^2 + eps)
//   site_post_norm  h[t,i] = alpha * a(gate) * f[t,i] * r_t * nw[i]   (r_t of f)
//                   x'[t,k,i] = post[t,k] * h[t,i] + sum_j comb[t,j,k] * x[t,j,i]
// Both are one pass over memory: a token's row stays in the registers of the threads
// that sum its squares until r_t is known.  HBM-bound (a large copy runs at 6.6 TB/s):
// branch_norm of 4096 x 4096 to bf16 18.5 us, 5.4 TB/s; the post mix of 4096 tokens of 4 x 4096
// with a bf16 branch and gate 99 us, 6.1 TB/s, of 1024 of 8 x 7168 96 us, 5.2; one token 3.0 us
// a launch, latency.
#include "mhc_norm.h"

namespace mhc {

// ---------------------------------------------------------------- norm before a branch
// W waves hold a token's row, Q quads a thread; with W = 1 a block has four tokens.
template <int W, int Q, bool BF16>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void branch_norm_kernel(
    const float* __restrict__ y, const float* __restrict__ nw, int T, int HQ, float eps,
    void* __restrict__ z) {
  constexpr int NT = 64 * W;
  const int wave = threadIdx.x >> 6;
  const int t = W == 1 ? blockIdx.x * 4 + wave : blockIdx.x;
  const int tid = W == 1 ? threadIdx.x & 63 : threadIdx.x;
  if (W == 1 && t >= T) return;
  float4 v[Q];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int q = tid + NT * i;
    v[i] = q < HQ ? nt_load4(y + ((size_t)t * HQ + q) * 4) : zero4();
  }
#pragma unroll
  for (int i = 0; i < Q; ++i) ss = sq4(v[i], ss);
  ss = wave_total(ss);
  if constexpr (W > 1) {
    __shared__ float part[W];
    if ((threadIdx.x & 63) == 0) part[wave] = ss;
    __syncthreads();
    ss = part[0];
#pragma unroll
    for (int w = 1; w < W; ++w) ss += part[w];
  }
  const float r = rms_inverse(ss, 4 * HQ, eps);
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int q = tid + NT * i;
    if (q >= HQ) break;
    const float4 o = zq8_norm(v[i], r, reinterpret_cast<const float4*>(nw)[q]);
    if constexpr (BF16)
      reinterpret_cast<uintx2*>(z)[(size_t)t * HQ + q] = bf16_quad(o);
    else
      reinterpret_cast<float4*>(z)[(size_t)t * HQ + q] = o;
  }
}

namespace {
template <int W, int Q>
void launch_branch_norm_at(const float* y, const float* nw, int T, int HQ, float eps, void* z,
                           bool bf16, hipStream_t st) {
  const dim3 grid((unsigned)(W == 1 ? (T + 3) / 4 : T)), block(W == 1 ? 256 : 64 * W);
  if (bf16)
    hipLaunchKernelGGL((branch_norm_kernel<W, Q, true>), grid, block, 0, st, y, nw, T, HQ, eps, z);
  else
    hipLaunchKernelGGL((branch_norm_kernel<W, Q, false>), grid, block, 0, st, y, nw, T, HQ, eps,
                       z);
}
}  // namespace

hipError_t launch_branch_norm(const float* y, const float* nw, int T, int H, float eps, void* z,
                              bool bf16, hipStream_t st) {
  const int HQ = H / 4;
  if (HQ <= 64)
    launch_branch_norm_at<1, 1>(y, nw, T, HQ, eps, z, bf16, st);
  else if (HQ <= 256)
    launch_branch_norm_at<1, 4>(y, nw, T, HQ, eps, z, bf16, st);
  else if (HQ <= 1024 && T > 2048)
    // more of a row in each thread, where the tokens' blocks of four waves no longer fit the chip
    // together; us with two and four waves: 1024, 2048, 2304 and 4096 tokens of 4096 to bf16 7.8 /
    // 6.8, 11.2 / 10.8, 12.1 / 12.8, 19.3 / 20.4, of 1028 3.7 / 3.5, 4.9 / 4.8, 5.2 / 5.6, 7.0 /
    // 7.8; one token 3.2 / 2.6
    launch_branch_norm_at<2, 8>(y, nw, T, HQ, eps, z, bf16, st);
  else if (HQ <= 1024)
    launch_branch_norm_at<4, 4>(y, nw, T, HQ, eps, z, bf16, st);
  else
    launch_branch_norm_at<8, 4>(y, nw, T, HQ, eps, z, bf16, st);
  return hipGetLastError();
}

// ---------------------------------------------------------------- post mix with the norm
template <int S>
__device__ __forceinline__ void mix_store(const float* pk, const float (*ck)[S], const float4* xv,
                                          float4 h, float* out, size_t t, int HQ, int q,
                                          int stream) {
#pragma unroll
  for (int k = 0; k < S; ++k)
    store_out(out + ((t * S + k) * HQ + q) * 4, post_mix4<S>(pk[k], &ck[0][k], S, xv, h, S),
              stream);
}

// A block takes NT*Q quads of a token (all HQ of them where PARTS is false: then the row of
// f that it sums is the row that it holds).  With PARTS the blocks of a token each sum
// the whole row: for few tokens.
template <int S, int F, int GATE, int NT, int Q, bool PARTS>
__global__ __launch_bounds__(NT) void post_norm_kernel(PostNorm p, int HQ, int parts, float eps) {
  constexpr int NW = NT / 64;
  const int part = PARTS ? blockIdx.x % parts : 0;
  const size_t t = PARTS ? blockIdx.x / parts : blockIdx.x;
  const int q0 = part * NT * Q + threadIdx.x;
  float pk[S], ck[S][S];
#pragma unroll
  for (int k = 0; k < S; ++k) pk[k] = p.post[t * S + k];
#pragma unroll
  for (int j = 0; j < S; ++j)
#pragma unroll
    for (int k = 0; k < S; ++k) ck[j][k] = p.comb[t * S * S + j * S + k];
  // threads past the row's end read its last quad, and neither count nor store it
  Raw<F> fv[Q];
  Raw<gate_kind<GATE>()> gv[Q];
  float4 xv[Q][S], w[Q];
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int q = min(q0 + NT * i, HQ - 1);
    fv[i] = load_raw<F>(p.f, nullptr, t, HQ, 0, q);
  }
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int q = min(q0 + NT * i, HQ - 1);
#pragma unroll
    for (int j = 0; j < S; ++j) xv[i][j] = nt_load4(p.x + ((t * S + j) * HQ + q) * 4);
    if constexpr (GATE != kNoGate)
      gv[i] = load_raw<gate_kind<GATE>()>(p.gate, nullptr, p.gate_rows ? t : 0, HQ, 0, q);
    w[i] = reinterpret_cast<const float4*>(p.nw)[q];
  }
  float ss = 0.f;
  if constexpr (PARTS) {
    for (int q = threadIdx.x; q < HQ; q += NT)
      ss = sq4(raw_values(load_raw<F>(p.f, nullptr, t, HQ, 0, q)), ss);
  } else {
#pragma unroll
    for (int i = 0; i < Q; ++i) ss = q0 + NT * i < HQ ? sq4(raw_values(fv[i]), ss) : ss;
  }
  ss = wave_total(ss);
  if constexpr (NW > 1) {
    __shared__ float sums[NW];
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = ss;
    __syncthreads();
    ss = sums[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) ss += sums[w];
  }
  const float ar = p.alpha * rms_inverse(ss, 4 * HQ, eps);
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int q = q0 + NT * i;
    if (q >= HQ) break;
    float4 h = mul4(scale4(raw_values(fv[i]), ar), w[i]);
    if constexpr (GATE != kNoGate) {
      float4 a, s;
      gate_quad<false>(raw_values(gv[i]), p.gate_act, a, s);
      h = mul4(h, a);
    }
    mix_store<S>(pk, ck, xv[i], h, p.x_out, t, HQ, q, p.stream);
  }
}

namespace {
template <int S, int F, int GATE, int NT, int Q, bool PARTS>
void launch_post_norm_at(const PostNorm& p, int T, int HQ, float eps, hipStream_t st) {
  const int parts = PARTS ? (HQ + NT * Q - 1) / (NT * Q) : 1;
  hipLaunchKernelGGL((post_norm_kernel<S, F, GATE, NT, Q, PARTS>), dim3((unsigned)T * parts),
                     dim3(NT), 0, st, p, HQ, parts, eps);
}
template <int S, int F, int GATE>
void launch_post_norm_g(const PostNorm& p, int T, int HQ, float eps, hipStream_t st) {
  if (HQ <= 256)
    launch_post_norm_at<S, F, GATE, 256, 1, false>(p, T, HQ, eps, st);
  else if (T <= (S > 4 || HQ <= 512 ? 64 : 24))
    // several blocks a token while they are few, us so and with one block, bf16 branch and gate: 4
    // streams of 4096 at 12, 24, 48 and 128 tokens 3.5 / 4.4, 4.9 / 4.9, 5.9 / 5.6, 7.8 / 6.6, of
    // 2048 at 48 and 192 3.9 / 4.1, 5.9 / 5.4; 8 of 4096 at 32, 64 and 96 6.6 / 8.1, 7.9 / 8.9, 9.8
    // / 9.5, of 7168 at 96 and 128 14.6 / 15.3, 17.7 / 16.1
    launch_post_norm_at<S, F, GATE, 256, 1, true>(p, T, HQ, eps, st);
  else if (HQ <= 1024)
    launch_post_norm_at<S, F, GATE, 512, 2, false>(p, T, HQ, eps, st);
  else
    launch_post_norm_at<S, F, GATE, 1024, 2, false>(p, T, HQ, eps, st);
}
template <int S, int F>
void launch_post_norm_f(const PostNorm& p, int T, int HQ, float eps, hipStream_t st) {
  if (!p.gate)
    launch_post_norm_g<S, F, kNoGate>(p, T, HQ, eps, st);
  else if (p.gate_kind == kF32)
    launch_post_norm_g<S, F, kGateF32>(p, T, HQ, eps, st);
  else
    launch_post_norm_g<S, F, kGateBF16>(p, T, HQ, eps, st);
}
}  // namespace

hipError_t launch_post_norm(const PostNorm& call, int T, int S, int H, float eps,
                            hipStream_t st) {
  // Stores that do not stay in the cache where the state read and the state written do not
  // both fit it: 4096 tokens of 4 x 4096 110 -> 99 us, 1024 of 8 x 7168 100 -> 96.
  PostNorm p = call;
  p.stream = (size_t)T * S * H * 8 > kCacheBytes;
  switch (S) {
#define MHC_S(SS)                                                  \
  case SS:                                                         \
    p.f_kind == kF32 ? launch_post_norm_f<SS, kF32>(p, T, H / 4, eps, st)  \
                     : launch_post_norm_f<SS, kBF16>(p, T, H / 4, eps, st); \
    break;
    MHC_S(1) MHC_S(2) MHC_S(3) MHC_S(4) MHC_S(5) MHC_S(6) MHC_S(7) MHC_S(8)
#undef MHC_S
    default:
      return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace mhc
