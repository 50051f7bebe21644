// mhc_pre_bwd.hip -- the gradient of the pre chain (include/mhc.h,
// mhc_site_pre_bwd), recomputed from the site's input x, which is fp32 or an
// 8-bit checkpoint.  Per token, with n = S*H:
//   raw = W x, ss = |x|^2, r = 1/sqrt(ss/n + eps), m = r raw, z = scale m + base
//   dpre_c  = (given) + sum_i dy_i x_c,i
//   dz      = dpre p(1-p), dpost 2 q(1-q) with post = 2 q, and exp(z) times the gradient that
//             the Sinkhorn rounds hand back: a pass c' = c/s, s = sum c + eps,
//             has dc = (dc' - sum dc' c') / s over the same row or column
//   u_r     = r scale dz_r,   alpha = -(sum_r scale dz_r m_r) r^2 / n
//   dx_c    = dx_in_c + pre_c dy + sum_r u_r W_r,c + alpha x_c
//   dW      = sum_t u_t x_t^T,  dbase = sum_t dz,  dscale_g = sum_t sum_g dz m
// Three to five launches: W split into bf16 planes (a group of few tokens does it on
// the way); the dots (raw, ss, dy.x) split over the hidden axis; the gates forward
// and backward, a block per four tokens (one where S > 4); the stream that writes
// dx and adds up dW, a wave owning 64 or 128 columns over a range of tokens; and the
// sums over the ranges and tokens (of a single range: in the stream's launch).  x
// and dy are read twice (neither fits on chip while a token's dots are open);
// everything else once.
// At 4096 tokens of 4 x 4096 from a checkpoint: 5 + 42 + 9 + 134 + 5 us, in fp32
// 5 + 70 + 9 + 165 + 5; at 1024 tokens of 8 x 7168: 11 + 60 + 11 + 175.
#include <type_traits>

#include "mhc_f8.h"
#include "mhc_kernels.h"
#include "mhc_waits.h"

namespace mhc {

namespace {

// an offset past every buffer of fewer than 2^31 - 16 bytes (a buffer of 2^31 has no
// columns to leave out), no lane's or row's part of 2^31 takes it round to zero
constexpr unsigned kOutside = 0x7ffffff0;
constexpr int kNonTemporal = 2;       // the cache policy bits of a buffer access
constexpr int kMaxChunk = 1024;       // tokens of a range of the stream (their gates in LDS)

__host__ __device__ constexpr int padded(int T) { return (T + 31) / 32 * 32; }
constexpr int rows_of(int S) { return (2 + S) * S; }
constexpr int steps_of(int S) { return (rows_of(S) + 15) / 16; }  // of 16 rows
constexpr int tiles_of(int S) { return (rows_of(S) + 31) / 32; }  // of 32 rows

typedef unsigned uintx4 __attribute__((ext_vector_type(4)));

// Q neighbouring floats of a buffer.
template <int Q>
using Columns = float __attribute__((ext_vector_type(Q)));
template <int Q, int POLICY>
__device__ __forceinline__ Columns<Q> load_columns(__amdgpu_buffer_rsrc_t buf, unsigned offset) {
  if constexpr (Q == 4)
    return __builtin_bit_cast(Columns<4>,
                              __builtin_amdgcn_raw_buffer_load_b128(buf, offset, 0, POLICY));
  else
    return __builtin_bit_cast(Columns<2>,
                              __builtin_amdgcn_raw_buffer_load_b64(buf, offset, 0, POLICY));
}
template <int Q>
__device__ __forceinline__ void store_columns(__amdgpu_buffer_rsrc_t buf, unsigned offset,
                                              Columns<Q> v) {
  if constexpr (Q == 4)
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(uintx4, v), buf, offset, 0,
                                           kNonTemporal);
  else
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(uintx2, v), buf, offset, 0,
                                          kNonTemporal);
}
}  // namespace

// ---------------------------------------------------------------- weight planes
// The two upper halves of two floats, as one dword.
__device__ __forceinline__ unsigned upper_halves(float lo, float hi) {
  return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}
__device__ __forceinline__ unsigned bf16_halves(float lo, float hi) {  // rounded to nearest
  return __builtin_bit_cast(unsigned, __builtin_convertvector(floatx2{lo, hi}, bf16x2));
}
// Two fp32 values as three bf16 each, high to low, one dword a plane: v = p0 + p1 + p2
// exactly, p0 being v rounded to eight bits, p1 the rest rounded to eight bits and p2
// what is left (seven bits and less).  |p1| <= 2^-8 and |p2| <= 2^-17 for v in [1, 2),
// either sign: of a product of two such values the planes' p1 p2, p2 p1 and p2 p2, left
// out below, are at most 2^-24 (1 + 2^-9) of it, and their signs do not follow its own.
// Cut instead of rounded, the rests are twice as large and of v's sign: up to 2^-21, and
// the loss of a sum grows with its length.  The conversion rounds two values in one
// instruction, so this costs what cutting does, but for p0, which is kept finite (an
// entry above the largest bf16 would round to an infinity): in fp32 37 tokens of 3 x 1028
// 24.2 us a call and 23.8, 1024 of 8 x 7168 307 and 305, 4096 of 4 x 4096 254 both.
__device__ __forceinline__ void planes2(float a, float b, unsigned out[3]) {
  constexpr float kMax = 0x1.fep127f;  // the largest bf16
  out[0] = bf16_halves(__builtin_amdgcn_fmed3f(a, -kMax, kMax),
                       __builtin_amdgcn_fmed3f(b, -kMax, kMax));
#pragma unroll
  for (int k = 1; k < 3; ++k) {
    a -= __uint_as_float(out[k - 1] << 16);
    b -= __uint_as_float(out[k - 1] & 0xffff0000u);
    out[k] = bf16_halves(a, b);
  }
}
// Eight fp32 values to their planes, one matrix operand each.
__device__ __forceinline__ void planes8(float4 a, float4 b, bf16x8 out[3]) {
  const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  union {
    unsigned u[4];
    bf16x8 v;
  } o[3];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    unsigned p[3];
    planes2(v[2 * i], v[2 * i + 1], p);
#pragma unroll
    for (int k = 0; k < 3; ++k) o[k].u[i] = p[k];
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) out[k] = o[k].v;
}

// W [R][S*H] as row operands of the dots of many tokens: for stream c, slice of 64
// columns, step of 32, plane and row tile of 16, 64 lanes of eight bf16 (row = lane % 16,
// columns 16g + 8 step on, g = lane / 16), zeros past R and H.
__global__ __launch_bounds__(256) void pre_bwd_planes_kernel(const float* __restrict__ w, int R,
                                                             int NRT, int S, int H, int HS,
                                                             long total,
                                                             bf16x8* __restrict__ out) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  const int lane = (int)(i & 63);
  const long f = i >> 6;
  const int rt = (int)(f % NRT);
  const long part = f / NRT;  // (c * HS + slice) * 2 + step
  const int step = (int)(part & 1), cs = (int)(part >> 1), c = cs / HS, slice = cs - c * HS;
  const int row = 16 * rt + (lane & 15);
  float4 v[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int col = 64 * slice + 16 * (lane >> 4) + 8 * step + 4 * q;
    v[q] = row < R && col < H
               ? *reinterpret_cast<const float4*>(w + ((size_t)row * S + c) * H + col)
               : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  bf16x8 o[3];
  planes8(v[0], v[1], o);
#pragma unroll
  for (int k = 0; k < 3; ++k) out[((part * 3 + k) * NRT + rt) * 64 + lane] = o[k];
}

// Exchange of the four lane groups with the four registers: register i of group g
// becomes register g of group i.
__device__ __forceinline__ void swap32(float& a, float& b) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}
__device__ __forceinline__ void swap16(float& a, float& b) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}
__device__ __forceinline__ void turn_groups(float& v0, float& v1, float& v2, float& v3) {
  swap32(v0, v2);
  swap32(v1, v3);
  swap16(v0, v1);
  swap16(v2, v3);
}

// ---------------------------------------------------------------- dots
// part[G][T][R + 1 + S]: the R dots, the sum of squares, the S products with dy.
// A wave takes 16*TT tokens and `steps` slices of 64 hidden columns in all S
// streams; the four waves of a block take neighbouring ranges and are added up
// in LDS, the G blocks of a token group by the gates kernel.
// A slice goes in two steps of 32 columns; entry 4q (q = 0, 1) of lane group g = lane /
// 16 is column 16g + 8 step + 4q of codes (a lane's 16 bytes) and 32 step + 16q + 4g of
// fp32.  W, which a few tokens need only once, is split into planes on the way.
// The dots run on v_mfma_f32_16x16x32_bf16 with W in three planes.  A decoded
// code is exact in bf16, so three products give fp32 dots; an fp32 x is split into
// planes as well and takes six (planes2 says what the three left out are).
// Every load of x and dy gives the four lane groups 64 neighbouring bytes of a
// token; dy, four floats a lane, is then turned between the groups to meet the
// codes' order.  Bound by waits: a wave asks in turn for dy, x, the planes and the
// scales, which two waves a SIMD hardly hide (one token of 4 x 4096: 4.5 us).
// SPLIT: a block takes one stream, for batches too short to fill the chip otherwise.  In
// fp32 at S = 8 and TT = 2 the kernel without it spills 14 registers (80 bytes a lane): 64
// tokens of 8 x 16384 166 us a call, 164 with planes that are cut and spill none.
template <int S, bool F8, int TT, bool SPLIT>
__global__ __launch_bounds__(256, 2) void pre_bwd_dots_kernel(
    const void* __restrict__ x, const unsigned char* __restrict__ xs,
    const float* __restrict__ w, const float* __restrict__ dy, int T, int H, int KB, int G,
    int HS, int steps, float* __restrict__ part) {
  constexpr int R = rows_of(S), NRT = steps_of(S), V = R + 1 + S, VP = 16 * NRT + 1 + S;
  constexpr int UC = S <= 4 && !SPLIT ? S : 1;  // unrolled further, the streams' loads spill
  __shared__ float sums[4][16 * TT][VP];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int tb = blockIdx.x / G, gi = blockIdx.x - tb * G, HQ = H >> 2;
  const int range = SPLIT ? gi / S : gi;
  const int c0 = SPLIT ? gi - range * S : 0, c1 = SPLIT ? c0 + 1 : S;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  size_t t[TT];
#pragma unroll
  for (int k = 0; k < TT; ++k) t[k] = min((tb * TT + k) * 16 + r, T - 1);
  floatx4 acc[TT][NRT];
  float ss[TT], dp[TT][S];
#pragma unroll
  for (int k = 0; k < TT; ++k) {
    ss[k] = 0.f;
#pragma unroll
    for (int c = 0; c < S; ++c) dp[k][c] = 0.f;
#pragma unroll
    for (int i = 0; i < NRT; ++i) acc[k][i] = floatx4{0.f, 0.f, 0.f, 0.f};
  }
  const int s0 = (range * 4 + wave) * steps, s1 = min(s0 + steps, HS);
  for (int sl = s0; sl < s1; ++sl) {
    float4 d[TT][4];  // columns 4i .. of the lane's: 16g + 4i (codes) or 16i + 4g
#pragma unroll
    for (int k = 0; k < TT; ++k) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int q = 16 * sl + 4 * i + g;
        d[k][i] = q < HQ ? reinterpret_cast<const float4*>(dy)[t[k] * HQ + q] : zero;
      }
      if constexpr (F8) {
        turn_groups(d[k][0].x, d[k][1].x, d[k][2].x, d[k][3].x);
        turn_groups(d[k][0].y, d[k][1].y, d[k][2].y, d[k][3].y);
        turn_groups(d[k][0].z, d[k][1].z, d[k][2].z, d[k][3].z);
        turn_groups(d[k][0].w, d[k][1].w, d[k][2].w, d[k][3].w);
      }
    }
#pragma unroll UC
    for (int c = c0; c < c1; ++c) {
      float dc[TT];
      intx4 code[TT];
      float scale[TT];
#pragma unroll
      for (int k = 0; k < TT; ++k) {
        dc[k] = 0.f;
        if constexpr (F8) {
          const size_t row = t[k] * S + c;
          code[k] = static_cast<const intx4*>(x)[row * KB * 8 + 4 * sl + g];
          scale[k] = f8_scale(xs[row * KB + (sl >> 1)]);
        }
      }
#pragma unroll
      for (int step = 0; step < 2; ++step) {
        const int q0 = 16 * sl + (F8 ? 4 * g + 2 * step : 8 * step + g);
        const int q1 = q0 + (F8 ? 1 : 4);
        bf16x8 wv[NRT][3];
#pragma unroll
        for (int i = 0; i < NRT; ++i) {  // rows past R: the last one, which nobody reads
          const float4* p = reinterpret_cast<const float4*>(w) +
                            ((size_t)min(16 * i + r, R - 1) * S + c) * HQ;
          planes8(q0 < HQ ? p[q0] : zero, q1 < HQ ? p[q1] : zero, wv[i]);
        }
#pragma unroll
        for (int k = 0; k < TT; ++k) {
          float4 xa, xb;
          bf16x8 xp[3];
          if constexpr (F8) {
            xp[0] = f8_to_bf16(code[k][2 * step], code[k][2 * step + 1], scale[k]);
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
            const float4* p = static_cast<const float4*>(x) + (t[k] * S + c) * HQ;
            xa = q0 < HQ ? p[q0] : zero;
            xb = q1 < HQ ? p[q1] : zero;
            planes8(xa, xb, xp);
          }
          ss[k] = dot4(xb, xb, dot4(xa, xa, ss[k]));
          dc[k] = dot4(d[k][2 * step + 1], xb, dot4(d[k][2 * step], xa, dc[k]));
#pragma unroll
          for (int i = 0; i < NRT; ++i) {
#pragma unroll
            for (int p = 0; p < 3; ++p)
#pragma unroll
              for (int m = 0; m < (F8 ? 1 : 3 - p); ++m)
                acc[k][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[i][p], xp[m], acc[k][i],
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
    float* mine = sums[wave][16 * k + r];
#pragma unroll
    for (int i = 0; i < NRT; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) mine[16 * i + 4 * g + v] = acc[k][i][v];
    const float s = swap32_sum(swap16_sum(ss[k]));
    if (g == 0) mine[16 * NRT] = s;
#pragma unroll
    for (int c = 0; c < S; ++c) {
      const float v = swap32_sum(swap16_sum(dp[k][c]));
      if (g == 0) mine[16 * NRT + 1 + c] = v;
    }
  }
  __syncthreads();
  const int first = tb * 16 * TT;
  for (int i = threadIdx.x; i < 16 * TT * V; i += 256) {
    const int k = i / V, v = i - k * V, at = v < R ? v : v - R + 16 * NRT;
    if (first + k < T)
      part[((size_t)gi * T + first + k) * V + v] =
          (sums[0][k][at] + sums[1][k][at]) + (sums[2][k][at] + sums[3][k][at]);
  }
}

// The dots of more than 16 tokens (more than 64 with S > 4), staged: a block
// takes 16 tokens a wave and walks units of one stream of one slice.  x (codes and
// scales, or fp32) and planes come into LDS by direct loads, two units ahead in
// three stages in turn (fp32: one ahead, two stages), dy a slice ahead (what a wave
// waits for: mhc_waits.h): the planes
// are read once a block, and no wave waits for one kind of load after the other.  A
// unit is read into registers before the next loads are asked for, since the
// compiler lets no read pass a load whose place it cannot tell apart (eight streams in
// fp32 spill three registers on the way, 16 bytes a lane).  A token's
// chunks of 16 bytes are turned in their row (codes: chunk c at place
// c ^ token / 4 % 4 of four; fp32: c ^ token % 16 of sixteen), so that 16 tokens read
// at one chunk meet all banks.
// The kernel above (with planes made beforehand) and this one, us: 4 x 4096,
// checkpoint, 16 tokens 5.5 and 6.3, 24: 7.4 and 6.3, 4096: 62 and 42; fp32 16: 7.3 and
// 6.4, 24: 10.3 and 6.3, 4096: 162 and 70 (x and dy alone: 22 and 56).  8 x 4096, where
// a unit's planes are 30 KiB and eight waves share them: checkpoint 64 tokens 12.1 and
// 16.6, 96: 16.4 and 16.0, 2048: 78 and 61 (86 with four waves).
// DIRECT: one group of tokens, which needs W once: its fp32 rows are staged instead
// and each wave makes its operands from them.  37 tokens of 3 x 1028 in fp32: 6.6 us
// against 8.7 with the planes' launch, and 5 us less a call; 128 of 8 x 4096 from a
// checkpoint 29 and 24, a call the same.
constexpr int staged_waves(int S) { return S <= 4 ? 4 : 8; }

template <int S, bool F8, bool DIRECT>
__global__ __launch_bounds__(64 * staged_waves(S)) void pre_bwd_dots_staged_kernel(
    const unsigned char* __restrict__ x, const unsigned char* __restrict__ xs,
    const unsigned char* __restrict__ w, const unsigned char* __restrict__ dy, int T, int H,
    int KB, int G, int HS, int steps, float* __restrict__ part) {
  constexpr int R = rows_of(S), NRT = steps_of(S), V = R + 1 + S, W = staged_waves(S);
  constexpr int NS = F8 ? 3 : 2;             // stages
  constexpr int LX = F8 ? 2 : 4;             // a wave's loads of x and scales a unit
  constexpr int LW = ((DIRECT ? 4 : 6) * NRT + W - 1) / W;  // and of planes, or of W
  constexpr int XB = F8 ? 16 * 64 + 64 * 4 : 16 * 256;  // a wave's bytes of them
  constexpr int STAGE = W * (XB + LW * 1024);
  // One variable a stage, by which the compiler can tell a read from the loads under way
  // into the others.  With four and eight streams it does so for the second of three stages
  // only: before the reads of the others, and of dyl at every slice, it waits for all
  // loads, so that the prefetch is drained there.
  __shared__ __align__(16) unsigned char stage0[STAGE];
  __shared__ __align__(16) unsigned char stage1[STAGE];
  __shared__ __align__(16) unsigned char stage2[NS > 2 ? STAGE : 16];
  __shared__ float4 dyl[16 * W * 16];
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tb = blockIdx.x / G, gi = blockIdx.x - tb * G, HQ = H >> 2;
  const int first = (tb * W + wave) * 16, t = first + r;  // this wave's tokens, this lane's
  const int s0 = gi * steps, units = (min(s0 + steps, HS) - s0) * S, last = units - 1;
  auto stage_of = [&](int i) -> unsigned char* {
    return i == 0 ? stage0 : i == 1 ? stage1 : stage2;
  };
  // a load of slice sl of rows k .. k + 3 (of `count`, past the end the last one) of
  // `pitch` quads each, from quad q0 on; quads past the hidden size are its last one
  auto fetch_quads = [&](const unsigned char* p, int k, int count, size_t pitch, size_t q0, int sl,
                         unsigned char* to) {
    const int row = k + (lane >> 4), q = min(16 * sl + ((lane ^ row) & 15), HQ - 1);
    load_to_lds(p + ((size_t)min(row, count - 1) * pitch + q0 + q) * 16, to);
  };
  auto fetch_dy = [&](int sl) {
#pragma unroll
    for (int i = 0; i < kDyLoads; ++i)
      fetch_quads(dy, first + 4 * i, T, HQ, 0, sl,
                  reinterpret_cast<unsigned char*>(dyl + wave * 256 + i * 64));
  };
  const size_t crow = (size_t)min(first + (lane >> 2), T - 1) * S;
  const size_t srow = (size_t)min(t, T - 1) * S;
  const int chunk = (lane & 3) ^ ((lane >> 4) & 3);
  auto fetch = [&](int u, int to) {  // unit u into stage `to`: LX + LW loads
    const int sl = s0 + u / S, c = u % S;
    unsigned char* st = stage_of(to);
    unsigned char* sx = st + wave * XB;
    if constexpr (F8) {
      load_to_lds(x + ((crow + c) * KB * 8 + 4 * sl + chunk) * 16, sx);
      load_byte_to_lds(xs + (srow + c) * KB + (sl >> 1), sx + 16 * 64);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        fetch_quads(x, first + 4 * i, T, (size_t)S * HQ, (size_t)c * HQ, sl, sx + i * 1024);
    }
    const unsigned char* wu = w + ((size_t)(c * HS + sl) * 6 * NRT * 64 + lane) * 16;
#pragma unroll
    for (int i = 0; i < LW; ++i) {
      const int j = wave + W * i;
      unsigned char* to = st + W * XB + j * 1024;
      if constexpr (DIRECT)
        fetch_quads(w, 4 * j, R, (size_t)S * HQ, (size_t)c * HQ, sl, to);
      else
        load_to_lds(wu + j * 1024, to);
    }
  };
  floatx4 acc[NRT];
  float ss = 0.f, dp[S];
  float4 d[4];
#pragma unroll
  for (int i = 0; i < S; ++i) dp[i] = 0.f;
#pragma unroll
  for (int i = 0; i < NRT; ++i) acc[i] = floatx4{0.f, 0.f, 0.f, 0.f};
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  fetch_dy(s0);
  fetch(0, 0);
  if constexpr (NS > 2) fetch(min(1, last), 1);
  int c = 0;
  for (int u0 = 0; u0 < units; u0 += NS) {
#pragma unroll
    for (int here = 0; here < NS; ++here) {
      const int u = u0 + here, sl = s0 + u / S;
      // this unit's stage has landed, and dy where it begins a slice; of three stages the
      // next unit's loads may be on their way
      if constexpr (NS == 2)
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      else if (c == 1)
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(dots_in_flight(S, 1, LX + LW))
                     : "memory");
      else
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(dots_in_flight(S, 0, LX + LW))
                     : "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      if (c == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 v = dyl[(wave * 16 + r) * 16 + ((4 * g + i) ^ r)];
          d[i] = 16 * sl + 4 * g + i < HQ ? v : zero;
        }
      }
      const unsigned char* st = stage_of(here);
      const unsigned char* sx = st + wave * XB;
      intx4 code;
      float4 xq[4];
      float scale;
      if constexpr (F8) {
        code = *reinterpret_cast<const intx4*>(sx + r * 64 + (g ^ ((r >> 2) & 3)) * 16);
        scale = f8_scale(*reinterpret_cast<const unsigned*>(sx + 16 * 64 + lane * 4) & 255u);
        if (u > last) code = intx4{0, 0, 0, 0};
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 v = reinterpret_cast<const float4*>(sx)[r * 16 + ((4 * g + i) ^ r)];
          xq[i] = u <= last && 16 * sl + 4 * g + i < HQ ? v : zero;
        }
      }
      // planes 3 step + p, or columns 4 step + e of W
      constexpr int WQ = DIRECT ? 4 : 6;
      typedef typename std::conditional<DIRECT, float4, bf16x8>::type Part;
      Part wr[WQ][NRT];
#pragma unroll
      for (int p = 0; p < WQ; ++p)
#pragma unroll
        for (int i = 0; i < NRT; ++i)
          wr[p][i] = reinterpret_cast<const Part*>(st + W * XB)[
              DIRECT ? (16 * i + r) * 16 + ((4 * g + p) ^ r) : (p * NRT + i) * 64 + lane];
      __builtin_amdgcn_sched_barrier(0);
      if (c == 0) {
        // the wave's own rows, read just now, make room for the next slice's
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        fetch_dy(min(sl + 1, s0 + last / S));
      }
      // past the end the last unit again, so that the counts above hold to the end
      fetch(min(u + NS - 1, last), (here + NS - 1) % NS);
      __builtin_amdgcn_sched_barrier(0);
      float dc = 0.f;
#pragma unroll
      for (int step = 0; step < 2; ++step) {
        constexpr int XP = F8 ? 1 : 3;
        bf16x8 o[XP];
        float4 xa, xb;
        if constexpr (F8) {
          union {
            bf16x8 v;
            unsigned u[4];
          } e;
          e.v = f8_to_bf16(code[2 * step], code[2 * step + 1], scale);
          xa = make_float4(__uint_as_float(e.u[0] << 16), __uint_as_float(e.u[0] & 0xffff0000u),
                           __uint_as_float(e.u[1] << 16), __uint_as_float(e.u[1] & 0xffff0000u));
          xb = make_float4(__uint_as_float(e.u[2] << 16), __uint_as_float(e.u[2] & 0xffff0000u),
                           __uint_as_float(e.u[3] << 16), __uint_as_float(e.u[3] & 0xffff0000u));
          o[0] = e.v;
        } else {
          xa = xq[2 * step];
          xb = xq[2 * step + 1];
          planes8(xa, xb, o);
        }
        ss = dot4(xb, xb, dot4(xa, xa, ss));
        dc = dot4(d[2 * step + 1], xb, dot4(d[2 * step], xa, dc));
#pragma unroll
        for (int i = 0; i < NRT; ++i) {
          bf16x8 wv[3];
          if constexpr (DIRECT) {
            const int q = 16 * sl + 4 * g + 2 * step;
            planes8(q < HQ ? wr[2 * step][i] : zero, q + 1 < HQ ? wr[2 * step + 1][i] : zero, wv);
          } else {
#pragma unroll
            for (int p = 0; p < 3; ++p) wv[p] = wr[step * 3 + p][i];
          }
#pragma unroll
          for (int p = 0; p < 3; ++p)
#pragma unroll
            for (int m = 0; m < (F8 ? 1 : 3 - p); ++m)
              acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[p], o[m], acc[i], 0, 0, 0);
        }
      }
#pragma unroll
      for (int i = 0; i < S; ++i) dp[i] += i == c && u <= last ? dc : 0.f;
      c = c + 1 == S ? 0 : c + 1;
    }
  }
  // nothing may land in this block's memory once another block has it
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  float* mine = part + ((size_t)gi * T + min(t, T - 1)) * V;
#pragma unroll
  for (int i = 0; i < NRT; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int at = 16 * i + 4 * g + v;
      if (t < T && at < R) mine[at] = acc[i][v];
    }
  ss = swap32_sum(swap16_sum(ss));
  if (t < T && g == 0) mine[R] = ss;
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const float v = swap32_sum(swap16_sum(dp[i]));
    if (t < T && g == 0) mine[R + 1 + i] = v;
  }
}

// ---------------------------------------------------------------- gates
// p (1 - p) of p = sigmoid(z).  Above 1/2, 1 - p is the difference of two close numbers
// (at z = 12 it has lost 12 of its 24 bits, from 17 on all): there it is e^-z p.
__device__ __forceinline__ float sigmoid_slope(float z, float p) {
  return z > 0.0f ? expf(-z) * p * p : p * (1.0f - p);
}

// One wave per four tokens (one where S > 4): the gates from the dots, then back.
//   side [S + 1][TP]   the pre gates and alpha (TP: T rounded up to 32)
//   red [R + 3][T]     dz and, per scale, the sum of dz * m
//   ua, ut             u in planes as the stream's operands (below), zero past R
//                      and past T
// hist (LDS): the matrix before every pass, 64 entries each.  The way back needs
// from it the entries and the reciprocal sums, which do not depend on the
// gradient: they are fetched one round ahead, so that a pass of the dependent
// chain is a product, two lane exchanges, a difference and a product.
// Four waves: all add up the dots' ranges, wave 0 takes the rounds while wave 1 takes
// the other gates, and each writes the results of a token of its own.
template <int S>
__global__ __launch_bounds__(256) void pre_bwd_gates_kernel(
    const float* __restrict__ part, int G, int T, int n, const float* __restrict__ scale,
    const float* __restrict__ base, int iters, float eps, const float* __restrict__ dpre,
    const float* __restrict__ dpost, const float* __restrict__ dcomb,
    unsigned short* __restrict__ ua, unsigned short* __restrict__ ut, float* __restrict__ side,
    float* __restrict__ red) {
  constexpr int L = S <= 4 ? 4 : 8, NU = L == 4 ? 4 : 1;
  constexpr int R = rows_of(S), KS = steps_of(S), NRT = tiles_of(S), V = R + 1 + S;
  constexpr int IN = NU * V, PARTS = 256 / IN;
  __shared__ float sums[PARTS][IN], raw[NU][V], dzs[NU][R];
  extern __shared__ float hist[];
  const int lane = threadIdx.x & 63, t0 = blockIdx.x * NU;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const size_t TP = padded(T);
  if (threadIdx.x < PARTS * IN) {  // every PARTS-th range of one value
    const int q = threadIdx.x / IN, i = threadIdx.x - q * IN, k = i / V, v = i - k * V;
    const size_t step = (size_t)T * V;
    const float* p = part + (size_t)min(t0 + k, T - 1) * V + v;
    float s = 0.f;
    int gi = q;
    for (; gi + 7 * PARTS < G; gi += 8 * PARTS) {
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = p[(gi + e * PARTS) * step];
      s += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
    }
    for (; gi + PARTS < G; gi += 2 * PARTS) s += p[gi * step] + p[(gi + PARTS) * step];
    if (gi < G) s += p[gi * step];
    sums[q][i] = s;
  }
  __syncthreads();
  if (threadIdx.x < IN) {
    float s = sums[0][threadIdx.x];
#pragma unroll
    for (int q = 1; q < PARTS; ++q) s += sums[q][threadIdx.x];
    raw[threadIdx.x / V][threadIdx.x % V] = s;
  }
  __syncthreads();
  if (wave == 1) {
    const int k = L == 4 ? lane >> 3 : 0, gt = L == 4 ? lane & 7 : lane;
    const size_t t = t0 + k;
    if (k < NU && t < (size_t)T && gt < 2 * S) {
      const float rinv = rms_inverse(raw[k][R], n, eps), m = raw[k][gt] * rinv;
      const float z = fmaf(scale[gt < S ? 0 : 1], m, base[gt]), p = sigmoid_exact_ends(z);
      if (gt < S) {
        const float d = raw[k][R + 1 + gt] + (dpre ? dpre[t * S + gt] : 0.f);
        side[gt * TP + t] = p;
        dzs[k][gt] = d * sigmoid_slope(z, p);
      } else {
        dzs[k][gt] = dpost[t * S + gt - S] * 2.0f * sigmoid_slope(z, p);
      }
    }
  }
  if (wave == 0) {
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
    // c: after the round; mid, old: before its column and its row pass
    float mid = hist[(2 * iters - 1) * 64 + lane], old = hist[(2 * iters - 2) * 64 + lane];
    float rmid = __builtin_amdgcn_rcpf(col_sum<L>(mid) + pad);
    float rold = __builtin_amdgcn_rcpf(row_sum<L>(old) + pad);
    for (int it = iters - 1; it >= 0; --it) {
      const int before = it > 0 ? it - 1 : 0;
      const float mid2 = hist[(2 * before + 1) * 64 + lane], old2 = hist[(2 * before) * 64 + lane];
      d = (d - col_sum<L>(d * c)) * rmid;
      d = valid ? d : 0.f;
      d = (d - row_sum<L>(d * mid)) * rold;
      d = valid ? d : 0.f;
      c = old;
      mid = mid2;
      old = old2;
      rmid = __builtin_amdgcn_rcpf(col_sum<L>(mid) + pad);
      rold = __builtin_amdgcn_rcpf(row_sum<L>(old) + pad);
    }
    if (valid) dzs[tu][r] = d * c;
  }
  __syncthreads();
  for (int k = wave; k < NU; k += 4) {
    const size_t t = t0 + k;
    const bool live = t < (size_t)T;
    const float rinv = rms_inverse(raw[k][R], n, eps);
    float gm[3] = {0.f, 0.f, 0.f};
    // token t as row i of ua's steps and as entry (h, e) of ut's step s
    const int i = (int)(t & 31), s = i >> 4, h = (i >> 2) & 1, e = ((i >> 3) & 1) * 4 + (i & 3);
    for (int r = lane; r < 32 * NRT; r += 64) {
      float uv = 0.f;
      if (live && r < R) {
        const int grp = r < S ? 0 : r < 2 * S ? 1 : 2;
        const float dz = dzs[k][r], p = dz * (raw[k][r] * rinv);
        gm[0] += grp == 0 ? p : 0.f;
        gm[1] += grp == 1 ? p : 0.f;
        gm[2] += grp == 2 ? p : 0.f;
        uv = scale[grp] * dz * rinv;
        red[(size_t)r * T + t] = dz;
      }
      unsigned p[3];
      planes2(uv, uv, p);
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        const unsigned short v = (unsigned short)p[q];
        if (r < 16 * KS)
          ua[((((t >> 5) * KS + (r >> 4)) * 3 + q) * 64 + i + 32 * ((r >> 3) & 1)) * 8 +
             (r & 7)] = v;
        ut[(((((t >> 5) * NRT + (r >> 5)) * 2 + s) * 3 + q) * 64 + (r & 31) + 32 * h) * 8 + e] = v;
      }
    }
    float dot = 0.f;
    for (int q = 0; q < 3; ++q) {
      gm[q] = sum_wave(gm[q]);
      dot = fmaf(scale[q], gm[q], dot);
    }
    if (lane == 0 && live) {
      side[S * TP + t] = -dot * rinv * rinv / (float)n;
      for (int q = 0; q < 3; ++q) red[(size_t)(R + q) * T + t] = gm[q];
    }
  }
}

// ---------------------------------------------------------------- stream
// dx and dW in one pass over dx_in, dy and x, both on v_mfma_f32_32x32x16_bf16.  A
// wave owns 32 groups of Q neighbouring columns, one group a lane, and walks a
// range of tokens 32 at a time; lane half h holds the tokens 8a + 4h + b (a, b < 4)
// of a step.  Product q takes the q-th column of every group, so that each lane
// moves Q neighbouring floats of 16 tokens and the results land where they are
// stored from:
//   dx: D[token][column] += u W over the rows, both in planes (six products, as in the
//       dots), started from dx_in + pre dy + alpha x
//   dW: D[row][column] += u^T x over the tokens, x exact in bf16 (fp32: in planes)
// The weight's planes are the lanes' own columns: each wave makes them once, in
// LDS.  u comes in operand order from the gates kernel:
//   ua [group of 32 tokens][step of 16 rows][plane][lane][8]: row i = lane % 32,
//      k = 8h + e for row 16 step + k of W
//   ut [group][tile of 32 rows][step of 16 tokens][plane][lane][8]: row lane % 32,
//      k = (h, e) for token 8 (2 step + e / 4) + 4h + e % 4
// The next step's loads start as soon as this one's have gone into the sums, and
// run under the products.
template <int S, bool F8, int Q>
__global__ __launch_bounds__(256, 1) void pre_bwd_stream_kernel(
    const void* __restrict__ x, const unsigned char* __restrict__ xs,
    const float* __restrict__ w, const float* __restrict__ dy, const bf16x8* __restrict__ ua,
    const bf16x8* __restrict__ ut, const float* __restrict__ side, const float* dx_in, int T,
    int H, int KB, int SB, int chunk, float* dx, float* __restrict__ dw_part,
    const float* __restrict__ red, float* __restrict__ dscale, float* __restrict__ dbase) {
  constexpr int R = rows_of(S), KS = steps_of(S), NRT = tiles_of(S);
  using Row = Columns<Q>;
  __shared__ bf16x8 wl[4][KS * 3 * Q][64];
  __shared__ float4 gate[S + 1][kMaxChunk / 4];  // side, for the block's tokens
  const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ci = blockIdx.x / SB, n = S * H;
  if (blockIdx.x >= SB && chunk >= T) {  // past a single range: red [R + 3][T] over the tokens
    const int row = (blockIdx.x - SB) * 4 + wave;
    if (row >= R + 3) return;
    float s = 0.f;
    for (int t = lane; t < T; t += 64) s += red[(size_t)row * T + t];
    s = sum_wave(s);
    if (lane == 0) *(row < R ? dbase + row : dscale + row - R) = s;
    return;
  }
  const int t_begin = ci * chunk, t_end = min(t_begin + chunk, T);
  const size_t TP = padded(T);
  const int group = ((blockIdx.x - ci * SB) * 4 + wave) * 32 + r;
  const bool in = group * Q < n;
  const int col = in ? group * Q : 0, cs = col / H, hc = col - cs * H;
  {
    const float* wc = w + col;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      Row v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int row = 16 * ks + 8 * h + e;
        v[e] = row < R ? *reinterpret_cast<const Row*>(wc + (size_t)row * n) : Row(0.f);
      }
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        bf16x8 o[3];
        planes8(make_float4(v[0][q], v[1][q], v[2][q], v[3][q]),
                make_float4(v[4][q], v[5][q], v[6][q], v[7][q]), o);
#pragma unroll
        for (int p = 0; p < 3; ++p) wl[wave][(ks * 3 + p) * Q + q][lane] = o[p];
      }
    }
  }
  floatx16 dw[NRT][Q];
#pragma unroll
  for (int i = 0; i < NRT; ++i)
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int v = 0; v < 16; ++v) dw[i][q][v] = 0.f;

  // what a step reads, token 8a + 4h + b at index 4a + b
  unsigned code[16], byte[16];
  Row xf[16], d[16], o[16];
  // A step's rows are buffers of their own (at most 2^31 bytes: n <= 2^24), a lane's
  // place in them an offset; tokens past the end and columns past n are out of
  // range, where loads give zero and stores are dropped.
  const int row_x = F8 ? S * KB * 128 : 4 * n, row_s = S * KB;
  const unsigned lane_n = in ? 4 * (4 * h * n + col) : kOutside;
  const unsigned lane_h = in ? 4 * (4 * h * H + hc) : kOutside;
  const unsigned lane_x = F8 ? (in ? 4 * h * row_x + cs * KB * 128 + hc : kOutside) : lane_n;
  const unsigned lane_s = in ? 4 * h * row_s + cs * KB + (hc >> 7) : kOutside;
  auto rows = [&](const void* p, int t0, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(static_cast<const char*>(p)) + (size_t)t0 * bytes, (short)0,
        p && t0 < t_end ? (unsigned)min(t_end - t0, 32) * (unsigned)bytes : 0u, 0x00020000);
  };
  auto load = [&](int t0) {
    const auto bx = rows(x, t0, row_x), bs = rows(xs, t0, row_s), bd = rows(dy, t0, 4 * H),
               bo = rows(dx_in, t0, 4 * n);
    unsigned lx = lane_x, ls = lane_s, lh = lane_h, ln = lane_n;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int k = 8 * (i >> 2) + (i & 3);
      // opaque: the sixteen offsets would be kept in registers across the steps
      asm volatile("" : "+v"(lx), "+v"(ls), "+v"(lh), "+v"(ln));
      if constexpr (F8) {
        if constexpr (Q == 4)
          code[i] = __builtin_amdgcn_raw_buffer_load_b32(bx, lx + k * row_x, 0, 0);
        else
          code[i] = __builtin_amdgcn_raw_buffer_load_b16(bx, lx + k * row_x, 0, 0);
        byte[i] = __builtin_amdgcn_raw_buffer_load_b8(bs, ls + k * row_s, 0, 0);
      } else {
        xf[i] = load_columns<Q, 0>(bx, lx + k * row_x);
      }
      d[i] = load_columns<Q, 0>(bd, lh + k * 4 * H);
      o[i] = load_columns<Q, kNonTemporal>(bo, ln + k * 4 * n);
    }
  };
  load(t_begin);
  for (int i = threadIdx.x; i < (S + 1) * (kMaxChunk / 4); i += 256) {
    const int c = i / (kMaxChunk / 4), k = i - c * (kMaxChunk / 4);
    if (4 * k < chunk && (size_t)t_begin + 4 * k < TP)
      gate[c][k] = *reinterpret_cast<const float4*>(side + c * TP + t_begin + 4 * k);
  }
  __syncthreads();
  for (int t0 = t_begin; t0 < t_end; t0 += 32) {
    float4 pg[4], al[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      pg[a] = gate[cs][(t0 - t_begin) / 4 + 2 * a + h];
      al[a] = gate[S][(t0 - t_begin) / 4 + 2 * a + h];
    }
    floatx16 acc[Q];
    constexpr int XP = F8 ? 1 : 3;
    union Operand {
      unsigned u[4];
      bf16x8 v;
    } xo[2][Q][XP];  // x as the operand of dW's two steps
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      float p[2], a[2];
      const float *pf = reinterpret_cast<const float*>(&pg[i >> 2]),
                  *af = reinterpret_cast<const float*>(&al[i >> 2]);
      float v[2][Q];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        p[k] = pf[(i + k) & 3];
        a[k] = af[(i + k) & 3];
        if constexpr (F8) {
          const float sc = f8_scale(byte[i + k]);
#pragma unroll
          for (int q = 0; q < Q; q += 2) {
            const bf16x2 two =
                q == 0 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)code[i + k], sc, false)
                       : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)code[i + k], sc, true);
            const unsigned b = __builtin_bit_cast(unsigned, two);
            v[k][q] = __uint_as_float(b << 16);
            v[k][q + 1] = __uint_as_float(b & 0xffff0000u);
          }
        } else {
#pragma unroll
          for (int q = 0; q < Q; ++q) v[k][q] = xf[i + k][q];
        }
      }
#pragma unroll
      for (int q = 0; q < Q; ++q) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
          acc[q][i + k] = fmaf(a[k], v[k][q], fmaf(p[k], d[i + k][q], o[i + k][q]));
        unsigned pl[3];
        if constexpr (F8)
          pl[0] = upper_halves(v[0][q], v[1][q]);
        else
          planes2(v[0][q], v[1][q], pl);
#pragma unroll
        for (int m = 0; m < XP; ++m) xo[i >> 3][q][m].u[(i & 7) >> 1] = pl[m];
      }
    }
    // u first: loads come back in order, and what is asked for after the next step's
    // rows would have to wait for them
    const size_t tg = t0 >> 5;
    bf16x8 um[NRT][2][3], uk[KS][3];
#pragma unroll
    for (int i = 0; i < NRT; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int p = 0; p < 3; ++p)
          um[i][s][p] = ut[(((tg * NRT + i) * 2 + s) * 3 + p) * 64 + lane];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int p = 0; p < 3; ++p) uk[ks][p] = ua[((tg * KS + ks) * 3 + p) * 64 + lane];
    __builtin_amdgcn_sched_barrier(0);
    load(t0 + 32);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < NRT; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
          for (int m = 0; m < (F8 ? 1 : 3 - p); ++m)
#pragma unroll
            for (int q = 0; q < Q; ++q)
              dw[i][q] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(um[i][s][p], xo[s][q][m].v,
                                                                 dw[i][q], 0, 0, 0);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int m = 0; m < 3; ++m) {
        bf16x8 wq[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) wq[q] = wl[wave][(ks * 3 + m) * Q + q][lane];
#pragma unroll
        for (int p = 0; p < 3 - m; ++p)
#pragma unroll
          for (int q = 0; q < Q; ++q)
            acc[q] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(uk[ks][p], wq[q], acc[q], 0, 0, 0);
      }
    const auto bo = rows(dx, t0, 4 * n);
    unsigned ln = lane_n;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int k = 8 * (i >> 2) + (i & 3);
      asm volatile("" : "+v"(ln));
      Row v;
#pragma unroll
      for (int q = 0; q < Q; ++q) v[q] = acc[q][i];
      store_columns<Q>(bo, ln + k * 4 * n, v);
    }
  }
  if (!in) return;
  float* part = dw_part + (size_t)ci * R * n + col;
#pragma unroll
  for (int k = 0; k < NRT; ++k)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int row = 32 * k + 8 * (i >> 2) + 4 * h + (i & 3);
      Row v;
#pragma unroll
      for (int q = 0; q < Q; ++q) v[q] = dw[k][q][i];
      if (row < R) *reinterpret_cast<Row*>(part + (size_t)row * n) = v;
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
    const float* p = red + (size_t)row * T;
    int t = threadIdx.x;
    for (; t + 7 * 256 < T; t += 8 * 256) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = p[t + k * 256];
      s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
    for (; t < T; t += 256) s += p[t];
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
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float4 v) { s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w); };
  int c = 0;
  for (; c + 4 <= chunks; c += 4) {
    float4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = p[(c + k) * quads];
#pragma unroll
    for (int k = 0; k < 4; ++k) add(v[k]);
  }
  for (; c < chunks; ++c) add(p[c * quads]);
  reinterpret_cast<float4*>(dw)[i] = s;
}

namespace {

// The split of a call's work: token groups of 16*TT tokens (staged: 16 a wave) times
// G ranges of the hidden axis for the dots (`steps` slices for each of 4 waves;
// staged: for the block), `chunks` token ranges of `chunk` for the stream; about
// 2048 and 1024 waves (8 and 4 per compute unit) where the shape has that many.
struct Plan {
  int TT, G, HS, steps, Q, SB, chunk, chunks;
  bool split, staged, direct;
  size_t planes, part, ua, ut, side, red, dw, floats;  // offsets and total, in floats
};
size_t round64(size_t v) { return (v + 63) / 64 * 64; }
int div_up(int a, int b) { return (a + b - 1) / b; }

Plan plan(int T, int S, int H, bool f8) {
  Plan p;
  const int R = rows_of(S);
  p.staged = T > (S <= 4 ? 16 : 64);
  p.TT = T <= 16 ? 1 : 2;
  const int groups = p.staged ? div_up(T, 16 * staged_waves(S)) : div_up(T, 16 * p.TT);
  const int waves = p.staged ? 1 : 4;  // of a block that divide its slices
  p.steps = div_up(p.HS = div_up(H, 64), waves * div_up(p.staged && S > 4 ? 256 : 512, groups));
  p.G = div_up(p.HS, waves * p.steps);
  p.direct = !p.staged || groups == 1;  // W split into planes by the dots themselves
  p.split = !p.staged && S > 1 && groups * p.G * S <= 512;
  if (p.split) p.G *= S;
  // The stream's split: of the counts of ranges that fill one to four rounds of the
  // compute units (a block each), the one with the fewest steps in a row, two more a
  // round for its beginning and end (3000 tokens of 4 x 7168: 336 blocks in three
  // ranges 240 us, 448 in four 205).  Four columns a lane instead of two, where a step
  // takes 1.85 times as long, from checkpoints of up to four streams (4096 tokens of
  // 4 x 4096: 146 and 135 us; fp32 170 and 165, but 2048 tokens 86 and 96).  Up to two
  // steps go in one range: with the sums beside it a launch less, and no slower (37
  // tokens of 3 x 1028: 11.0 us for both; 100: 11.3 in two, 17.0 in one).
  const int groups32 = padded(T) / 32, least = div_up(T, kMaxChunk);
  int c = 1;
  float best = 0.f;
  for (int Q = 2; Q <= (f8 && S <= 4 && T > 64 ? 4 : 2); Q += 2)
    for (int r = 1; r <= 4; ++r) {
      const int SB = div_up(S * H, 128 * Q), fill = 256 * r / SB;
      const int k = T <= 64 ? 1 : fill < least ? least : fill < groups32 ? fill : groups32;
      const float cost = (float)(((long)SB * k + 255) / 256) * (float)(div_up(groups32, k) + 2) *
                         (Q == 4 ? 1.85f : 1.f);
      if (best == 0.f || cost < best) best = cost, c = k, p.Q = Q, p.SB = SB;
    }
  p.chunk = div_up(groups32, c) * 32;
  p.chunks = div_up(T, p.chunk);
  size_t at = 0;
  p.planes = at;  // 64 lanes of 16 bytes for each step, plane and row tile
  // (the staged dots read a unit in multiples of 4 or 8 of them, past the last one)
  if (!p.direct) at += ((size_t)S * p.HS * 2 * 3 * div_up(R, 16) + 7) * 64 * 4;
  p.part = at;
  at += round64((size_t)p.G * T * (R + 1 + S));
  // three planes of two bytes, 32 tokens by 16 (32) rows a step (tile)
  p.ua = at;
  at += (size_t)groups32 * div_up(R, 16) * 3 * 64 * 4;
  p.ut = at;
  at += (size_t)groups32 * div_up(R, 32) * 2 * 3 * 64 * 4;
  p.side = at;
  at += round64((size_t)groups32 * 32 * (S + 1));
  p.red = at;
  at += round64((size_t)T * (R + 3));
  p.dw = at;
  if (p.chunks > 1) at += round64((size_t)p.chunks * R * S * H);
  p.floats = at;
  return p;
}

template <int S, bool F8, int TT, bool SPLIT>
void dots(const PreBwd& a, const Plan& p, int T, int H, int KB, float* work, hipStream_t st) {
  hipLaunchKernelGGL((pre_bwd_dots_kernel<S, F8, TT, SPLIT>),
                     dim3((unsigned)(div_up(T, 16 * TT) * p.G)), dim3(256), 0, st, a.x,
                     a.x_scales, a.fn_w, a.dy, T, H, KB, p.G, p.HS, p.steps, work + p.part);
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
  float *part = work + p.part, *side = work + p.side, *red = work + p.red;
  float* dw = p.chunks > 1 ? work + p.dw : a.dfn_w;
  auto staged = [&](auto kernel, const void* w) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(div_up(T, 16 * staged_waves(S)) * p.G)),
                       dim3(64 * staged_waves(S)), 0, st,
                       static_cast<const unsigned char*>(a.x), a.x_scales,
                       static_cast<const unsigned char*>(w),
                       reinterpret_cast<const unsigned char*>(a.dy), T, H, KB, p.G, p.HS, p.steps,
                       part);
  };
  constexpr bool MANY = S > 1;
  if (p.staged && p.direct) {
    staged(pre_bwd_dots_staged_kernel<S, F8, true>, a.fn_w);
  } else if (p.staged) {
    constexpr int NRT = steps_of(S);
    const long frags = (long)S * p.HS * 2 * NRT * 64;
    hipLaunchKernelGGL(pre_bwd_planes_kernel, dim3((unsigned)((frags + 255) / 256)), dim3(256), 0,
                       st, a.fn_w, R, NRT, S, H, p.HS, frags,
                       reinterpret_cast<bf16x8*>(work + p.planes));
    staged(pre_bwd_dots_staged_kernel<S, F8, false>, work + p.planes);
  } else if (p.TT == 2) {
    if constexpr (S > 4)  // staged with fewer
      p.split ? dots<S, F8, 2, MANY>(a, p, T, H, KB, work, st)
              : dots<S, F8, 2, false>(a, p, T, H, KB, work, st);
  } else {
    p.split ? dots<S, F8, 1, MANY>(a, p, T, H, KB, work, st)
            : dots<S, F8, 1, false>(a, p, T, H, KB, work, st);
  }
  hipLaunchKernelGGL((pre_bwd_gates_kernel<S>), dim3((unsigned)(padded(T) / NU)),
                     dim3(256), (size_t)iters * 2 * 64 * sizeof(float), st, part, p.G, T, n,
                     a.scale, a.base, iters, eps, a.dpre, a.dpost, a.dcomb,
                     reinterpret_cast<unsigned short*>(work + p.ua),
                     reinterpret_cast<unsigned short*>(work + p.ut), side, red);
  const bool one = p.chunks == 1;
  // beside a single range the sums over the tokens, a row a wave
  auto stream = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(p.SB * p.chunks + (one ? (R + 6) / 4 : 0))),
                       dim3(256), 0, st, a.x, a.x_scales, a.fn_w, a.dy,
                       reinterpret_cast<const bf16x8*>(work + p.ua),
                       reinterpret_cast<const bf16x8*>(work + p.ut), side, a.dx_in, T, H, KB, p.SB,
                       p.chunk, a.dx, dw, red, a.dscale, a.dbase);
  };
  if constexpr (F8 && S <= 4) {
    if (p.Q == 4)
      stream(pre_bwd_stream_kernel<S, F8, 4>);
    else
      stream(pre_bwd_stream_kernel<S, F8, 2>);
  } else {
    stream(pre_bwd_stream_kernel<S, F8, 2>);
  }
  if (one) return;
  const long quads = (long)R * n / 4;
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

// The gates kernel keeps 512 bytes of history a round in 64 KiB of LDS, and its sums.
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
