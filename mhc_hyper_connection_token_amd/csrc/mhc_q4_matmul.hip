// mhc_q4_matmul.hip -- out[m,n] = sum_k a[m,k] w[n,k] with 4-bit groups (mhc_q4.h):
//   out[m,n] = sum_g scale[n,g] * (sum_{k in g} a[m,k] code[n,k] - zero[n,g] sum_{k in g} a[m,k])
// so that the matrix instructions multiply the codes themselves, which are exact in any type,
// and a scale is applied once to a group's sum, in fp32.
// Three kernels by the number of rows M of a:
//   1        the vector ALU, lanes along the depth: nothing of the weight is staged;
//   2 .. 16  v_mfma_f32_16x16x32_bf16 (int8 activations: v_mfma_i32_16x16x32_i8, exact per
//            block of 32), the depth split over a block's waves;
//   more     tiles of v_mfma_f32_32x32x16_bf16.
// fp32 activations go into the matrix instructions as three bf16 planes that add up to the
// value.  Few rows are bound by reading the weight once; their floor is what a plain read of
// the same bytes takes, 3.5 us for 8.4 MB, 6.9 for 33.5, 16.5 for 100.
#include <algorithm>
#include <type_traits>

#include "mhc_kernels.h"
#include "mhc_q4.h"

namespace mhc {

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

struct Q4Args {
  const unsigned char* a;
  const float* ad;  // scales of int8 activations, [M][K/32]
  const unsigned char* codes;
  const unsigned short* scales;
  const unsigned char* zeros;
  void* out;
  int M, N, K, KG, f16, bf16_out;
};


__device__ __forceinline__ void octet_values(const Octet<kActBF16>& o, float* v) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = __uint_as_float((unsigned)o.v[e] << 16);
    v[2 * e + 1] = __uint_as_float((unsigned)o.v[e] & 0xffff0000u);
  }
}

// A product rounded by itself, also where it is subtracted from next.
__device__ __forceinline__ float mul_rounded(float a, float b) {
#pragma clang fp contract(off)
  return a * b;
}

__device__ __forceinline__ void store_one(const Q4Args& p, size_t at, float v) {
  if (p.bf16_out)
    static_cast<__hip_bfloat16*>(p.out)[at] = __float2bfloat16(v);
  else
    static_cast<float*>(p.out)[at] = v;
}

}  // namespace

// ---------------------------------------------------------------- one row
// A lane holds the activations of a block of 32 columns and meets the rows of the weight with
// them, the block's 16 bytes of each: R rows at a time, `iters` times, the next R on their
// way.  A wave's 64 lanes cover 2048 columns; the block's W waves are KS slices of the depth
// times W / KS runs of R * iters rows, whose sums meet in LDS.  us at 4096 x 4096, 16384 x 4096
// and 28672 x 7168 (int8; bf16; bf16): 4.2, 9.3, 24.4 (4.4 TB/s); fp32 9.3 at the second, 9.8
// with 64-column groups and zero points.  What is left
// above a plain read is the conversion and the products (2 instructions a weight) that the loads
// do not hide, and the first loads' latency.  R = 2, 4, 8: 9.8, 10.3, 12.3 at 16384 x 4096 in bf16,
// 8.5, 8.8, 8.9 in int8.
constexpr int kVectorRows = 64;  // rows of a wave at most

template <int A, int GS, bool ZEROS, int R, int W>
__global__ __launch_bounds__(64 * W) void q4_vector_kernel(Q4Args p, int KS, int iters) {
  __shared__ float part[W][kVectorRows];
  __shared__ floatx4 turn[A == kActF32 ? W : 1][A == kActF32 ? 64 * 9 : 1];  // (by slice)
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int KB = p.K / kQ4Block;
  const int slice = wave % KS, runs = W / KS, rows = R * iters;
  const int n0 = (blockIdx.x * runs + wave / KS) * rows;
  const size_t pitch = (size_t)KB * 16;
  for (int b0 = 0; b0 < KB; b0 += KS * 64) {
    const int k0 = b0 + slice * 64;
    if (A != kActF32 && k0 >= KB) break;
    // lanes past the end read the last block, times zeros
    const int k = min(k0 + lane, KB - 1);
    const bool in = k0 + lane < KB;
    const unsigned code_at = k * 16u, group = k >> GS;
    intx4 cn[R];
    // a row's scale and zero point as they were loaded: converted here, they would be waited for
    unsigned short sn[R];
    unsigned char zn[R];
    auto fetch = [&](int n) {  // rows past the end: the last one, whose sums are not stored
#pragma unroll
      for (int i = 0; i < R; ++i)
        cn[i] = __builtin_nontemporal_load(reinterpret_cast<const intx4*>(
            p.codes + (size_t)min(n + i, p.N - 1) * pitch + code_at));
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const size_t at = (size_t)min(n + i, p.N - 1) * p.KG + group;
        sn[i] = p.scales[at];
        if constexpr (ZEROS) zn[i] = p.zeros[at];
      }
    };
    // the activations first: loads are waited for in the order they were asked for in
    intx2 aq[4];
    float av[32], ad = 0.f, as = 0.f;
    int qs = 0;
    if constexpr (A == kActF32) {
      // The waves of a slice share its activations: each asks for a part of them, in whole
      // blocks, and all of them lie in LDS then.  us at 4096 x 4096, 7168 x 7168 and 16384 x 4096
      // so 5.1, 9.9 and 9.3; with a wave's own turned about in LDS 5.1, 10.6 and 9.9; with loads
      // of a lane's own 128 bytes, 64 lines each, 6.4, 11.0 and 10.8.
      const int run = wave / KS;
      if (b0 > 0) __syncthreads();
      floatx4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i * runs < 8)
          v[i] = reinterpret_cast<const floatx4*>(
              p.a)[min(k0 + 8 * (i * runs + run) + (lane >> 3), KB - 1) * 8 + (lane & 7)];
      if (k0 < KB) fetch(n0);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i * runs < 8) turn[slice][(8 * (i * runs + run) + (lane >> 3)) * 9 + (lane & 7)] = v[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const floatx4 u = turn[slice][lane * 9 + i];
#pragma unroll
        for (int e = 0; e < 4; ++e) av[4 * i + e] = in ? u[e] : 0.f;
      }
    } else {
      Octet<A> ao[4];
#pragma unroll
      for (int o = 0; o < 4; ++o)
        ao[o] = *reinterpret_cast<const Octet<A>*>(
            p.a + (unsigned)(k * kQ4Block + 8 * o) * (unsigned)act_size<A>());
      if constexpr (A == kActQ8) ad = p.ad[k];
      fetch(n0);
#pragma unroll
      for (int o = 0; o < 4; ++o) {
        if (!in) __builtin_memset(&ao[o], 0, sizeof(ao[o]));
        if constexpr (A == kActQ8) {
          aq[o] = ao[o].v;
          qs = __builtin_amdgcn_sdot4(aq[o][0], 0x01010101, qs, false);
          qs = __builtin_amdgcn_sdot4(aq[o][1], 0x01010101, qs, false);
        } else {
          octet_values(ao[o], av + 8 * o);
        }
      }
      if (A == kActQ8 && !in) ad = 0.f;
    }
    if constexpr (A != kActQ8) {
#pragma unroll
      for (int d = 0; d < 4; ++d) {  // in the products' order
        float u = av[4 * d];
#pragma unroll
        for (int e = 1; e < 8; ++e) u += av[16 * (e >> 2) + 4 * d + (e & 3)];
        as += u;
      }
    }
    if (k0 >= KB) continue;  // (this wave, but for the barriers)
    for (int it = 0; it < iters; ++it) {
      intx4 cv[R];
      float sv[R], zv[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        cv[i] = cn[i];
        sv[i] = q4_scale(sn[i], p.f16);
        zv[i] = ZEROS ? (float)zn[i] : 8.f;
      }
      if (it + 1 < iters) fetch(n0 + R * (it + 1));
      float acc[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if constexpr (A == kActQ8) {
          int v = -(int)zv[i] * qs;
#pragma unroll
          for (int d = 0; d < 4; ++d) {  // columns 4 d .. + 3 and 16 + 4 d .. + 3
            v = __builtin_amdgcn_sdot4(aq[d >> 1][d & 1], q4_low(cv[i][d]), v, false);
            v = __builtin_amdgcn_sdot4(aq[2 + (d >> 1)][d & 1], q4_high(cv[i][d]), v, false);
          }
          acc[i] = sv[i] * ((float)v * ad);
        } else {
          // Four chains, and the zero points last: one chain from minus zero point times sum on
          // has twice the error, 8e-7 of the result at 488 x 128, groups of 64.
          float u[4];
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const int lo = q4_low(cv[i][d]), hi = q4_high(cv[i][d]);
            const floatx2 c[4] = {q4_to_f32<false>(lo), q4_to_f32<true>(lo), q4_to_f32<false>(hi),
                                  q4_to_f32<true>(hi)};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float v = av[16 * (e >> 2) + 4 * d + (e & 3)];
              u[d] = e == 0 ? c[0][0] * v : fmaf(c[e >> 1][e & 1], v, u[d]);
            }
          }
          acc[i] = sv[i] * fmaf(-zv[i], as, (u[0] + u[1]) + (u[2] + u[3]));
        }
      }
#pragma unroll
      for (int i = 0; i < R; ++i) acc[i] = sum_wave(acc[i]);
      if (lane == 0)
#pragma unroll
        for (int i = 0; i < R; ++i) {
          float* to = &part[wave][R * it + i];
          *to = b0 == 0 ? acc[i] : *to + acc[i];
        }
    }
  }
  __syncthreads();
  // (a slice past the end of the depth has no sums)
  const int full = min(KS, (KB + 63) / 64);
  for (int i = threadIdx.x; i < runs * rows; i += 64 * W) {
    const int run = i / rows, row = i - run * rows, n = (blockIdx.x * runs + run) * rows + row;
    float v = part[run * KS][row];
    for (int k = 1; k < full; ++k) v += part[run * KS + k][row];
    if (n < p.N) store_one(p, n, v);
  }
}

// ---------------------------------------------------------------- up to 16 rows
// A block takes 16*NF columns n, the depth in stages of one superblock (128 columns) a
// wave; the waves' sums are added in order at the end.  A stage lies in LDS: the
// codes, the scales and zero points as floats, and the activations as the instructions take
// them (fp32 as its three planes).  It comes by way of registers, the weight from two stages
// ahead on, in whole lines (a wave's load is 1 KB of one row).  Sixteen rows read straight
// into the instructions' layout instead are sixteen lines a load, for the two bytes of a
// scale as well, and every wave loads the activations again.
// us at 2, 8 and 16 rows of 16384 x 4096: bf16 10.1, 11.6, 12.5; fp32 11.0, 15.4, 18.6; int8
// 10.2, 13.0, 14.0; with the activations read by every wave 16.6 at 8 rows in bf16.  What is
// left above the floor: two barriers a stage of 1024 columns, 700 clocks each.
// A row, of codes and of activations, is 16 bytes longer than it needs, so that sixteen rows
// read at one place meet all banks.
// Which four octets (mhc_q4.h) an instruction sums: of a superblock's sixteen, lane group g
// takes octet i of block g in instruction i where a group is the superblock, and octet 2 i + g %
// 2 of block 2 k + g / 2 in instruction i of group k where it is two blocks.  Where a group is one
// block, and with int8 activations, whose scales change by block, an instruction sums one block:
// lane group g takes its dword g, columns 4 g .. + 3 and 16 + 4 g .. + 3, and activations in
// fp32 and bf16 are put into LDS in that order.  (Octets of one block would be two dwords a lane
// and block: 8 x 7168 x 7168 in int8 16.1 us, so 12.7.)
// FEW (at most four rows): row r of the instruction is row r / 4 of a, and a lane ends with
// one sum, of row lane / 16.  With fp32 activations the rows 4 m, + 1, + 2 are the three
// planes of row m, so one instruction does what takes three from five rows on.
template <int A, int GS, bool FEW, int NF, int W>
struct RowsLayout {
  static constexpr int NG = 4 >> GS;                       // groups in a superblock
  static constexpr int CPITCH = 64 * W + 16;       // of a row of codes
  static constexpr int CODES = 16 * NF * CPITCH;  // bytes of a stage
  static constexpr int SCALES = 16 * NF * W * NG * 8;
  static constexpr int PITCH = 128 * W * (A == kActQ8 ? 1 : 2) + 16;  // of a row of a
  static constexpr int DPITCH = 4 * W + 4;        // floats, of a row of its scales
  static int bytes(int M) {
    return CODES + SCALES + M * (PITCH * (A == kActF32 ? 3 : 1) + (A == kActQ8 ? DPITCH * 4 : 0));
  }
};

template <int A, int GS, bool FEW, int NF, int W>
__global__ __launch_bounds__(64 * W) void q4_rows_kernel(Q4Args p) {
  using L = RowsLayout<A, GS, FEW, NF, W>;
  constexpr int NT = 64 * W, NG = L::NG;
  constexpr int GB = 1 << GS;                       // blocks of 32 a group
  constexpr int IG = A == kActQ8 ? 0 : GS;          // ... that an instruction's octets come from
  constexpr int MV = FEW ? 1 : 4;                   // sums a lane ends with, per tile
  constexpr int PL = A == kActF32 && !FEW ? 3 : 1;  // instructions a tile and block
  constexpr int UR = 4 * W, UA = 8 * W * act_size<A>();  // 16-byte units of a row, of codes and a
  constexpr int RA = FEW ? 4 : 16;
  constexpr int NS = (16 * NF * W * NG + NT - 1) / NT, NA = (RA * UA + NT - 1) / NT;
  static_assert(L::CODES >= NF * MV * W * 64 * 4, "the sums fit where the codes were");
  extern __shared__ __align__(16) unsigned char lds[];
  float2* const scales = reinterpret_cast<float2*>(lds + L::CODES);
  unsigned char* const acts = lds + L::CODES + L::SCALES;
  float* const dacts = reinterpret_cast<float*>(acts + p.M * L::PITCH);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16 * NF;
  const int KB = p.K / kQ4Block, SB = (p.K + 127) / 128;

  // Rows past the end read the last row; their results are not stored.
  intx4 cn[2][NF], an[NA];
  unsigned short sn[2][NS];
  unsigned char zn[2][NS];
  float dn = 0.f;
  // Where a thread's loads begin: 64-bit products cost too much to be formed a stage.  No
  // register that is loaded into gets a value of its own in between, which would wait for the
  // load: past the end of the depth the last columns are read, and zeros take their place in
  // LDS.
  const unsigned char *ap[NA], *bp[NF];
  size_t sp[NS];
#pragma unroll
  for (int i = 0; i < NA; ++i)
    ap[i] = p.a + (size_t)((threadIdx.x + NT * i) / UA) * p.K * act_size<A>();
#pragma unroll
  for (int i = 0; i < NF; ++i)
    bp[i] = p.codes + (size_t)min(n0 + (int)(NT * i + threadIdx.x) / UR, p.N - 1) * KB * 16;
#pragma unroll
  for (int i = 0; i < NS; ++i)
    sp[i] = (size_t)min(n0 + (int)(threadIdx.x + NT * i) / (W * NG), p.N - 1) * p.KG;
  auto fetch_a = [&](int sb) {
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int col = 128 * sb + (threadIdx.x + NT * i) % UA * (16 / act_size<A>());
      if ((NT * i + 64 * wave) / UA < p.M)  // (whole waves)
        an[i] = *reinterpret_cast<const intx4*>(
            ap[i] + (unsigned)(min(col, p.K - 16 / act_size<A>()) * act_size<A>()));
    }
    if constexpr (A == kActQ8)
      dn = p.ad[(size_t)min((int)threadIdx.x / (4 * W), p.M - 1) * KB +
                min(4 * sb + (int)threadIdx.x % (4 * W), KB - 1)];
  };
  auto fetch_w = [&](int sb, auto turn) {  // a block past the end: the last one, times zeros
    constexpr int T = decltype(turn)::value;
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      const unsigned at = min(4 * sb + (int)(threadIdx.x % UR), KB - 1) * 16u;
      cn[T][i] = __builtin_nontemporal_load(reinterpret_cast<const intx4*>(bp[i] + at));
    }
#pragma unroll
    for (int i = 0; i < NS; ++i)
      sn[T][i] = p.scales[sp[i] + (unsigned)min(sb * NG + (int)((threadIdx.x + NT * i) % (W * NG)),
                                                p.KG - 1)];
    if (p.zeros)
#pragma unroll
      for (int i = 0; i < NS; ++i)
        zn[T][i] = p.zeros[sp[i] + (unsigned)min(
                                       sb * NG + (int)((threadIdx.x + NT * i) % (W * NG)),
                                       p.KG - 1)];
  };
  auto place = [&](int sb, auto turn) {
    constexpr int T = decltype(turn)::value;
    if ((sb + W) * 128 > p.K) {  // the last stage, where it is short
#pragma unroll
      for (int i = 0; i < NA; ++i)
        if (128 * sb + (int)(threadIdx.x + NT * i) % UA * (16 / act_size<A>()) >= p.K)
          an[i] = intx4{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      const int row = (NT * i + threadIdx.x) / UR, unit = threadIdx.x % UR;
      reinterpret_cast<intx4*>(lds)[row * (L::CPITCH / 16) + unit] = cn[T][i];
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int id = threadIdx.x + NT * i, row = id / (W * NG), k = id % (W * NG);
      if (16 * NF * W * NG % NT == 0 || row < 16 * NF)
        scales[k * 16 * NF + row] =
            make_float2(q4_scale(sn[T][i], p.f16), p.zeros ? (float)zn[T][i] : 8.f);
    }
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int m = (NT * i + 64 * wave) / UA, c = (threadIdx.x + NT * i) % UA;
      if (m >= p.M) break;
      if constexpr (A == kActF32) {
        float v[4];
        __builtin_memcpy(v, &an[i], 16);
#pragma unroll
        for (int l = 0; l < 3; ++l) {  // the top eight significant bits, and what they leave
          unsigned u[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const unsigned lo = __float_as_uint(v[2 * h]), hi = __float_as_uint(v[2 * h + 1]);
            u[h] = __builtin_amdgcn_perm(hi, lo, 0x07060302);
            v[2 * h] -= __uint_as_float(lo & 0xffff0000u);
            v[2 * h + 1] -= __uint_as_float(hi & 0xffff0000u);
          }
          const int to = IG == 0 ? (c >> 3) * 64 + (c & 3) * 16 + (c >> 2 & 1) * 8 : 8 * c;
          __builtin_memcpy(
              __builtin_assume_aligned(acts + (3 * m + l) * L::PITCH + to, 8), u, 8);
        }
      } else if constexpr (A == kActBF16 && IG == 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // columns 8 c + 4 h .. + 3 of the row
          const int u[2] = {an[i][2 * h], an[i][2 * h + 1]};
          __builtin_memcpy(
              __builtin_assume_aligned(acts + m * L::PITCH + (c >> 2) * 64 + (c & 1) * 32 + h * 16 +
                                           (c >> 1 & 1) * 8, 8), u, 8);
        }
      } else {
        __builtin_memcpy(__builtin_assume_aligned(acts + m * L::PITCH + 16 * c, 16), &an[i], 16);
      }
    }
    if constexpr (A == kActQ8) {
      const int m = threadIdx.x / (4 * W);
      if (m < p.M) dacts[m * L::DPITCH + threadIdx.x % (4 * W)] = dn;
    }
  };

  const int am = min(FEW ? r >> 2 : r, p.M - 1);
  float acc[NF][MV];
#pragma unroll
  for (int j = 0; j < NF; ++j)
#pragma unroll
    for (int v = 0; v < MV; ++v) acc[j][v] = 0.f;

  auto multiply = [&] {
    intx4 cv[NF];
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      const unsigned char* at = lds + (16 * j + r) * L::CPITCH + 64 * wave;
      if constexpr (IG == 2) {
        cv[j] = reinterpret_cast<const intx4*>(at)[g];
      } else if constexpr (IG == 1) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const intx2 c = reinterpret_cast<const intx2*>(at)[4 * k + g];
          cv[j][2 * k] = c[0];
          cv[j][2 * k + 1] = c[1];
        }
      } else {
#pragma unroll
        for (int b = 0; b < 4; ++b) cv[j][b] = reinterpret_cast<const int*>(at)[4 * b + g];
      }
    }
    // the codes of the lane's octet in each instruction, four to a dword
    const auto codes = [&](int j, int b) -> intx2 {
      const intx4 v = cv[j];
      if constexpr (IG == 0) {
        return intx2{q4_low(v[b]), q4_high(v[b])};
      } else {
        const int p = IG == 2 ? b & 1 : b >> 1, high = IG == 2 ? b >> 1 : b & 1;
        return q4_octet(v[2 * p], v[2 * p + 1], high);
      }
    };
    float4 dv[MV];
    if constexpr (A == kActQ8)
#pragma unroll
      for (int v = 0; v < MV; ++v)
        dv[v] = *reinterpret_cast<const float4*>(
            dacts + min(FEW ? g : 4 * g + v, p.M - 1) * L::DPITCH + 4 * wave);
    floatx4 sum[NF], ones;
    float2 sz[NF];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (b % GB == 0) {
        ones = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          sum[j] = floatx4{0.f, 0.f, 0.f, 0.f};
          sz[j] = scales[(wave * NG + b / GB) * 16 * NF + 16 * j + r];
        }
      }
      if constexpr (A == kActQ8) {
        const int* at =
            reinterpret_cast<const int*>(acts + am * L::PITCH + 128 * wave + 32 * b) + g;
        const long ax = (long)(unsigned)at[0] | ((long)at[4] << 32);
        const intx4 none{0, 0, 0, 0};
        const intx4 q =
            __builtin_amdgcn_mfma_i32_16x16x32_i8(ax, 0x0101010101010101L, none, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          const intx2 c = codes(j, b);
          const long cx = (long)(unsigned)c[0] | ((long)c[1] << 32);
          const intx4 t = __builtin_amdgcn_mfma_i32_16x16x32_i8(ax, cx, none, 0, 0, 0);
          const int z = (int)sz[j].y;
#pragma unroll
          for (int v = 0; v < MV; ++v)
            sum[j][v] = fmaf((float)(t[v] - z * q[v]),
                             b == 0 ? dv[v].x : b == 1 ? dv[v].y : b == 2 ? dv[v].z : dv[v].w,
                             sum[j][v]);
        }
      } else {
        bf16x8 one, ax[PL];
#pragma unroll
        for (int v = 0; v < 8; ++v) one[v] = (__bf16)1.0f;
#pragma unroll
        for (int l = 0; l < PL; ++l) {
          const int row = A == kActBF16 ? am : FEW ? 3 * am + min(r & 3, 2) : 3 * am + l;
          const int octet = IG == 2   ? 4 * g + b
                            : IG == 1 ? 8 * (b >> 1) + 4 * (g >> 1) + 2 * (b & 1) + (g & 1)
                                      : 4 * b + g;
          __builtin_memcpy(&ax[l],
                           __builtin_assume_aligned(
                               acts + row * L::PITCH + 256 * wave + 16 * octet, 16), 16);
          ones = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ax[l], one, ones, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          const bf16x8 cx = q4_to_bf16(codes(j, b));
#pragma unroll
          for (int l = 0; l < PL; ++l)
            sum[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ax[l], cx, sum[j], 0, 0, 0);
        }
      }
      if (b % GB == GB - 1) {
        if (A == kActF32 && FEW) ones[0] += ones[1] + ones[2];
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          if (A == kActF32 && FEW) sum[j][0] += sum[j][1] + sum[j][2];
#pragma unroll
          for (int v = 0; v < MV; ++v) {
            const float t = A == kActQ8 ? sum[j][v] : fmaf(-sz[j].y, ones[v], sum[j][v]);
            acc[j][v] = fmaf(sz[j].x, t, acc[j][v]);
          }
        }
      }
    }
  };
  auto step = [&](int sb, auto turn) {
    place(sb, turn);
    __syncthreads();
    // asked for in the order of use, which is the order that loads are waited for in
    if (sb + W < SB) fetch_a(sb + W);
    if (sb + 2 * W < SB) fetch_w(sb + 2 * W, turn);
    if (sb + wave < SB) multiply();
    __syncthreads();
  };
  constexpr std::integral_constant<int, 0> even{};
  constexpr std::integral_constant<int, 1> odd{};
  fetch_w(0, even);
  fetch_a(0);
  if (W < SB) fetch_w(W, odd);
  for (int sb = 0; sb < SB; sb += 2 * W) {
    step(sb, even);
    if (sb + W < SB) step(sb + W, odd);
  }
  float* sums = reinterpret_cast<float*>(lds);  // no longer than the codes were
#pragma unroll
  for (int j = 0; j < NF; ++j)
#pragma unroll
    for (int v = 0; v < MV; ++v) sums[(wave * NF * MV + j * MV + v) * 64 + lane] = acc[j][v];
  __syncthreads();
  for (int i = threadIdx.x; i < NF * MV * 64; i += NT) {
    const int l = i & 63, f = i >> 6;
    float s = sums[i];
#pragma unroll
    for (int w = 1; w < W; ++w) s += sums[w * NF * MV * 64 + i];
    const int n = n0 + 16 * (f / MV) + (l & 15), m = FEW ? l >> 4 : 4 * (l >> 4) + f % MV;
    if (m < p.M && n < p.N) store_one(p, (size_t)m * p.N + n, s);
  }
}

// ---------------------------------------------------------------- tiles
// A block takes BM = 32*FM*WM rows of a and BN = 32*FN*WN columns n; WM x WN waves, each with
// FM x FN tiles of v_mfma_f32_32x32x16_bf16, times KG groups of such waves that take the
// superblocks (128 columns) of the depth in turn and are added in order at the end.  A stage
// (a superblock for each group of waves) is asked for while the one before is multiplied and
// goes by way of registers into LDS: into one of two buffers, one barrier a stage, or, where
// two do not fit, into the one that every wave has done with.
// In LDS: the codes; the activations as bf16 (fp32 ones and int8 codes times their scale as
// three planes), with the sums of each group of columns, which the zero points multiply; the
// scales and zero points as floats.  A group's products start from minus zero point times
// sum and end times the scale in the sums that are kept, in fp32.
// The 16-byte units of a row are placed so that sixteen rows read at one unit meet all banks.
// What bounds it: a stage of a 128 x 128 tile in bf16 takes 4000 clocks of its unit, of which
// the matrix instructions fill 1030, the vector ones (staging and sums 700, conversion to bf16
// and scaling the rest) 1680 and LDS 1240; two waves a SIMD leave a third of the time to waits.
// Its 85 KB of LDS keep it to one block a unit (150 registers would allow three waves), the 96 x
// 128 tile's 137 KB and 248 registers as well.  fp32 and int8 multiply three planes, whose
// tiles of more than 32 rows have one buffer only. Memory is not it: with two stages on their way
// instead of one 97 and 98 us at 333 x 7168 x 7168 (then with tiles of 32 x 128).
template <int A, int GS, int FM, int FN, int WM, int WN, int KG>
struct TileLayout {
  static constexpr int PL = A == kActBF16 ? 1 : 3, NG = 4 >> GS;
  static constexpr int BM = 32 * FM * WM, BN = 32 * FN * WN;
  static constexpr int CODES = BN * 64, ACTS = PL * BM * 256;  // bytes of a superblock
  static constexpr int SUMS = BM * NG * 4, SCALES = BN * NG * 8;
  static constexpr int PART = CODES + ACTS + SUMS + SCALES, STAGE = KG * PART;
  static constexpr int LAST = (KG - 1) * WM * WN * FM * FN * 4096;  // the groups' sums
  static constexpr int BUFS = 2 * STAGE <= 160 * 1024 ? 2 : 1;
  static constexpr int BYTES = BUFS * STAGE > LAST ? BUFS * STAGE : LAST;
};

// Sum over aligned groups of N neighbouring lanes, N up to 32, in every lane.
template <int N>
__device__ __forceinline__ float sum_lanes(float v) {
  if (N >= 2) v += dpp<0xB1>(v);
  if (N >= 4) v += dpp<0x4E>(v);
  if (N >= 8) v += dpp<0x141>(v);
  if (N >= 16) v += dpp<0x128>(v);
  return N >= 32 ? swap16_sum(v) : v;
}

template <int A, int GS, int FM, int FN, int WM, int WN, int KG>
__global__ __launch_bounds__(64 * WM * WN * KG) void q4_tile_kernel(Q4Args p, int MT, int NT) {
  using L = TileLayout<A, GS, FM, FN, WM, WN, KG>;
  constexpr int W = WM * WN * KG, TH = 64 * W, PL = L::PL, NG = L::NG, GB = 1 << GS;
  constexpr int BM = L::BM, BN = L::BN;
  constexpr int UA = 8 * act_size<A>();  // 16-byte units of a row of a, of a superblock
  constexpr int NA = KG * BM * UA / TH, NB = (KG * BN * 4 + TH - 1) / TH;
  constexpr int NS = (KG * BN * NG + TH - 1) / TH;
  static_assert(KG * BM * UA % TH == 0, "whole loads");
  extern __shared__ __align__(16) unsigned char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, h = lane >> 5;
  const int wm = wave % WM, wn = wave / WM % WN, kg = wave / (WM * WN);
  const int KB = p.K / kQ4Block, SB = (p.K + 127) / 128;

  // Blocks go to the eight dies in turn: give each die a run of tiles, rows first, so that
  // the tiles that read the same columns of the weight share its L2.
  const int tiles = MT * NT;
  int id = blockIdx.x;
  {
    const int per = tiles / 8, rest = tiles % 8, die = id % 8, at = id / 8;
    id = die * per + min(die, rest) + at;
  }
  const int m0 = id % MT * BM, n0 = id / MT * BN;

  intx4 an[NA], bn[NB];
  float dn[A == kActQ8 ? NA : 1];
  unsigned short sn[NS];
  unsigned char zn[NS];
  // Where a thread's loads begin (64-bit products cost too much to be formed a stage); rows past
  // the end read the last row, and are not stored.  As above, past the end of the depth the
  // last columns are read, and zeros take their place in LDS.
  const unsigned char *ap[NA], *bp[NB];
  size_t sp[NS];
#pragma unroll
  for (int i = 0; i < NA; ++i)
    ap[i] = p.a + (size_t)min(m0 + (int)(threadIdx.x + TH * i) / UA % BM, p.M - 1) * p.K *
                      act_size<A>();
#pragma unroll
  for (int i = 0; i < NB; ++i)
    bp[i] = p.codes + (size_t)min(n0 + (int)(threadIdx.x + TH * i) / 4 % BN, p.N - 1) * KB * 16;
#pragma unroll
  for (int i = 0; i < NS; ++i)
    sp[i] = (size_t)min(n0 + (int)(threadIdx.x + TH * i) / NG % BN, p.N - 1) * p.KG;
  auto fetch = [&](int sb) {
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int at = threadIdx.x + TH * i;
      const int col = 128 * (sb + at / UA / BM) + at % UA * (16 / act_size<A>());
      an[i] = *reinterpret_cast<const intx4*>(
          ap[i] + (unsigned)(min(col, p.K - 16 / act_size<A>()) * act_size<A>()));
      if constexpr (A == kActQ8)
        dn[i] = p.ad[(size_t)(ap[i] - p.a) / kQ4Block + min(col / kQ4Block, KB - 1)];
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int at = threadIdx.x + TH * i;
      const int k = min(4 * (sb + at / 4 / BN) + (at & 3), KB - 1);
      bn[i] = *reinterpret_cast<const intx4*>(bp[i] + (unsigned)(k * 16));
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int at = threadIdx.x + TH * i;
      const size_t g = sp[i] + (unsigned)min((sb + at / NG / BN) * NG + at % NG, p.KG - 1);
      sn[i] = p.scales[g];
      if (p.zeros) zn[i] = p.zeros[g];
    }
  };
  auto place = [&](unsigned char* to, int sb) {
    if ((sb + KG) * 128 > p.K) {  // the last stage, where it is short
#pragma unroll
      for (int i = 0; i < NA; ++i) {
        const int at = threadIdx.x + TH * i;
        if (128 * (sb + at / UA / BM) + at % UA * (16 / act_size<A>()) >= p.K)
          an[i] = intx4{0, 0, 0, 0};
      }
    }
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int at = threadIdx.x + TH * i, row = at / UA, c = at % UA, m = row % BM;
      unsigned char* part = to + row / BM * L::PART;
      unsigned char* acts = part + L::CODES;
      float total = 0.f;
      if constexpr (A == kActBF16) {
        reinterpret_cast<intx4*>(acts)[m * 16 + (c ^ (m & 15))] = an[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          bf16x2 v, one;
          const int u = an[i][e], ones = 0x3f803f80;
          __builtin_memcpy(&v, &u, 4);
          __builtin_memcpy(&one, &ones, 4);
          total = __builtin_amdgcn_fdot2_f32_bf16(v, one, total, false);
        }
      } else {
        constexpr int NV = A == kActF32 ? 4 : 16;  // columns of a unit
        float v[NV];
        if constexpr (A == kActF32) {
          __builtin_memcpy(v, &an[i], 16);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            v[e] = mul_rounded((float)((signed char)(an[i][e >> 2] >> (8 * (e & 3)))), dn[i]);
        }
#pragma unroll
        for (int e = 0; e < NV; ++e) total += v[e];
#pragma unroll
        for (int l = 0; l < 3; ++l) {  // the top eight significant bits, and what they leave
          unsigned u[NV / 2];
#pragma unroll
          for (int e = 0; e < NV / 2; ++e) {
            const unsigned lo = __float_as_uint(v[2 * e]), hi = __float_as_uint(v[2 * e + 1]);
            u[e] = __builtin_amdgcn_perm(hi, lo, 0x07060302);
            v[2 * e] -= __uint_as_float(lo & 0xffff0000u);
            v[2 * e + 1] -= __uint_as_float(hi & 0xffff0000u);
          }
          unsigned char* plane = acts + (l * BM + m) * 256;
          if constexpr (A == kActF32) {
            __builtin_memcpy(__builtin_assume_aligned(
                                 plane + ((c >> 1) ^ (m & 15)) * 16 + (c & 1) * 8, 8), u, 8);
          } else {
#pragma unroll
            for (int o = 0; o < 2; ++o)
              __builtin_memcpy(
                  __builtin_assume_aligned(plane + ((2 * c + o) ^ (m & 15)) * 16, 16), u + 4 * o,
                  16);
          }
        }
      }
      total = sum_lanes<UA / NG>(total);
      if (c % (UA / NG) == 0)
        reinterpret_cast<float*>(acts + L::ACTS)[c / (UA / NG) * BM + m] = -total;
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int at = threadIdx.x + TH * i, row = at / 4, n = row % BN;
      if (KG * BN * 4 % TH == 0 || row < KG * BN)
        reinterpret_cast<intx4*>(to + row / BN * L::PART)[n * 4 + ((at & 3) ^ ((n >> 2) & 3))] =
            bn[i];
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int at = threadIdx.x + TH * i, row = at / NG, k = at % NG;
      if (KG * BN * NG % TH == 0 || row < KG * BN)
        reinterpret_cast<float2*>(to + row / BN * L::PART + L::CODES + L::ACTS +
                                  L::SUMS)[k * BN + row % BN] =
            make_float2(q4_scale(sn[i], p.f16), p.zeros ? (float)zn[i] : 8.f);
    }
  };

  floatx16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  auto multiply = [&](const unsigned char* part) {
    const unsigned char* acts = part + L::CODES;
    const float* sums = reinterpret_cast<const float*>(acts + L::ACTS);
    const float2* scales = reinterpret_cast<const float2*>(acts + L::ACTS + L::SUMS);
    constexpr int ROLL = GS == 0 ? 1 : NG;
    // A lane half reads NO dwords, as many octets, at a time: whole blocks, every second one,
    // or, where a group is one block, half of it, octets h and 2 + h.
    constexpr int NO = GB > 1 ? 4 : 2, NU = 2 * GB / NO;
#pragma unroll ROLL
    for (int k = 0; k < NG; ++k) {
      float2 sz[FN];
      bf16x8 bx[FN][2 * GB];
      int c[FN][NU][NO];
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int n = (wn * FN + j) * 32 + r;
        sz[j] = scales[k * BN + n];
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          const int first = NO * (GB > 1 ? 2 * u + h : h);  // of the group's dwords
          __builtin_memcpy(
              c[j][u],
              __builtin_assume_aligned(
                  part + (n * 4 + ((k * GB + (first >> 2)) ^ ((n >> 2) & 3))) * 16 +
                      (first & 3) * 4, 4 * NO),
              4 * NO);
        }
      }
      // Left alone, the second read moves in among the products, which then wait for it: 500 x
      // 7168 x 7168 in bf16 96 us, so 90.
      if constexpr (NU > 1) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
          for (int i = 0; i < NO; ++i)
            bx[j][NO * u + i] =
                q4_to_bf16(q4_octet(c[j][u][2 * i % NO], c[j][u][2 * i % NO + 1], i / (NO / 2)));
      // the tiles take turns, so that no product waits for the one before it
      floatx16 t[FM][FN];
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const floatx4 c = *reinterpret_cast<const floatx4*>(
              sums + k * BM + (wm * FM + i) * 32 + 8 * v + 4 * h);
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) t[i][j][4 * v + e] = sz[j].y * c[e];
        }
#pragma unroll
      for (int l = 0; l < PL; ++l) {
        bf16x8 ax[FM][2 * GB];
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int b = 0; b < 2 * GB; ++b) {
            const int m = (wm * FM + i) * 32 + r;
            const int octet =
                GB > 1 ? 4 * (k * GB + 2 * (b / NO) + h) + b % NO : 4 * k + 2 * b + h;
            __builtin_memcpy(&ax[i][b],
                             __builtin_assume_aligned(
                                 acts + ((l * BM + m) * 16 + (octet ^ (m & 15))) * 16, 16), 16);
          }
#pragma unroll
        for (int b = 0; b < 2 * GB; ++b)
#pragma unroll
          for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
              t[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ax[i][b], bx[j][b], t[i][j], 0, 0,
                                                                 0);
      }
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[i][j][v] = fmaf(sz[j].x, t[i][j][v], acc[i][j][v]);
    }
  };

  fetch(0);
  int turn = 0;
  for (int sb = 0; sb < SB; sb += KG, turn ^= L::BUFS - 1) {
    unsigned char* stage = lds + turn * L::STAGE;
    if (L::BUFS == 1 && sb > 0) __syncthreads();
    place(stage, sb);
    __syncthreads();  // (of two buffers, the one written next was read before this)
    if (sb + KG < SB) fetch(sb + KG);
    // Waves that multiply go before waves that stage: 333 x 7168 x 7168 in int8 166 -> 150 us,
    // the other types and sizes up to 3 % (100 x 28672 x 7168 in bf16 94.4 -> 91.8).
    __builtin_amdgcn_s_setprio(1);
    if (KG == 1 || sb + kg < SB) multiply(stage + kg * L::PART);
    __builtin_amdgcn_s_setprio(0);
  }
  if constexpr (KG > 1) {
    float4* last = reinterpret_cast<float4*>(lds);
    __syncthreads();
    if (kg > 0) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            last[(((wave - WM * WN) * FM + i) * FN + j) * 256 + v * 64 + lane] =
                make_float4(acc[i][j][4 * v], acc[i][j][4 * v + 1], acc[i][j][4 * v + 2],
                            acc[i][j][4 * v + 3]);
    }
    __syncthreads();
    if (kg > 0) return;
#pragma unroll
    for (int k = 1; k < KG; ++k)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const float4 o =
                last[((((k - 1) * WM * WN + wave) * FM + i) * FN + j) * 256 + v * 64 + lane];
            acc[i][j][4 * v] += o.x;
            acc[i][j][4 * v + 1] += o.y;
            acc[i][j][4 * v + 2] += o.z;
            acc[i][j][4 * v + 3] += o.w;
          }
  }
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int n = n0 + (wn * FN + j) * 32 + r;
    if (n >= p.N) continue;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int m = m0 + (wm * FM + i) * 32 + 8 * (v >> 2) + 4 * h + (v & 3);
        if (m < p.M) store_one(p, (size_t)m * p.N + n, acc[i][j][v]);
      }
  }
}

namespace {
template <int A, int GS, int FM, int FN, int WM, int WN, int KG>
void launch_q4_tile(const Q4Args& p, hipStream_t st) {
  using L = TileLayout<A, GS, FM, FN, WM, WN, KG>;
  const int MT = (p.M + L::BM - 1) / L::BM, NT = (p.N + L::BN - 1) / L::BN, lds = L::BYTES;
  hipLaunchKernelGGL((q4_tile_kernel<A, GS, FM, FN, WM, WN, KG>), dim3((unsigned)(MT * NT)),
                     dim3(64 * WM * WN * KG), lds, st, p, MT, NT);
}
template <int A, int GS, bool FEW, int NF, int W>
void launch_q4_rows(const Q4Args& p, hipStream_t st) {
  const int lds = RowsLayout<A, GS, FEW, NF, W>::bytes(p.M);
  hipLaunchKernelGGL((q4_rows_kernel<A, GS, FEW, NF, W>), dim3((p.N + 16 * NF - 1) / (16 * NF)),
                     dim3(64 * W), lds, st, p);
}
// Columns and waves of a block: one block of 16 columns a unit up to 4096, and long stages of
// sixteen waves up to 8192; past that eight waves, two blocks a unit, and with fp32 planes, many
// columns in bf16 or very many in int8 the activations staged for 64 columns instead of 32.  us at
// K = 4096 in (16 columns, 16 waves) / (32, 16) / (32, 8) / (64, 8), fp32 past four rows in 8
// waves all: 8 rows in bf16 4096 6.1 / 7.3 / 7.3 / 9.2, 8192 10.4 / 8.5 / 8.1 / 9.9, 12288 14.5 /
// 13.8 / 11.0 / 10.6, 16384 18.5 / 15.1 / 12.1 / 11.6; 16 rows in bf16 8192 12.5 / 9.5 / 10.2 /
// 11.0, 65536 - / 56 / 44 / 42; in fp32 8192 24.8 / 16.5 / 16.7 / 16.9, 12288 34.8 / 27.9 / 27.9 /
// 17.5; in int8 16384 21.5 / 17.5 / 13.9 / 14.1, 65536 - / 58 / 42 / 49; 2 rows in bf16 8192 8.8 /
// 7.5 / 6.9 / 8.9, 24576 21.3 / 17.8 / 15.0 / 17.5, in int8 16384 15.7 / 13.0 / 10.3 / 11.1, 65536
// - / 41 / 30 / 28.
template <int A, int GS, bool FEW>
void launch_q4_few(const Q4Args& p, hipStream_t st) {
  constexpr int W = A == kActF32 && !FEW ? 8 : 16;  // 16 rows' planes of 16 superblocks: 197 KB
  if (p.N <= 4096)
    launch_q4_rows<A, GS, FEW, 1, W>(p, st);
  else if (p.N <= 8192)
    launch_q4_rows<A, GS, FEW, 2, W>(p, st);
  else if (A == kActQ8 ? !FEW || p.N < 28672 : FEW || (A == kActBF16 && p.N < 16384))
    launch_q4_rows<A, GS, FEW, 2, 8>(p, st);
  else if constexpr (FEW == (A == kActQ8))
    launch_q4_rows<A, GS, FEW, 4, 8>(p, st);
}
template <int A, int GS, int R, int W>
void launch_q4_vector(const Q4Args& p, hipStream_t st) {
  int KS = 1;  // slices: as many as there are, up to the block's waves
  while (KS < W && KS * 2048 < p.K) KS *= 2;
  // one round of 16 waves a unit
  const int most = kVectorRows / R;
  const long want = ((long)p.N * KS + 4096L * R - 1) / (4096L * R);
  const int iters = want < 1 ? 1 : want > most ? most : (int)want;
  const int rows = W / KS * R * iters;
  const dim3 grid((p.N + rows - 1) / rows);
  if (p.zeros)
    hipLaunchKernelGGL((q4_vector_kernel<A, GS, true, R, W>), grid, dim3(64 * W), 0, st, p, KS,
                       iters);
  else
    hipLaunchKernelGGL((q4_vector_kernel<A, GS, false, R, W>), grid, dim3(64 * W), 0, st, p, KS,
                       iters);
}
// Tiles by the rounds of 256 blocks they take: the smallest that need one, with several groups
// of waves on each; us in bf16 in 32 x 64 / 32 x 128 / 64 x 128 / 128 x 128: 48 x 7168 x 7168 25
// / 35 / 48 / 82, 64 x 16384 x 4096 29 / 23 / 30 / 49, 100 x 7168 x 7168 44 / 34 / 49 / 87, 128 x
// 16384 x 4096 54 / 34 / 32 / 52, 512 x 4096 x 4096 53 / 34 / 32 / 52; in fp32 and int8 at 64 x
// 16384 x 4096 58 / 41 / 64 / 106 and 49 / 35 / 57 / 107, at 128 x 16384 x 4096 108 / 73 / 67 /
// 109 and 91 / 67 / 62 / 107. Past one round a tile's cost goes with its size, nearly, and small
// ones waste less of the last round: in bf16 32 x 128, 96 x 128 and 128 x 128 take 78, 69 and 89
// us at 333 x 7168 x 7168 (groups of 64: 95, 82, 108), 99, 130 and 90 at 500 rows, 118, 121 and
// 105 at 512 x 16384 x 4096, 47, 42 and 51 at 288 x 9000 x 4096, 64, 54 and 65 at 384 x 8192 x
// 4096 in groups of 64. In fp32 (three planes of 96 rows do not fit twice) and int8 the two ends
// are 181, 190 and 149, 185 at the first, 241, 192 and 201, 187 at 500 rows, 104, 110 and 88, 109
// at 288 x 9000 x 4096.
template <int A, int GS>
void launch_q4_tiles(const Q4Args& p, hipStream_t st) {
  auto blocks = [&](long bm, long bn) {
    return ((p.M + bm - 1) / bm) * ((p.N + bn - 1) / bn);
  };
  auto rounds = [&](long bm, long bn) { return (blocks(bm, bn) + 255) / 256; };
  const long least = std::min(5 * rounds(32, 128), 16 * rounds(128, 128));
  if (blocks(32, 64) <= 256)
    launch_q4_tile<A, GS, 1, 1, 1, 2, 4>(p, st);
  else if (blocks(32, 128) <= 256)
    launch_q4_tile<A, GS, 1, 1, 1, 4, 2>(p, st);
  else if (blocks(64, 128) <= 256)
    launch_q4_tile<A, GS, 2, 1, 1, 4, 2>(p, st);
  else if (A == kActBF16 && 12 * rounds(96, 128) < least) {
    if constexpr (A == kActBF16) launch_q4_tile<A, GS, 3, 1, 1, 4, 2>(p, st);
  } else if (5 * rounds(32, 128) == least)
    launch_q4_tile<A, GS, 1, 1, 1, 4, 2>(p, st);
  else
    launch_q4_tile<A, GS, 2, 1, 2, 4, 1>(p, st);
}
template <int A, int GS>
void launch_q4_g(const Q4Args& p, hipStream_t st) {
  if (p.M == 1)
    launch_q4_vector<A, GS, 2, 8>(p, st);
  else if (p.M <= 4)
    launch_q4_few<A, GS, true>(p, st);
  else if (p.M <= 16)
    launch_q4_few<A, GS, false>(p, st);
  else
    launch_q4_tiles<A, GS>(p, st);
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
