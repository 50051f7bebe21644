// mhc_f8_matmul.hip -- out[m,n] = sum_k A[m,k] * B[n,k] of two 8-bit block
// matrices (mhc_f8.h), summed in fp32.
//
// Codes travel as bytes to the registers and become bf16 there, the block scale
// multiplied in by the same conversion (v_cvt_scalef32_pk_bf16_fp8, two codes per
// instruction): a code has four significant bits and the scale is a power of
// two, so the bf16 value is exact and the product runs on the bf16 matrix
// instructions.  The 8-bit ones were measured and are not used: they line up the
// eight products of a group on the largest one and keep 14 bits (a product 2^-14
// of another in its group is lost), which leaves 1.5e-5 of a sum of normal
// deviates and 5e-5 where a few columns are loud, against 9e-8 for bf16.
//
// The weight rows (n) are the instruction's row operand and the activation rows
// (m) its column operand, so a lane ends with four consecutive n of one m: one
// 16-byte store.  Both operands use one order of k within a block, whichever
// the loads give: a sum over the block does not depend on it.
#include "mhc_f8.h"
#include "mhc_kernels.h"

namespace mhc {

namespace {

__device__ __forceinline__ void store_quad(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<floatx4*>(p) = floatx4{a, b, c, d};
}
__device__ __forceinline__ unsigned bf16_pair(float a, float b) {
  const __hip_bfloat162 h = __float22bfloat162_rn(make_float2(a, b));
  unsigned u;
  __builtin_memcpy(&u, &h, 4);
  return u;
}
__device__ __forceinline__ void store_quad(__hip_bfloat16* p, float a, float b, float c,
                                           float d) {
  *reinterpret_cast<uint2*>(p) = make_uint2(bf16_pair(a, b), bf16_pair(c, d));
}

// 16 bytes from global memory to LDS without a register: lane i's bytes land at
// base + 16 * i (base the same for the whole wave).
__device__ __forceinline__ void load_to_lds(const unsigned char* src, unsigned char* base) {
  __builtin_amdgcn_global_load_lds(
      (const __attribute__((address_space(1))) void*)src,
      (__attribute__((address_space(3))) void*)base, 16, 0, 0);
}

}  // namespace

// ---------------------------------------------------------------- few rows
// At most 16*MT rows of A: a block takes 16 columns n, its W waves take the k
// blocks in turn and their sums are added in wave order through LDS.  The
// weight is read once, straight to registers, U blocks of it in flight per wave.
template <int MT, int W, int U, typename O>
__global__ __launch_bounds__(64 * W) void f8_matmul_narrow_kernel(
    const unsigned char* __restrict__ a, const unsigned char* __restrict__ as,
    const unsigned char* __restrict__ b, const unsigned char* __restrict__ bs, int bshift, int M,
    int N, int KB, O* __restrict__ out) {
  __shared__ floatx4 part[W][MT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16;
  // rows past the end read the last row; their results are not stored
  const int n = min(n0 + r, N - 1);
  const size_t pitch = (size_t)KB * kF8Block;
  const unsigned char* brow = b + n * pitch + 16 * g;
  const unsigned char* bsrow = bs + (size_t)(n >> bshift) * KB;
  const unsigned char* arow[MT];
  const unsigned char* asrow[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = min(16 * i + r, M - 1);
    arow[i] = a + m * pitch + 16 * g;
    asrow[i] = as + (size_t)m * KB;
  }
  floatx4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = floatx4{0.f, 0.f, 0.f, 0.f};
  for (int kb = wave; kb < KB; kb += W * U) {
    intx4 bv[U][2], av[U][MT][2];
    unsigned bsv[U], asv[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // a block past the end reads the row's last one, its weight codes as zeros
      const int k = min(kb + W * u, KB - 1);
      const size_t at = (size_t)k * kF8Block;
      bv[u][0] = __builtin_nontemporal_load(reinterpret_cast<const intx4*>(brow + at));
      bv[u][1] = __builtin_nontemporal_load(reinterpret_cast<const intx4*>(brow + at + 64));
      if (kb + W * u >= KB) bv[u][0] = bv[u][1] = intx4{0, 0, 0, 0};
      bsv[u] = bsrow[k];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        av[u][i][0] = *reinterpret_cast<const intx4*>(arow[i] + at);
        av[u][i][1] = *reinterpret_cast<const intx4*>(arow[i] + at + 64);
        asv[u][i] = asrow[i][k];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float sb = f8_scale(bsv[u]);
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const intx4 bq = bv[u][h >> 1];
        const bf16x8 bx = f8_to_bf16(bq[2 * (h & 1)], bq[2 * (h & 1) + 1], sb);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const intx4 aq = av[u][i][h >> 1];
          const bf16x8 ax =
              f8_to_bf16(aq[2 * (h & 1)], aq[2 * (h & 1) + 1], f8_scale(asv[u][i]));
          acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bx, ax, acc[i], 0, 0, 0);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  for (int i = threadIdx.x; i < MT * 64; i += 64 * W) {
    const int l = i & 63, mt = i >> 6;
    floatx4 s = part[0][mt][l];
#pragma unroll
    for (int w = 1; w < W; ++w) s += part[w][mt][l];
    const int m = 16 * mt + (l & 15), nq = n0 + 4 * (l >> 4);
    if (m < M && nq < N) store_quad(out + (size_t)m * N + nq, s[0], s[1], s[2], s[3]);
  }
}

// ---------------------------------------------------------------- tiles
// A block takes BM rows m and BN columns n; WM x WN waves, each with FM x FN
// products of v_mfma_f32_32x32x16_bf16.  The codes of one k block (128 bytes a
// row) are staged in LDS by direct loads, two stages in turn: the loads of the
// next block run under the products of this one, and one barrier a block keeps
// both sides in step.  Within a row's 128 bytes the 16-byte chunk c lies at place
// c ^ (row & 7), so that eight rows read at one chunk meet all banks; the place
// is chosen on the global side, since the direct load writes lanes in order.
template <int FM, int FN, int WM, int WN, typename O>
__global__ __launch_bounds__(64 * WM * WN, (WM * WN + 3) / 4) void f8_matmul_tile_kernel(
    const unsigned char* __restrict__ a, const unsigned char* __restrict__ as,
    const unsigned char* __restrict__ b, const unsigned char* __restrict__ bs, int bshift, int M,
    int N, int KB, int MT, int NT, O* __restrict__ out) {
  constexpr int W = WM * WN, BM = 32 * FM * WM, BN = 32 * FN * WN;
  constexpr int LOADS = (BM + BN) / 8 / W;  // wave loads (8 rows of 128 bytes) a stage
  static_assert(LOADS * 8 * W == BM + BN && BM % 8 == 0, "whole wave loads");
  __shared__ __align__(16) unsigned char stage[2][(BM + BN) * kF8Block];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 31, h = lane >> 5;
  const int wm = wave % WM, wn = wave / WM;

  // Blocks go to the eight dies in turn: give each die a run of tiles, and walk
  // them eight rows of tiles at a time, so that its L2 sees few panels at once.
  const int tiles = MT * NT;
  int id = blockIdx.x;
  {
    const int per = tiles / 8, rest = tiles % 8, die = id % 8, at = id / 8;
    id = die * per + min(die, rest) + at;
  }
  const int band = id / (8 * NT), in_band = id - band * 8 * NT;
  const int rows = min(8, MT - band * 8);
  const int m0 = (band * 8 + in_band % rows) * BM, n0 = (in_band / rows) * BN;

  const size_t pitch = (size_t)KB * kF8Block;
  // this wave's share of a stage: wave load i covers staged rows 8*(i*W + wave)
  const unsigned char* src[LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const int row = 8 * (i * W + wave) + (lane >> 3);
    const int chunk = (lane & 7) ^ (row & 7);
    src[i] = (row < BM ? a + min(m0 + row, M - 1) * pitch
                       : b + min(n0 + row - BM, N - 1) * pitch) + chunk * 16;
  }
  const unsigned char* asrow[FM];
  const unsigned char* bsrow[FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
    asrow[i] = as + (size_t)min(m0 + (wm * FM + i) * 32 + r, M - 1) * KB;
#pragma unroll
  for (int j = 0; j < FN; ++j)
    bsrow[j] = bs + (size_t)(min(n0 + (wn * FN + j) * 32 + r, N - 1) >> bshift) * KB;

  floatx16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  unsigned sa[FM], sb[FN];
  auto fetch = [&](int kb, int buf) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      load_to_lds(src[i] + (size_t)kb * kF8Block, &stage[buf][8 * (i * W + wave) * kF8Block]);
  };
  auto scales = [&](int kb) {
#pragma unroll
    for (int i = 0; i < FM; ++i) sa[i] = asrow[i][kb];
#pragma unroll
    for (int j = 0; j < FN; ++j) sb[j] = bsrow[j][kb];
  };
  if (KB > 0) {
    fetch(0, 0);
    scales(0);
  }
  for (int kb = 0; kb < KB; ++kb) {
    // stage kb has landed (this wave's part; the barrier adds the others'), and
    // every wave is done with the other buffer
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    float fa[FM], fb[FN];
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[i] = f8_scale(sa[i]);
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[j] = f8_scale(sb[j]);
    if (kb + 1 < KB) {
      fetch(kb + 1, (kb + 1) & 1);
      scales(kb + 1);
    }
    const unsigned char* arow = &stage[kb & 1][(wm * FM * 32 + r) * kF8Block];
    const unsigned char* brow = &stage[kb & 1][(BM + wn * FN * 32 + r) * kF8Block];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int place = ((2 * c + h) ^ (r & 7)) * 16;
      intx4 av[FM], bv[FN];
#pragma unroll
      for (int i = 0; i < FM; ++i)
        av[i] = *reinterpret_cast<const intx4*>(arow + i * 32 * kF8Block + place);
#pragma unroll
      for (int j = 0; j < FN; ++j)
        bv[j] = *reinterpret_cast<const intx4*>(brow + j * 32 * kF8Block + place);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        bf16x8 ax[FM], bx[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) bx[j] = f8_to_bf16(bv[j][2 * s], bv[j][2 * s + 1], fb[j]);
#pragma unroll
        for (int i = 0; i < FM; ++i) ax[i] = f8_to_bf16(av[i][2 * s], av[i][2 * s + 1], fa[i]);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bx[j], ax[i], acc[i][j], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int m = m0 + (wm * FM + i) * 32 + r;
    if (m >= M) continue;
    O* orow = out + (size_t)m * N;
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int n = n0 + (wn * FN + j) * 32 + 8 * v + 4 * h;
        if (n < N)
          store_quad(orow + n, acc[i][j][4 * v], acc[i][j][4 * v + 1], acc[i][j][4 * v + 2],
                     acc[i][j][4 * v + 3]);
      }
  }
}

namespace {

template <typename O>
struct Args {
  const unsigned char *a, *as, *b, *bs;
  int bshift, M, N, KB;
  O* out;
  hipStream_t st;
};

template <int MT, int W, int U, typename O>
void narrow(const Args<O>& p) {
  hipLaunchKernelGGL((f8_matmul_narrow_kernel<MT, W, U, O>), dim3((p.N + 15) / 16),
                     dim3(64 * W), 0, p.st, p.a, p.as, p.b, p.bs, p.bshift, p.M, p.N, p.KB,
                     p.out);
}
template <int FM, int FN, int WM, int WN, typename O>
void tile(const Args<O>& p) {
  const int MT = (p.M + 32 * FM * WM - 1) / (32 * FM * WM);
  const int NT = (p.N + 32 * FN * WN - 1) / (32 * FN * WN);
  hipLaunchKernelGGL((f8_matmul_tile_kernel<FM, FN, WM, WN, O>), dim3((unsigned)(MT * NT)),
                     dim3(64 * WM * WN), 0, p.st, p.a, p.as, p.b, p.bs, p.bshift, p.M, p.N, p.KB,
                     MT, NT, p.out);
}
long tiles_of(long M, long N, long bm, long bn) {
  return ((M + bm - 1) / bm) * ((N + bn - 1) / bn);
}

template <typename O>
void matmul(const Args<O>& p) {
  if (p.M <= 16) {
    narrow<1, 8, 4>(p);
  } else if (tiles_of(p.M, p.N, 256, 256) >= 192) {
    tile<4, 2, 2, 4>(p);
  } else if (tiles_of(p.M, p.N, 128, 128) >= 192) {
    tile<2, 2, 2, 2>(p);
  } else {
    tile<1, 1, 2, 2>(p);
  }
}
}  // namespace

hipError_t launch_f8_matmul(const unsigned char* a, const unsigned char* as,
                            const unsigned char* b, const unsigned char* bs, bool square, int M,
                            int N, int K, void* out, bool bf16, hipStream_t st) {
  const int KB = K / kF8Block, bshift = square ? 7 : 0;
  if (bf16)
    matmul(Args<__hip_bfloat16>{a, as, b, bs, bshift, M, N, KB,
                                static_cast<__hip_bfloat16*>(out), st});
  else
    matmul(Args<float>{a, as, b, bs, bshift, M, N, KB, static_cast<float*>(out), st});
  return hipGetLastError();
}

}  // namespace mhc
