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

}  // namespace

// ---------------------------------------------------------------- few rows
// At most 16*MT rows of A: a block takes 16*NF columns n, its W waves take the k
// blocks in turn and their sums are added in wave order through LDS.  The
// weight is read once, straight to registers, U blocks of it in flight per wave.
template <int MT, int NF, int W, int U, typename O>
__global__ __launch_bounds__(64 * W) void f8_matmul_narrow_kernel(
    const unsigned char* __restrict__ a, const unsigned char* __restrict__ as,
    const unsigned char* __restrict__ b, const unsigned char* __restrict__ bs, int bshift, int M,
    int N, int KB, int pitch_o, O* __restrict__ out) {
  __shared__ floatx4 part[W][MT * NF][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16 * NF;
  // rows past the end read the last row; their results are not stored
  const size_t pitch = (size_t)KB * kF8Block;
  const unsigned char *brow[NF], *bsrow[NF], *arow[MT], *asrow[MT];
#pragma unroll
  for (int j = 0; j < NF; ++j) {
    const int n = min(n0 + 16 * j + r, N - 1);
    brow[j] = b + n * pitch + 16 * g;
    bsrow[j] = bs + (size_t)(n >> bshift) * KB;
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = min(16 * i + r, M - 1);
    arow[i] = a + m * pitch + 16 * g;
    asrow[i] = as + (size_t)m * KB;
  }
  floatx4 acc[MT][NF];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  for (int kb = wave; kb < KB; kb += W * U) {
    intx4 bv[U][NF][2], av[U][MT][2];
    unsigned bsv[U][NF], asv[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // a block past the end reads the row's last one, its codes as zeros
      const int k = min(kb + W * u, KB - 1);
      const size_t at = (size_t)k * kF8Block;
#pragma unroll
      for (int j = 0; j < NF; ++j) {
        bv[u][j][0] = *reinterpret_cast<const intx4*>(brow[j] + at);
        bv[u][j][1] = *reinterpret_cast<const intx4*>(brow[j] + at + 64);
        bsv[u][j] = bsrow[j][k];
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        av[u][i][0] = *reinterpret_cast<const intx4*>(arow[i] + at);
        av[u][i][1] = *reinterpret_cast<const intx4*>(arow[i] + at + 64);
        asv[u][i] = asrow[i][k];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kb + W * u >= KB) {  // of both operands: zero times an infinity is not zero
#pragma unroll
        for (int j = 0; j < NF; ++j) bv[u][j][0] = bv[u][j][1] = intx4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < MT; ++i) av[u][i][0] = av[u][i][1] = intx4{0, 0, 0, 0};
      }
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        bf16x8 ax[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const intx4 q = av[u][i][h >> 1];
          ax[i] = f8_to_bf16(q[2 * (h & 1)], q[2 * (h & 1) + 1], f8_scale(asv[u][i]));
        }
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          const intx4 q = bv[u][j][h >> 1];
          const bf16x8 bx =
              f8_to_bf16(q[2 * (h & 1)], q[2 * (h & 1) + 1], f8_scale(bsv[u][j]));
#pragma unroll
          for (int i = 0; i < MT; ++i)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bx, ax[i], acc[i][j], 0, 0, 0);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) part[wave][i * NF + j][lane] = acc[i][j];
  __syncthreads();
  for (int i = threadIdx.x; i < MT * NF * 64; i += 64 * W) {
    const int l = i & 63, f = i >> 6;
    floatx4 s = part[0][f][l];
#pragma unroll
    for (int w = 1; w < W; ++w) s += part[w][f][l];
    const int m = 16 * (f / NF) + (l & 15), nq = n0 + 16 * (f % NF) + 4 * (l >> 4);
    if (m < M && nq < N) store_quad(out + (size_t)m * pitch_o + nq, s[0], s[1], s[2], s[3]);
  }
}

// ---------------------------------------------------------------- tiles
namespace {
constexpr int kPanel = 32;  // k blocks whose scales are held in LDS
}
// A block takes BM rows m and BN columns n; WM x WN waves, each with FM x FN
// products of v_mfma_f32_32x32x16_bf16, which at 32 x 32 run at twice the rate of
// the 16 x 16 ones.  The codes of one k block (128 bytes a row) are staged in LDS
// by direct loads, NS stages in turn: while one block is multiplied the loads of
// the NS - 1 after it are under way, and one barrier a block keeps the waves in
// step.  With KG > 1 a stage holds KG blocks, each for a group of waves of its own
// (WM x WN waves again), and the groups' sums are added in order at the end: more
// waves on a tile where there are few tiles.  A lane's 16 bytes are read a chunk
// ahead of their use and converted next to it; converted on the way into LDS instead
// (once, not by every wave) the bytes in LDS double, and 333 x 7168 x 7168 took 79 us
// against 55.
// Within a row's 128 bytes the 16-byte chunk c lies at place c ^ (row / 2 % 8), so
// that sixteen rows read at one chunk meet all 64 banks; the place is chosen on
// the global side, since a direct load writes its lanes in order.
// What bounds it: with neither loads nor conversions the products alone take
// 442 us at 4096 x 16384 x 4096 (1240 TFLOP/s; the library's bf16 product of these
// sizes 420), with them 540: the conversions cost 50, the staging 50.  The staging is
// not all asynchronous (see the stages below), nor is a panel of scales, whose loads are
// waited for one after the other.
template <int FM, int FN, int WM, int WN, int NS, int KG, typename O>
__global__ __launch_bounds__(64 * WM * WN * KG, 2) void f8_matmul_tile_kernel(
    const unsigned char* __restrict__ a, const unsigned char* __restrict__ as,
    const unsigned char* __restrict__ b, const unsigned char* __restrict__ bs, int bshift, int M,
    int N, int KB, int pitch_o, int MT, int NT, O* __restrict__ out) {
  constexpr int W = WM * WN * KG, BM = 32 * FM * WM, BN = 32 * FN * WN, ROWS = BM + BN;
  constexpr int LOADS = KG * ROWS / 8 / W;  // wave loads (8 rows of 128 bytes) a stage
  constexpr int STAGE = KG * ROWS * kF8Block;
  static_assert(LOADS * 8 * W == KG * ROWS && BM % 8 == 0, "whole wave loads");
  static_assert(kPanel % KG == 0 && (KG - 1) * WM * WN * FM * FN * 4096 <= STAGE, "sums fit");
  // One variable a stage, by which the compiler can tell a read from the loads under way
  // into the others.  It does at some places only: elsewhere (four of the eight chunks of
  // two stages in 256 x 256 tiles, the first of three stages in 64 x 64) it waits for every
  // load before it reads, and what was asked for a chunk before is waited for there.
  __shared__ __align__(16) unsigned char stage0[STAGE];
  __shared__ __align__(16) unsigned char stage1[STAGE];
  __shared__ __align__(16) unsigned char stage2[NS > 2 ? STAGE : 16];
  __shared__ unsigned char panel[kPanel][ROWS];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, h = lane >> 5;
  const int wm = wave % WM, wn = wave / WM % WN, kg = wave / (WM * WN);
  const int KI = (KB + KG - 1) / KG;  // stages of KG blocks

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
    const int row = 8 * (i * W + wave) % ROWS + (lane >> 3);
    const int chunk = (lane & 7) ^ ((row >> 1) & 7);
    src[i] = (row < BM ? a + min(m0 + row, M - 1) * pitch
                       : b + min(n0 + row - BM, N - 1) * pitch) + chunk * 16;
  }
  floatx16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  auto stage_of = [&](int i) -> unsigned char* {
    return i == 0 ? stage0 : i == 1 ? stage1 : stage2;
  };
  // part p of three of this wave's loads of the KG blocks ki, into stage `to` (a block
  // past the end: the last one, which nobody reads)
  auto fetch = [&](int ki, int to, int p) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      if (i * 3 / LOADS == p) {
        const int kb = KG == 1 ? ki : min(ki * KG + 8 * (i * W + wave) / ROWS, KB - 1);
        load_to_lds(src[i] + (size_t)kb * kF8Block,
                    stage_of(to) + 8 * (i * W + wave) * kF8Block);
      }
  };
  // The scale bytes of the next kPanel blocks, turned so that a lane reads its row's
  // beside its neighbours': straight from memory every lane would meet a line of
  // its own, for each row of products and each block.
  auto load_panel = [&](int kb) {
    for (int row = threadIdx.x; row < ROWS; row += 64 * W) {
      const unsigned char* p =
          row < BM ? as + (size_t)min(m0 + row, M - 1) * KB
                   : bs + (size_t)(min(n0 + row - BM, N - 1) >> bshift) * KB;
      const int count = min(kPanel, KB - kb);
      int i = 0;
      if (KB % 4 == 0)
        for (; i + 4 <= count; i += 4) {
          const unsigned v = *reinterpret_cast<const unsigned*>(p + kb + i);
#pragma unroll
          for (int e = 0; e < 4; ++e) panel[i + e][row] = (unsigned char)(v >> (8 * e));
        }
      for (; i < count; ++i) panel[i][row] = p[kb + i];
    }
  };
  float fa[FM], fb[FN];
  // Stage ki has landed (this wave's part; the barrier adds the others') while the
  // NS - 2 stages after it may be on their way, and every wave has taken what it
  // needs of the stage before it and of the panel.
  auto turn = [&](int ki) {
    if (NS > 2 && ki + NS - 2 < KI)
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(LOADS * (NS - 2)) : "memory");
    else
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (ki % (kPanel / KG) == 0) {
      load_panel(ki * KG);
      __syncthreads();
    }
    const unsigned char* scales = panel[ki % (kPanel / KG) * KG + kg];
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[i] = f8_scale(scales[(wm * FM + i) * 32 + r]);
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[j] = f8_scale(scales[BM + (wn * FN + j) * 32 + r]);
  };
  intx4 av[2][FM], bv[2][FN];
  auto read = [&](int from, int c, int to) {
    const unsigned char* arow = stage_of(from) + (kg * ROWS + wm * FM * 32 + r) * kF8Block;
    const unsigned char* brow = stage_of(from) + (kg * ROWS + BM + wn * FN * 32 + r) * kF8Block;
    const int place = ((2 * c + h) ^ ((r >> 1) & 7)) * 16;
#pragma unroll
    for (int j = 0; j < FN; ++j)
      bv[to][j] = *reinterpret_cast<const intx4*>(brow + j * 32 * kF8Block + place);
#pragma unroll
    for (int i = 0; i < FM; ++i)
      av[to][i] = *reinterpret_cast<const intx4*>(arow + i * 32 * kF8Block + place);
  };
  if (KI > 0) {
#pragma unroll
    for (int k = 0; k < NS - 1; ++k)
#pragma unroll
      for (int p = 0; p < 3; ++p)
        if (k < KI) fetch(k, k, p);
    turn(0);
    read(0, 0, 0);
    if (NS - 1 < KI) fetch(NS - 1, NS - 1, 0);
  }
  for (int k0 = 0; k0 < KI; k0 += NS) {
#pragma unroll
    for (int here = 0; here < NS; ++here) {
      const int ki = k0 + here, free = (here + NS - 1) % NS;
      if (ki >= KI) break;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float ga[FM], gb[FN];
#pragma unroll
        for (int i = 0; i < FM; ++i) ga[i] = fa[i];
#pragma unroll
        for (int j = 0; j < FN; ++j) gb[j] = fb[j];
        // The next chunk is read while this one is multiplied; with the last chunk in
        // registers the stage is done with, the next one is turned to, and the loads
        // of a later one into the free stage begin, a third at a time.
        if (c < 3) {
          read(here, c + 1, (c + 1) & 1);
          if (c < 2 && ki + NS - 1 < KI) fetch(ki + NS - 1, free, c + 1);
        } else if (ki + 1 < KI) {
          turn(ki + 1);
          read((here + 1) % NS, 0, 0);
          if (ki + NS < KI) fetch(ki + NS, here, 0);
        }
        if (KG > 1 && ki * KG + kg >= KB) continue;  // a group past the end
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          bf16x8 ax[FM], bx[FN];
#pragma unroll
          for (int j = 0; j < FN; ++j)
            bx[j] = f8_to_bf16(bv[c & 1][j][2 * s], bv[c & 1][j][2 * s + 1], gb[j]);
#pragma unroll
          for (int i = 0; i < FM; ++i) {
            ax[i] = f8_to_bf16(av[c & 1][i][2 * s], av[c & 1][i][2 * s + 1], ga[i]);
#pragma unroll
            for (int j = 0; j < FN; ++j)
              acc[i][j] =
                  __builtin_amdgcn_mfma_f32_32x32x16_bf16(bx[j], ax[i], acc[i][j], 0, 0, 0);
          }
        }
      }
    }
  }
  if constexpr (KG > 1) {  // the groups' sums, in their order, through the first stage
    float4* sums = reinterpret_cast<float4*>(stage0);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __syncthreads();
    if (kg > 0) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            sums[(((wave - WM * WN) * FM + i) * FN + j) * 256 + v * 64 + lane] =
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
                sums[((((k - 1) * WM * WN + wave) * FM + i) * FN + j) * 256 + v * 64 + lane];
            acc[i][j][4 * v] += o.x;
            acc[i][j][4 * v + 1] += o.y;
            acc[i][j][4 * v + 2] += o.z;
            acc[i][j][4 * v + 3] += o.w;
          }
  }
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int m = m0 + (wm * FM + i) * 32 + r;
    if (m >= M) continue;
    O* orow = out + (size_t)m * pitch_o;
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
  int bshift, M, N, KB, pitch_o;
  O* out;
  hipStream_t st;
};

template <int MT, int NF, int W, int U, typename O>
void narrow(const Args<O>& p) {
  hipLaunchKernelGGL((f8_matmul_narrow_kernel<MT, NF, W, U, O>),
                     dim3((p.N + 16 * NF - 1) / (16 * NF)), dim3(64 * W), 0, p.st, p.a, p.as,
                     p.b, p.bs, p.bshift, p.M, p.N, p.KB, p.pitch_o, p.out);
}
template <int FM, int FN, int WM, int WN, int NS, int KG, typename O>
void tile(const Args<O>& p) {
  const int MT = (p.M + 32 * FM * WM - 1) / (32 * FM * WM);
  const int NT = (p.N + 32 * FN * WN - 1) / (32 * FN * WN);
  hipLaunchKernelGGL((f8_matmul_tile_kernel<FM, FN, WM, WN, NS, KG, O>),
                     dim3((unsigned)(MT * NT)), dim3(64 * WM * WN * KG), 0, p.st, p.a, p.as, p.b,
                     p.bs, p.bshift, p.M, p.N, p.KB, p.pitch_o, MT, NT, p.out);
}
long tiles_of(long M, long N, long bm, long bn) {
  return ((M + bm - 1) / bm) * ((N + bn - 1) / bn);
}

// Columns of one launch: its threads stay below the 2^32 that a grid's dimension may
// have (64 a column at most, in the narrow kernel), its rounding up in an int.
constexpr int kLaunchCols = 1 << 24;

template <typename O>
void matmul(const Args<O>& p) {
  if (p.N > kLaunchCols) {
    for (int n0 = 0; n0 < p.N;) {
      Args<O> part = p;
      part.b += (size_t)n0 * p.KB * kF8Block;
      part.bs += (size_t)(n0 >> p.bshift) * p.KB;
      part.out += n0;
      part.N = p.N - n0 < kLaunchCols ? p.N - n0 : kLaunchCols;
      n0 += part.N;
      matmul(part);
    }
    return;
  }
  // Few rows: the weight streams through the narrow kernel, 16 columns a block for as
  // many blocks as there are.  From five rows on and where 64 columns a block still fill
  // the 256 units: 32 blocks of the depth in flight at a time.  us at 16 and at 64
  // columns, 8 rows: N = 8192 9.6 and 12.0 at K = 4096, 16.6 and 21.5 at 8192; N = 12288
  // 13.0 and 12.2, 23.3 and 21.9 (the crossing); N = 16384 16.4 and 13.5, 30.4 and 24.7; N
  // = 24576, a round and a half, 23.3 and 23.5, 46 and 52; N = 32768 30.0 and 25.5, 60 and
  // 57.  One row: 12.7 and 13.2, 22.3 and 24.4 at N = 16384, 22.3 and 25.2 at 32768.
  // Shallow products, and from 17 rows on, take the tiles with four blocks of the depth at
  // a time: 16 columns and tiles, at K = 2048, 1 x 8192 7.3 and 8.3, 1 x 16384 12.1 and
  // 9.9, 1 x 24576 16.8 and 17.3, 16 x 5120 10.4 and 7.8, 16 x 16384 18.7 and 10.1; at
  // K = 4096 16 x 8192 11.6 and 13.7; 32 x 8192 x 4096 14.6 and, narrow, 17.9, 32 x 4096 x
  // 4096 13.8 and 9.9.
  auto rounds = [&](int b) { return (tiles_of(p.M, p.N, b, b) + 255) / 256; };
  const long tiles64 = tiles_of(p.M, p.N, 64, 64);
  const int side = p.M < p.N ? p.M : p.N;
  const bool shallow = p.KB <= 16 && (p.N >= 16384 || (p.M > 8 && p.N >= 5120));
  if (p.M <= 16 && !shallow) {
    p.M > 4 && p.N >= 16384 ? narrow<1, 4, 8, 4>(p) : narrow<1, 1, 16, 2>(p);
  } else if (p.M <= 32 && p.N < 5120) {
    narrow<2, 1, 16, 2>(p);
  // One tile to a compute unit at most: eight waves on it, in four groups that take
  // every fourth block of the depth (100 x 7168 x 7168 23 us against 36 with four waves
  // and no groups, 128 x 4096 x 1024 7.1 and 7.6, 70 x 4096 x 256 5.2 and 4.7).
  } else if (p.M <= 32 || (tiles64 <= 256 && p.KB >= 8)) {
    tile<2, 1, 1, 2, 2, 4>(p);
  // By the rounds of 256 tiles: one of 256 x 256 takes 3.1 times as long as one of 128 x
  // 128 (4096 rows, K = 4096, us in large and in small tiles: N = 4096 110 and 130, 4608
  // 184 and 156, 6144 192 and 195, 7168 198 and 224, 8192 251 and 267; 4096 x 9216 x 2048
  // 163 and 152; 128 x 65536 x 1024 33 and 25).
  } else if (31 * rounds(256) <= 10 * rounds(128)) {
    tile<4, 2, 2, 4, 2, 1>(p);
  // 128 x 128 against 64 x 64, three of those to a unit: 1024 x 4096 x 4096 41 and 49 us,
  // 512 x 4096 x 4096 37 and 27; 65536 x 128 x 4096 84 and 106, 32768 x 64 x 4096 43 and 33.
  } else if (side > 64 && tiles_of(p.M, p.N, 128, 128) >= 192) {
    tile<2, 1, 2, 4, 2, 1>(p);
  } else {
    tile<1, 1, 2, 2, 3, 1>(p);
  }
}
}  // namespace

hipError_t launch_f8_matmul(const unsigned char* a, const unsigned char* as,
                            const unsigned char* b, const unsigned char* bs, bool square, int M,
                            int N, int K, void* out, bool bf16, hipStream_t st) {
  const int KB = K / kF8Block, bshift = square ? 7 : 0;
  if (bf16)
    matmul(Args<__hip_bfloat16>{a, as, b, bs, bshift, M, N, KB, N,
                                static_cast<__hip_bfloat16*>(out), st});
  else
    matmul(Args<float>{a, as, b, bs, bshift, M, N, KB, N, static_cast<float*>(out), st});
  return hipGetLastError();
}

}  // namespace mhc
