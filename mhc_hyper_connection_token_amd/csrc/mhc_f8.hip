// mhc_f8.hip -- the 8-bit block format: encode along rows, along columns, in
// 128 x 128 squares, the transpose of an encoded matrix, and decode.
//
// All of it streams: a matrix is read once and its codes written once.  The
// row kernel gives a half-wave one block of 128 entries (a quad per lane), so a
// block's maximum is five lane exchanges and its codes one dword per lane.  The
// tile kernel holds 128 x 128 entries in registers (16 rows of a quad column
// per thread), takes the maxima along either axis from there, and turns the
// codes of the other axis through LDS so that both are written in whole lines.
#include "mhc_f8.h"
#include "mhc_kernels.h"

namespace mhc {

namespace {
constexpr int kRowsUnroll = 4;  // blocks per half-wave, all loads in flight at once
// Rows of a tile that a thread holds: 8 gives 4 waves per SIMD (at 16 the registers
// leave 2: 16.0 against 12.3 us for 1001 x 7168 bf16 both ways; at 4 a block's 1024
// threads spill).
constexpr int kTileRows = 8;
constexpr int kTileThreads = 32 * kF8Block / kTileRows;
}

template <typename E>
__global__ __launch_bounds__(256) void f8_encode_rows_kernel(const E* __restrict__ x,
                                                             unsigned nblocks, unsigned KB,
                                                             int cols,
                                                             unsigned char* __restrict__ codes,
                                                             unsigned char* __restrict__ scales) {
  const int lane = threadIdx.x & 63, l = lane & 31;
  const unsigned wave = blockIdx.x * 4u + (threadIdx.x >> 6);
  const unsigned b0 = wave * (2 * kRowsUnroll) + (lane >> 5);
  float4 v[kRowsUnroll];
#pragma unroll
  for (int u = 0; u < kRowsUnroll; ++u) {
    const unsigned b = b0 + 2 * u;
    v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (b < nblocks) {
      const unsigned row = b / KB;
      const int col = (int)(b - row * KB) * kF8Block + 4 * l;
      if (col < cols) v[u] = load_quad<E>(x + (size_t)row * cols + col);
    }
  }
#pragma unroll
  for (int u = 0; u < kRowsUnroll; ++u) {
    const unsigned b = b0 + 2 * u;
    const unsigned a = umax_half(max(max(f8_size(v[u].x), f8_size(v[u].y)),
                                     max(f8_size(v[u].z), f8_size(v[u].w))));
    const unsigned byte = f8_scale_byte(a);
    const unsigned q = f8_pack(v[u].x, v[u].y, v[u].z, v[u].w, f8_inverse(byte));
    if (b < nblocks) {
      reinterpret_cast<unsigned*>(codes)[(size_t)b * 32 + l] = q;
      if (l == 0) scales[b] = (unsigned char)byte;
    }
  }
}

// One 128 x 128 tile per block.  Thread (rg, cq): rows kTileRows*rg and on,
// columns 4*cq .. +3.  E = unsigned char reads codes with their row scales (xs).
// codes / codes_t: either may be null; with SQUARE one scale serves the tile.
template <typename E, bool SQUARE>
__global__ __launch_bounds__(kTileThreads) void f8_encode_tile_kernel(
    const E* __restrict__ x, const unsigned char* __restrict__ xs, int rows, int cols, int KB,
    int RB, unsigned char* __restrict__ codes, unsigned char* __restrict__ scales,
    unsigned char* __restrict__ codes_t, unsigned char* __restrict__ scales_t) {
  constexpr int NR = kTileRows, NG = kF8Block / NR, NW = NR / 4;
  __shared__ unsigned cmax[NG][kF8Block];
  __shared__ __align__(16) unsigned turn[kF8Block * 32];
  const int tid = threadIdx.x, cq = tid & 31, rg = tid >> 5;
  const int rb = blockIdx.x / KB, kb = blockIdx.x - rb * KB;
  const int row0 = rb * kF8Block + rg * NR, col = kb * kF8Block + 4 * cq;
  float4 v[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row0 + i < rows && col < cols) {
      if constexpr (sizeof(E) == 1) {
        const size_t at = (size_t)(row0 + i) * KB + kb;
        v[i] = f8_unpack(reinterpret_cast<const unsigned*>(x)[at * 32 + cq], f8_scale(xs[at]));
      } else {
        v[i] = load_quad<E>(x + (size_t)(row0 + i) * cols + col);
      }
    }
  }
  unsigned m[4] = {0u, 0u, 0u, 0u}, row_byte[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const unsigned a0 = f8_size(v[i].x), a1 = f8_size(v[i].y);
    const unsigned a2 = f8_size(v[i].z), a3 = f8_size(v[i].w);
    m[0] = max(m[0], a0);
    m[1] = max(m[1], a1);
    m[2] = max(m[2], a2);
    m[3] = max(m[3], a3);
    row_byte[i] = SQUARE ? 0 : max(max(a0, a1), max(a2, a3));
  }
  unsigned tile_byte = 0;
  if (SQUARE) {
    const unsigned a = umax_half(max(max(m[0], m[1]), max(m[2], m[3])));
    if (cq == 0) cmax[0][rg] = a;
    __syncthreads();
    unsigned t = 0;
#pragma unroll
    for (int g = 0; g < NG; ++g) t = max(t, cmax[0][g]);
    tile_byte = f8_scale_byte(t);
  } else if (codes_t) {
    *reinterpret_cast<uint4*>(&cmax[rg][4 * cq]) = make_uint4(m[0], m[1], m[2], m[3]);
  }
  const size_t pitch = (size_t)KB * kF8Block, pitch_t = (size_t)RB * kF8Block;
  if (codes) {
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const unsigned byte = SQUARE ? tile_byte : f8_scale_byte(umax_half(row_byte[i]));
      if (row0 + i < rows) {
        reinterpret_cast<unsigned*>(codes + (row0 + i) * pitch)[kb * 32 + cq] =
            f8_pack(v[i].x, v[i].y, v[i].z, v[i].w, f8_inverse(byte));
        if (!SQUARE && cq == 0) scales[(size_t)(row0 + i) * KB + kb] = (unsigned char)byte;
      }
    }
  }
  if (SQUARE && tid == 0) {
    if (codes) scales[(size_t)rb * KB + kb] = (unsigned char)tile_byte;
    if (codes_t) scales_t[(size_t)kb * RB + rb] = (unsigned char)tile_byte;
  }
  if (!codes_t) return;
  if (!SQUARE) {
    __syncthreads();
    uint4 t = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const uint4 c = *reinterpret_cast<const uint4*>(&cmax[g][4 * cq]);
      t = make_uint4(max(t.x, c.x), max(t.y, c.y), max(t.z, c.z), max(t.w, c.w));
    }
    m[0] = t.x, m[1] = t.y, m[2] = t.z, m[3] = t.w;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const unsigned byte = SQUARE ? tile_byte : f8_scale_byte(m[j]);
    if (!SQUARE && rg == 0 && col + j < cols)
      scales_t[(size_t)(col + j) * RB + rb] = (unsigned char)byte;
    const float inv = f8_inverse(byte);
    // The 16-byte chunk of a column is put where its number xor the column quad
    // says, so that neither these writes nor the reads below meet the same banks.
    const int at = (4 * cq + j) * 32, chunk = rg * NW / 4, part = rg * NW % 4;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const float4* p = v + 4 * i;
      const float e0 = j == 0 ? p[0].x : j == 1 ? p[0].y : j == 2 ? p[0].z : p[0].w;
      const float e1 = j == 0 ? p[1].x : j == 1 ? p[1].y : j == 2 ? p[1].z : p[1].w;
      const float e2 = j == 0 ? p[2].x : j == 1 ? p[2].y : j == 2 ? p[2].z : p[2].w;
      const float e3 = j == 0 ? p[3].x : j == 1 ? p[3].y : j == 2 ? p[3].z : p[3].w;
      turn[at + (chunk ^ (cq & 7)) * 4 + part + i] = f8_pack(e0, e1, e2, e3, inv);
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 1024 / kTileThreads; ++k) {
    const int idx = k * kTileThreads + tid, c = idx >> 3, ch = idx & 7;
    if (kb * kF8Block + c < cols)
      *reinterpret_cast<uint4*>(codes_t + (size_t)(kb * kF8Block + c) * pitch_t + rb * kF8Block +
                                ch * 16) =
          *reinterpret_cast<const uint4*>(&turn[c * 32 + (ch ^ ((c >> 2) & 7)) * 4]);
  }
}

__global__ __launch_bounds__(256) void f8_decode_kernel(const unsigned char* __restrict__ codes,
                                                        const unsigned char* __restrict__ scales,
                                                        unsigned nblocks, unsigned KB, int cols,
                                                        float* __restrict__ out) {
  const int lane = threadIdx.x & 63, l = lane & 31;
  const unsigned wave = blockIdx.x * 4u + (threadIdx.x >> 6);
  const unsigned b0 = wave * (2 * kRowsUnroll) + (lane >> 5);
  unsigned q[kRowsUnroll], s[kRowsUnroll];
#pragma unroll
  for (int u = 0; u < kRowsUnroll; ++u) {
    const unsigned b = b0 + 2 * u;
    q[u] = s[u] = 0;
    if (b < nblocks) {
      q[u] = __builtin_nontemporal_load(reinterpret_cast<const unsigned*>(codes) +
                                        (size_t)b * 32 + l);
      s[u] = scales[b];
    }
  }
#pragma unroll
  for (int u = 0; u < kRowsUnroll; ++u) {
    const unsigned b = b0 + 2 * u;
    const unsigned row = b / KB;
    const int col = (int)(b - row * KB) * kF8Block + 4 * l;
    if (b < nblocks && col < cols)
      *reinterpret_cast<float4*>(out + (size_t)row * cols + col) = f8_unpack(q[u], f8_scale(s[u]));
  }
}

namespace {
unsigned row_grid(unsigned nblocks) {
  const unsigned per = 4u * 2u * kRowsUnroll;
  return nblocks / per + (nblocks % per != 0);
}
template <typename E>
void encode(const E* x, const unsigned char* xs, int rows, int cols, bool square,
            unsigned char* codes, unsigned char* scales, unsigned char* codes_t,
            unsigned char* scales_t, hipStream_t st) {
  const int KB = (cols + kF8Block - 1) / kF8Block;
  const int RB = (int)(((long)rows + kF8Block - 1) / kF8Block);
  const dim3 tiles((unsigned)RB * KB);
  if (square)
    hipLaunchKernelGGL((f8_encode_tile_kernel<E, true>), tiles, dim3(kTileThreads), 0, st, x, xs,
                       rows, cols, KB, RB, codes, scales, codes_t, scales_t);
  else
    hipLaunchKernelGGL((f8_encode_tile_kernel<E, false>), tiles, dim3(kTileThreads), 0, st, x, xs,
                       rows, cols, KB, RB, codes, scales, codes_t, scales_t);
}
}  // namespace

hipError_t launch_f8_encode(const void* x, bool bf16, int rows, int cols, bool square,
                            unsigned char* codes, unsigned char* scales, unsigned char* codes_t,
                            unsigned char* scales_t, hipStream_t st) {
  const unsigned KB = (unsigned)((cols + kF8Block - 1) / kF8Block);
  if (!square && !codes_t) {
    const unsigned nblocks = (unsigned)rows * KB;
    if (bf16)
      hipLaunchKernelGGL((f8_encode_rows_kernel<__hip_bfloat16>), dim3(row_grid(nblocks)),
                         dim3(256), 0, st, static_cast<const __hip_bfloat16*>(x), nblocks, KB,
                         cols, codes, scales);
    else
      hipLaunchKernelGGL((f8_encode_rows_kernel<float>), dim3(row_grid(nblocks)), dim3(256), 0,
                         st, static_cast<const float*>(x), nblocks, KB, cols, codes, scales);
  } else if (bf16) {
    encode(static_cast<const __hip_bfloat16*>(x), nullptr, rows, cols, square, codes, scales,
           codes_t, scales_t, st);
  } else {
    encode(static_cast<const float*>(x), nullptr, rows, cols, square, codes, scales, codes_t,
           scales_t, st);
  }
  return hipGetLastError();
}

hipError_t launch_f8_repack(const unsigned char* codes, const unsigned char* scales, int rows,
                            int cols, unsigned char* codes_t, unsigned char* scales_t,
                            hipStream_t st) {
  const int KB = (cols + kF8Block - 1) / kF8Block;
  const int RB = (int)(((long)rows + kF8Block - 1) / kF8Block);
  hipLaunchKernelGGL((f8_encode_tile_kernel<unsigned char, false>), dim3((unsigned)RB * KB),
                     dim3(kTileThreads), 0, st, codes, scales, rows, cols, KB, RB,
                     static_cast<unsigned char*>(nullptr), static_cast<unsigned char*>(nullptr),
                     codes_t, scales_t);
  return hipGetLastError();
}

hipError_t launch_f8_decode(const unsigned char* codes, const unsigned char* scales, int rows,
                            int cols, float* out, hipStream_t st) {
  const unsigned KB = (unsigned)((cols + kF8Block - 1) / kF8Block);
  const unsigned nblocks = (unsigned)rows * KB;
  hipLaunchKernelGGL(f8_decode_kernel, dim3(row_grid(nblocks)), dim3(256), 0, st, codes, scales,
                     nblocks, KB, cols, out);
  return hipGetLastError();
}

}  // namespace mhc
