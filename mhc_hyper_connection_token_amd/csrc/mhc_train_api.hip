// mhc_train_api.hip -- the C ABI of the 8-bit blocks and of the site's backward
// passes (declared in include/mhc.h): argument checks and kernel launches.
#include <cmath>

#include "mhc.h"
#include "mhc_checks.h"
#include "mhc_kernels.h"

using mhc::check_ptr;
using mhc::check_shape;
using mhc::overlaps;
using mhc::Span;
using mhc::span;

namespace {

constexpr long kMaxF8Blocks = 1L << 28;  // bounds the launch grids
constexpr int kMaxF8Cols = 1 << 28;

size_t blocks_of(size_t n) { return (n + 127) / 128; }

int check_matrix(int rows, int cols) {
  if (rows < 0 || cols < 1) return MHC_EINVAL;
  if (cols % 4 != 0) return MHC_EALIGN;
  if (cols > kMaxF8Cols || (long)rows * (long)blocks_of(cols) > kMaxF8Blocks)
    return MHC_EUNSUPPORTED;
  return MHC_OK;
}

// The spans of a codes / scales pair; empty ones for a null pointer.
struct Pair {
  Span codes, scales;
};
Pair pair_span(const void* codes, const void* scales, size_t rows, size_t cols, bool square) {
  if (!codes) return Pair{span(nullptr, 0), span(nullptr, 0)};
  const size_t kb = blocks_of(cols);
  return Pair{span(codes, rows * kb * 128),
              span(scales, (square ? blocks_of(rows) : rows) * kb)};
}

// Each of out[] apart from every in[] and from the other outputs.
int check_apart(const Span* out, int no, const Span* in, int ni) {
  for (int i = 0; i < no; ++i) {
    for (int k = 0; k < ni; ++k)
      if (overlaps(out[i], in[k])) return MHC_EOVERLAP;
    for (int k = i + 1; k < no; ++k)
      if (overlaps(out[i], out[k])) return MHC_EOVERLAP;
  }
  return MHC_OK;
}

int check_ptrs(const void* const* ptrs, int n) {
  for (int i = 0; i < n; ++i)
    if (!ptrs[i]) return MHC_EINVAL;
  for (int i = 0; i < n; ++i)
    if (int rc = check_ptr(ptrs[i])) return rc;
  return MHC_OK;
}

// Span of [rows][H] kept in fp32, or as codes where scales are given.
Pair kept_span(const void* p, const unsigned char* scales, size_t rows, size_t H) {
  if (scales) return pair_span(p, scales, rows, H, false);
  return Pair{span(p, rows * H * 4), span(nullptr, 0)};
}

int status(hipError_t e) { return e == hipSuccess ? MHC_OK : MHC_EHIP; }

}  // namespace

extern "C" {

// ---------------------------------------------------------------- 8-bit blocks
int mhc_f8_encode_check(const void* x, int x_type, int rows, int cols, int square,
                        const unsigned char* codes, const unsigned char* scales,
                        const unsigned char* codes_t, const unsigned char* scales_t) {
  int rc = check_matrix(rows, cols);
  if (rc) return rc;
  if (x_type != MHC_F32 && x_type != MHC_BF16) return MHC_EINVAL;
  if (rows == 0) return MHC_OK;
  if (!x || (!codes && !codes_t) || !codes != !scales || !codes_t != !scales_t)
    return MHC_EINVAL;
  const void* ptrs[] = {x, codes, scales, codes_t, scales_t};
  for (const void* p : ptrs)
    if (p && (rc = check_ptr(p))) return rc;
  const Pair o = pair_span(codes, scales, rows, cols, square != 0);
  const Pair t = pair_span(codes_t, scales_t, cols, rows, square != 0);
  const Span out[] = {o.codes, o.scales, t.codes, t.scales};
  const Span in[] = {span(x, (size_t)rows * cols * (x_type == MHC_F32 ? 4 : 2))};
  return check_apart(out, 4, in, 1);
}

int mhc_f8_encode(const void* x, int x_type, int rows, int cols, int square,
                  unsigned char* codes, unsigned char* scales, unsigned char* codes_t,
                  unsigned char* scales_t, void* stream) {
  int rc = mhc_f8_encode_check(x, x_type, rows, cols, square, codes, scales, codes_t, scales_t);
  if (rc || rows == 0) return rc;
  return status(mhc::launch_f8_encode(x, x_type == MHC_BF16, rows, cols, square != 0, codes,
                                      scales, codes_t, scales_t,
                                      static_cast<hipStream_t>(stream)));
}

int mhc_f8_repack(const unsigned char* codes, const unsigned char* scales, int rows, int cols,
                  unsigned char* codes_t, unsigned char* scales_t, void* stream) {
  int rc = check_matrix(rows, cols);
  if (rc || rows == 0) return rc;
  const void* ptrs[] = {codes, scales, codes_t, scales_t};
  if ((rc = check_ptrs(ptrs, 4))) return rc;
  const Pair i = pair_span(codes, scales, rows, cols, false);
  const Pair o = pair_span(codes_t, scales_t, cols, rows, false);
  const Span out[] = {o.codes, o.scales}, in[] = {i.codes, i.scales};
  if ((rc = check_apart(out, 2, in, 2))) return rc;
  return status(mhc::launch_f8_repack(codes, scales, rows, cols, codes_t, scales_t,
                                      static_cast<hipStream_t>(stream)));
}

int mhc_f8_decode(const unsigned char* codes, const unsigned char* scales, int rows, int cols,
                  float* out, void* stream) {
  int rc = check_matrix(rows, cols);
  if (rc || rows == 0) return rc;
  const void* ptrs[] = {codes, scales, out};
  if ((rc = check_ptrs(ptrs, 3))) return rc;
  const Pair i = pair_span(codes, scales, rows, cols, false);
  const Span o[] = {span(out, (size_t)rows * cols * 4)}, in[] = {i.codes, i.scales};
  if ((rc = check_apart(o, 1, in, 2))) return rc;
  return status(mhc::launch_f8_decode(codes, scales, rows, cols, out,
                                      static_cast<hipStream_t>(stream)));
}

int mhc_f8_matmul_check(const unsigned char* a, const unsigned char* a_scales,
                        const unsigned char* b, const unsigned char* b_scales, int b_square,
                        int M, int N, int K, const void* out, int out_type) {
  if (M < 0 || N < 1 || K < 0) return MHC_EINVAL;
  if (out_type != MHC_F32 && out_type != MHC_BF16) return MHC_EINVAL;
  if (N % 4 != 0 || K % 128 != 0) return MHC_EALIGN;
  if (K > kMaxF8Cols || (long)M * N >= mhc::kMaxElems) return MHC_EUNSUPPORTED;
  if (M == 0) return MHC_OK;
  int rc;
  if (!out) return MHC_EINVAL;
  if ((rc = check_ptr(out))) return rc;
  if (K == 0) return MHC_OK;
  const void* ptrs[] = {a, a_scales, b, b_scales};
  if ((rc = check_ptrs(ptrs, 4))) return rc;
  const Pair pa = pair_span(a, a_scales, M, K, false);
  const Pair pb = pair_span(b, b_scales, N, K, b_square != 0);
  const Span o[] = {span(out, (size_t)M * N * (out_type == MHC_F32 ? 4 : 2))};
  const Span in[] = {pa.codes, pa.scales, pb.codes, pb.scales};
  return check_apart(o, 1, in, 4);
}

int mhc_f8_matmul(const unsigned char* a, const unsigned char* a_scales, const unsigned char* b,
                  const unsigned char* b_scales, int b_square, int M, int N, int K, void* out,
                  int out_type, void* stream) {
  int rc = mhc_f8_matmul_check(a, a_scales, b, b_scales, b_square, M, N, K, out, out_type);
  if (rc || M == 0) return rc;
  return status(mhc::launch_f8_matmul(a, a_scales, b, b_scales, b_square != 0, M, N, K, out,
                                      out_type == MHC_BF16, static_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------- backward passes
int mhc_site_post_bwd_check(const float* g, const void* x, const unsigned char* x_scales,
                            const void* f, const unsigned char* f_scales, const float* post,
                            const float* comb, int T, int streams, int hidden, const float* dx,
                            const float* df, const float* dpost, const float* dcomb) {
  int rc = check_shape(T, streams, hidden);
  if (rc || T == 0) return rc;
  const void* ptrs[] = {g, x, f, post, comb, dx, df, dpost, dcomb};
  if ((rc = check_ptrs(ptrs, 9))) return rc;
  if (x_scales && (rc = check_ptr(x_scales))) return rc;
  if (f_scales && (rc = check_ptr(f_scales))) return rc;
  const size_t S = streams, H = hidden, Tz = T;
  const Pair px = kept_span(x, x_scales, Tz * S, H), pf = kept_span(f, f_scales, Tz, H);
  const Span in[] = {span(g, Tz * S * H * 4), px.codes, px.scales, pf.codes, pf.scales,
                     span(post, Tz * S * 4), span(comb, Tz * S * S * 4)};
  const Span out[] = {span(dx, Tz * S * H * 4), span(df, Tz * H * 4), span(dpost, Tz * S * 4),
                      span(dcomb, Tz * S * S * 4)};
  return check_apart(out, 4, in, 7);
}

int mhc_site_post_bwd(const float* g, const void* x, const unsigned char* x_scales,
                      const void* f, const unsigned char* f_scales, const float* post,
                      const float* comb, int T, int streams, int hidden, float* dx, float* df,
                      float* dpost, float* dcomb, void* stream) {
  int rc = mhc_site_post_bwd_check(g, x, x_scales, f, f_scales, post, comb, T, streams, hidden,
                                   dx, df, dpost, dcomb);
  if (rc || T == 0) return rc;
  const mhc::PostBwd p{g, x, x_scales, f, f_scales, post, comb, dx, df, dpost, dcomb};
  return status(mhc::launch_post_bwd(p, T, streams, hidden, static_cast<hipStream_t>(stream)));
}

size_t mhc_site_pre_bwd_work_bytes(int T, int streams, int hidden) {
  if (T < 1 || check_shape(T, streams, hidden) || (long)streams * hidden > (1L << 24)) return 0;
  return mhc::pre_bwd_work_bytes(T, streams, hidden);
}

int mhc_site_pre_bwd_check(const void* x, const unsigned char* x_scales, const float* fn_w,
                           const float* scale, const float* base, int T, int streams, int hidden,
                           int iters, float eps, const float* dy, const float* dpre,
                           const float* dpost, const float* dcomb, const float* dx_in,
                           const float* dx, const float* dfn_w, const float* dscale,
                           const float* dbase, const void* work, size_t work_bytes) {
  int rc = check_shape(T, streams, hidden);
  if (rc) return rc;
  if (iters < 1 || !(eps > 0.0f) || !std::isfinite(eps)) return MHC_EINVAL;
  const size_t S = streams, H = hidden, Tz = T, R = (2 + S) * S;
  if (iters > mhc::pre_bwd_max_iters() || S * H > (1UL << 24)) return MHC_EUNSUPPORTED;
  const void* sums[] = {dfn_w, dscale, dbase};
  if ((rc = check_ptrs(sums, 3))) return rc;
  const Span ds[] = {span(dfn_w, R * S * H * 4), span(dscale, 12), span(dbase, R * 4)};
  if (T == 0) return check_apart(ds, 3, nullptr, 0);
  const void* ptrs[] = {x, fn_w, scale, base, dy, dpost, dcomb, dx, work};
  if ((rc = check_ptrs(ptrs, 9))) return rc;
  const void* maybe[] = {x_scales, dpre, dx_in};
  for (const void* p : maybe)
    if (p && (rc = check_ptr(p))) return rc;
  const size_t need = mhc::pre_bwd_work_bytes(T, streams, hidden);
  if (work_bytes < need) return MHC_EINVAL;
  const Pair px = kept_span(x, x_scales, Tz * S, H);
  const Span in[] = {px.codes, px.scales, span(fn_w, R * S * H * 4), span(scale, 12),
                     span(base, R * 4), span(dy, Tz * H * 4),
                     span(dpre, dpre ? Tz * S * 4 : 0), span(dpost, Tz * S * 4),
                     span(dcomb, Tz * S * S * 4),
                     span(dx_in, dx_in && dx_in != dx ? Tz * S * H * 4 : 0)};
  const Span out[] = {span(dx, Tz * S * H * 4), ds[0], ds[1], ds[2], span(work, need)};
  return check_apart(out, 5, in, 10);
}

int mhc_site_pre_bwd(const void* x, const unsigned char* x_scales, const float* fn_w,
                     const float* scale, const float* base, int T, int streams, int hidden,
                     int iters, float eps, const float* dy, const float* dpre,
                     const float* dpost, const float* dcomb, const float* dx_in, float* dx,
                     float* dfn_w, float* dscale, float* dbase, void* work, size_t work_bytes,
                     void* stream) {
  int rc = mhc_site_pre_bwd_check(x, x_scales, fn_w, scale, base, T, streams, hidden, iters, eps,
                                  dy, dpre, dpost, dcomb, dx_in, dx, dfn_w, dscale, dbase, work,
                                  work_bytes);
  if (rc) return rc;
  const mhc::PreBwd p{x,     x_scales, fn_w,  scale, base, dy,    dpre,
                      dpost, dcomb,    dx_in, dx,    dfn_w, dscale, dbase};
  return status(mhc::launch_pre_bwd(p, T, streams, hidden, iters, eps, work,
                                    static_cast<hipStream_t>(stream)));
}

}  // extern "C"
