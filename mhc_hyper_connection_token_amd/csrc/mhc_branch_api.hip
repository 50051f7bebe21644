// mhc_branch_api.hip -- the C ABI of the norms around a branch, their gradients and the
// 4-bit groups (declared in include/mhc.h): argument checks and kernel launches.
#include <cfloat>
#include <cmath>

#include "mhc.h"
#include "mhc_checks.h"
#include "mhc_kernels.h"

using mhc::check_apart;
using mhc::check_ptr;
using mhc::check_ptrs;
using mhc::check_shape;
using mhc::kept_span;
using mhc::Pair;
using mhc::Span;
using mhc::span;

namespace {

constexpr int kMaxNormHidden = 8192;  // a row that a block's registers hold
constexpr int kMaxQ4Rows = 1 << 24;    // these three bound the launch grids
constexpr int kMaxQ4Cols = 1 << 20;
constexpr int kMaxQ4Tokens = 1 << 20;

int status(hipError_t e) { return e == hipSuccess ? MHC_OK : MHC_EHIP; }

bool real_type(int t) { return t == MHC_F32 || t == MHC_BF16; }
size_t type_size(int t) { return t == MHC_F32 ? 4 : 2; }

int check_norm(int T, int streams, int hidden, float eps) {
  if (int rc = check_shape(T, streams, hidden)) return rc;
  // (the reciprocal root takes numbers under the smallest normal one for zero)
  if (!(eps >= FLT_MIN) || !std::isfinite(eps)) return MHC_EINVAL;
  return hidden > kMaxNormHidden ? MHC_EUNSUPPORTED : MHC_OK;
}

// A gate's type, rows and activation, where there is one.
int check_gate(const void* gate, int type, int rows, int act, float alpha, int T) {
  if (!std::isfinite(alpha)) return MHC_EINVAL;
  if (!gate) return MHC_OK;
  if (!real_type(type) || act < MHC_GATE_PLAIN || act > MHC_GATE_SILU) return MHC_EINVAL;
  if (rows != 1 && rows != T) return MHC_EINVAL;
  return check_ptr(gate);
}

int check_q4(int N, int K, int group) {
  if (N < 1 || K < 1 || (group != 32 && group != 64 && group != 128)) return MHC_EINVAL;
  if (K % 32 != 0) return MHC_EALIGN;
  return N > kMaxQ4Rows || K > kMaxQ4Cols ? MHC_EUNSUPPORTED : MHC_OK;
}

struct Q4Spans {
  Span codes, scales, zeros;
};
Q4Spans q4_spans(const void* codes, const void* scales, const void* zeros, size_t N, size_t K,
                 size_t group) {
  const size_t groups = N * ((K + group - 1) / group);
  return Q4Spans{span(codes, N * (K / 2)), span(scales, groups * 2),
                 span(zeros, zeros ? groups : 0)};
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------- norm before a branch
int mhc_branch_norm_check(const float* y, const float* nw, int T, int hidden, float norm_eps,
                          const void* z, int z_type) {
  int rc = check_norm(T, 1, hidden, norm_eps);
  if (rc) return rc;
  if (!real_type(z_type)) return MHC_EINVAL;
  if (T == 0) return MHC_OK;
  const void* ptrs[] = {y, nw, z};
  if ((rc = check_ptrs(ptrs, 3))) return rc;
  const size_t n = (size_t)T * hidden;
  const Span in[] = {span(y, n * 4), span(nw, (size_t)hidden * 4)};
  const Span out[] = {span(z, n * type_size(z_type))};
  return check_apart(out, 1, in, 2);
}

int mhc_branch_norm(const float* y, const float* nw, int T, int hidden, float norm_eps, void* z,
                    int z_type, void* stream) {
  int rc = mhc_branch_norm_check(y, nw, T, hidden, norm_eps, z, z_type);
  if (rc || T == 0) return rc;
  return status(mhc::launch_branch_norm(y, nw, T, hidden, norm_eps, z, z_type == MHC_BF16,
                                        static_cast<hipStream_t>(stream)));
}

size_t mhc_norm_bwd_work_bytes(int T, int hidden) {
  if (T < 1 || check_norm(T, 1, hidden, 1.0f)) return 0;
  return mhc::norm_bwd_work_bytes(T, hidden, 2);
}

int mhc_branch_norm_bwd_check(const void* dz, int dz_type, const void* y,
                              const unsigned char* y_scales, const float* nw, int T, int hidden,
                              float norm_eps, const float* dy, const float* dnw,
                              const void* work, size_t work_bytes) {
  int rc = check_norm(T, 1, hidden, norm_eps);
  if (rc) return rc;
  if (!real_type(dz_type) || !dnw) return MHC_EINVAL;
  if ((rc = check_ptr(dnw))) return rc;
  if (T == 0) return MHC_OK;
  const size_t H = hidden, n = T * H, need = mhc_norm_bwd_work_bytes(T, hidden);
  const void* ptrs[] = {dz, y, nw, dy, work};
  if ((rc = check_ptrs(ptrs, need ? 5 : 4))) return rc;
  if (y_scales && (rc = check_ptr(y_scales))) return rc;
  if (work_bytes < need) return MHC_EINVAL;
  const Pair py = kept_span(y, y_scales, T, H);
  const Span in[] = {span(dz, n * type_size(dz_type)), py.codes, py.scales, span(nw, H * 4)};
  const Span out[] = {span(dy, n * 4), span(dnw, H * 4), span(work, need)};
  return check_apart(out, 3, in, 4);
}

int mhc_branch_norm_bwd(const void* dz, int dz_type, const void* y,
                        const unsigned char* y_scales, const float* nw, int T, int hidden,
                        float norm_eps, float* dy, float* dnw, void* work, size_t work_bytes,
                        void* stream) {
  int rc = mhc_branch_norm_bwd_check(dz, dz_type, y, y_scales, nw, T, hidden, norm_eps, dy, dnw,
                                     work, work_bytes);
  if (rc) return rc;
  const mhc::NormBwd p{dz, y, y_scales, nw, dy, dnw, dz_type == MHC_BF16};
  return status(mhc::launch_norm_bwd(p, T, hidden, norm_eps, work,
                                     static_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------- norm behind a branch
int mhc_site_post_norm_check(const float* x, const void* f, int f_type, const float* nw,
                             const void* gate, int gate_type, int gate_rows, int gate_act,
                             float alpha, const float* post, const float* comb, int T,
                             int streams, int hidden, float norm_eps, const float* x_out) {
  int rc = check_norm(T, streams, hidden, norm_eps);
  if (rc) return rc;
  if (!real_type(f_type)) return MHC_EINVAL;
  if ((rc = check_gate(gate, gate_type, gate_rows, gate_act, alpha, T))) return rc;
  if (T == 0) return MHC_OK;
  const void* ptrs[] = {x, f, nw, post, comb, x_out};
  if ((rc = check_ptrs(ptrs, 6))) return rc;
  const size_t S = streams, H = hidden, Tz = T;
  const Span in[] = {span(x, Tz * S * H * 4), span(f, Tz * H * type_size(f_type)),
                     span(nw, H * 4), span(gate, gate ? gate_rows * H * type_size(gate_type) : 0),
                     span(post, Tz * S * 4), span(comb, Tz * S * S * 4)};
  const Span out[] = {span(x_out, Tz * S * H * 4)};
  return check_apart(out, 1, in, 6);
}

int mhc_site_post_norm(const float* x, const void* f, int f_type, const float* nw,
                       const void* gate, int gate_type, int gate_rows, int gate_act, float alpha,
                       const float* post, const float* comb, int T, int streams, int hidden,
                       float norm_eps, float* x_out, void* stream) {
  int rc = mhc_site_post_norm_check(x, f, f_type, nw, gate, gate_type, gate_rows, gate_act, alpha,
                                    post, comb, T, streams, hidden, norm_eps, x_out);
  if (rc || T == 0) return rc;
  const mhc::PostNorm p{x,     f,    nw,    gate, post, comb, x_out, alpha, f_type == MHC_BF16,
                        gate_type == MHC_BF16, gate_rows != 1, gate_act};
  return status(mhc::launch_post_norm(p, T, streams, hidden, norm_eps,
                                      static_cast<hipStream_t>(stream)));
}

int mhc_site_post_norm_bwd_check(const float* g, const void* x, const unsigned char* x_scales,
                                 const void* f, int f_type, const unsigned char* f_scales,
                                 const float* nw, const void* gate, int gate_type, int gate_rows,
                                 int gate_act, float alpha, const float* post, const float* comb,
                                 int T, int streams, int hidden, float norm_eps, const float* dx,
                                 const float* df, const float* dpost, const float* dcomb,
                                 const float* dnw, const float* dgate, const void* work,
                                 size_t work_bytes) {
  int rc = check_norm(T, streams, hidden, norm_eps);
  if (rc) return rc;
  if (!f_scales && !real_type(f_type)) return MHC_EINVAL;
  if ((rc = check_gate(gate, gate_type, gate_rows, gate_act, alpha, T))) return rc;
  const size_t S = streams, H = hidden, Tz = T;
  // dgate has the gate's rows: with one row it is a sum over the tokens, also over none
  const bool row = gate && gate_rows == 1;
  if (!dnw || !gate != !dgate) {
    if (!dnw || T > 0 || row) return MHC_EINVAL;
  }
  if ((rc = check_ptr(dnw)) || (dgate && (rc = check_ptr(dgate)))) return rc;
  const Span sums[] = {span(dnw, H * 4), span(dgate, dgate ? gate_rows * H * 4 : 0)};
  if (T == 0) return check_apart(sums, 2, nullptr, 0);
  const size_t need = mhc_norm_bwd_work_bytes(T, hidden);
  const void* ptrs[] = {g, x, f, nw, post, comb, dx, df, dpost, dcomb, work};
  if ((rc = check_ptrs(ptrs, need ? 11 : 10))) return rc;
  if (x_scales && (rc = check_ptr(x_scales))) return rc;
  if (f_scales && (rc = check_ptr(f_scales))) return rc;
  if (work_bytes < need) return MHC_EINVAL;
  const Pair px = kept_span(x, x_scales, Tz * S, H), pf = kept_span(f, f_scales, Tz, H);
  const Span in[] = {span(g, Tz * S * H * 4), px.codes, px.scales,
                     f_scales ? pf.codes : span(f, Tz * H * type_size(f_type)), pf.scales,
                     span(nw, H * 4), span(gate, gate ? gate_rows * H * type_size(gate_type) : 0),
                     span(post, Tz * S * 4), span(comb, Tz * S * S * 4)};
  const Span out[] = {span(dx, Tz * S * H * 4), span(df, Tz * H * 4), span(dpost, Tz * S * 4),
                      span(dcomb, Tz * S * S * 4), sums[0], sums[1], span(work, need)};
  return check_apart(out, 7, in, 9);
}

int mhc_site_post_norm_bwd(const float* g, const void* x, const unsigned char* x_scales,
                           const void* f, int f_type, const unsigned char* f_scales,
                           const float* nw, const void* gate, int gate_type, int gate_rows,
                           int gate_act, float alpha, const float* post, const float* comb, int T,
                           int streams, int hidden, float norm_eps, float* dx, float* df,
                           float* dpost, float* dcomb, float* dnw, float* dgate, void* work,
                           size_t work_bytes, void* stream) {
  int rc = mhc_site_post_norm_bwd_check(g, x, x_scales, f, f_type, f_scales, nw, gate, gate_type,
                                        gate_rows, gate_act, alpha, post, comb, T, streams,
                                        hidden, norm_eps, dx, df, dpost, dcomb, dnw, dgate, work,
                                        work_bytes);
  if (rc) return rc;
  const mhc::PostNormBwd p{g,    x,     x_scales, f,     f_scales, nw,
                           gate, post,  comb,     dx,    df,       dpost,
                           dcomb, dnw,  dgate,    alpha, f_scales ? 2 : f_type == MHC_BF16,
                           gate_type == MHC_BF16, gate_rows != 1, gate_act};
  return status(mhc::launch_post_norm_bwd(p, T, streams, hidden, norm_eps, work,
                                          static_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------- 4-bit groups
int mhc_q4_encode_check(const void* w, int w_type, int N, int K, int group,
                        const unsigned char* codes, const void* scales,
                        const unsigned char* zeros) {
  int rc = check_q4(N, K, group);
  if (rc) return rc;
  if (!real_type(w_type)) return MHC_EINVAL;
  const void* ptrs[] = {w, codes, scales};
  if ((rc = check_ptrs(ptrs, 3))) return rc;
  if (zeros && (rc = check_ptr(zeros))) return rc;
  const Q4Spans q = q4_spans(codes, scales, zeros, N, K, group);
  const Span in[] = {span(w, (size_t)N * K * type_size(w_type))};
  const Span out[] = {q.codes, q.scales, q.zeros};
  return check_apart(out, 3, in, 1);
}

int mhc_q4_encode(const void* w, int w_type, int N, int K, int group, unsigned char* codes,
                  void* scales, unsigned char* zeros, void* stream) {
  int rc = mhc_q4_encode_check(w, w_type, N, K, group, codes, scales, zeros);
  if (rc) return rc;
  return status(mhc::launch_q4_encode(w, w_type == MHC_BF16, N, K, group, codes, scales, zeros,
                                      static_cast<hipStream_t>(stream)));
}

int mhc_q4_decode(const unsigned char* codes, const void* scales, int scale_type,
                  const unsigned char* zeros, int N, int K, int group, float* out,
                  void* stream) {
  int rc = check_q4(N, K, group);
  if (rc) return rc;
  if (scale_type != MHC_BF16 && scale_type != MHC_F16) return MHC_EINVAL;
  const void* ptrs[] = {codes, scales, out};
  if ((rc = check_ptrs(ptrs, 3))) return rc;
  if (zeros && (rc = check_ptr(zeros))) return rc;
  const Q4Spans q = q4_spans(codes, scales, zeros, N, K, group);
  const Span o[] = {span(out, (size_t)N * K * 4)}, in[] = {q.codes, q.scales, q.zeros};
  if ((rc = check_apart(o, 1, in, 3))) return rc;
  return status(mhc::launch_q4_decode(codes, scales, scale_type == MHC_F16, zeros, N, K, group,
                                      out, static_cast<hipStream_t>(stream)));
}

int mhc_q4_matmul_check(const void* a, int a_type, const float* a_scales,
                        const unsigned char* codes, const void* scales, int scale_type,
                        const unsigned char* zeros, int M, int N, int K, int group,
                        const void* out, int out_type) {
  int rc;
  if (M < 0) return MHC_EINVAL;
  if ((rc = check_q4(N, K, group))) return rc;
  if ((!real_type(a_type) && a_type != MHC_I8) || !real_type(out_type) ||
      (scale_type != MHC_BF16 && scale_type != MHC_F16))
    return MHC_EINVAL;
  if (M > kMaxQ4Tokens || (long)M * N >= mhc::kMaxElems) return MHC_EUNSUPPORTED;
  if (M == 0) return MHC_OK;
  const void* ptrs[] = {a, codes, scales, out};
  if ((rc = check_ptrs(ptrs, 4))) return rc;
  if ((a_type == MHC_I8) != (a_scales != nullptr)) return MHC_EINVAL;
  if (a_scales && (rc = check_ptr(a_scales))) return rc;
  if (zeros && (rc = check_ptr(zeros))) return rc;
  const Q4Spans q = q4_spans(codes, scales, zeros, N, K, group);
  const size_t Mz = M, Kz = K;
  const Span in[] = {span(a, Mz * Kz * (a_type == MHC_I8 ? 1 : type_size(a_type))),
                     span(a_scales, a_scales ? Mz * (Kz / 32) * 4 : 0), q.codes, q.scales,
                     q.zeros};
  const Span o[] = {span(out, Mz * N * type_size(out_type))};
  return check_apart(o, 1, in, 5);
}

int mhc_q4_matmul(const void* a, int a_type, const float* a_scales, const unsigned char* codes,
                  const void* scales, int scale_type, const unsigned char* zeros, int M, int N,
                  int K, int group, void* out, int out_type, void* stream) {
  int rc = mhc_q4_matmul_check(a, a_type, a_scales, codes, scales, scale_type, zeros, M, N, K,
                               group, out, out_type);
  if (rc || M == 0) return rc;
  const mhc::Q4Matmul q{a,   a_scales, codes, scales, zeros,
                        out, a_type == MHC_I8 ? 2 : a_type == MHC_BF16, scale_type == MHC_F16,
                        out_type == MHC_BF16};
  return status(mhc::launch_q4_matmul(q, M, N, K, group, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
