/*
 * mhc.h -- C ABI of the MI355X (gfx950) mHC site library (libmhc.so).
 *
 * The library runs the per-token, per-site mHC (manifold-constrained
 * hyper-connections) residual program on one GPU, as two calls:
 *
 *   mhc_site_pre   mixes GEMV + RMS rescale + gates + Sinkhorn + collapse
 *   mhc_site_post  post mix of the branch output back into the streams
 *
 * The operation is the one described on the docs.rs page "memra_engine
 * 0.125.0 src/memra_engine/hyper.rs", module documentation ("ARITHMETIC
 * CONTRACT" and "MEMORY LAYOUT"), with the row order of the mixes given by the
 * doc comment of HyperTopology::rows and the post mix by the doc comment of the
 * page's `post` function.  The gate forms the page leaves open are fixed here:
 * pre = sigmoid, post = 2*sigmoid, comb = Sinkhorn-Knopp of exp(.), one
 * iteration being a row pass then a column pass, each dividing by (sum + eps).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - All tensor pointers are DEVICE pointers to dense arrays, fp32 unless a
 *    call says otherwise, owned by the caller; each must be 16-byte aligned.  Outputs are fully overwritten (no
 *    zeroing needed, prior contents never read).  The library keeps no pointer
 *    after a call returns.
 *  - Layout is token-major: x[T][S][H], element (t,k,i) at (t*S+k)*H+i, so one
 *    token's S*H slab is contiguous.  S = streams, H = hidden, R = (2+S)*S.
 *  - `stream` is a hipStream_t (NULL = the null stream).  Calls only enqueue
 *    work and do not wait for the device, except that a call which must grow
 *    the library scratch (below) allocates device memory with hipMalloc.
 *    Results are ready once the stream reaches the enqueued work.
 *  - Every argument check happens on the host BEFORE any GPU work is enqueued;
 *    a call that returns an error has enqueued nothing.
 *  - Calls on the same device share one library-owned scratch area (partial
 *    sums of the split reduction, the packed weight of the large-batch
 *    kernel).  Two calls enqueued on DIFFERENT streams of the same device must
 *    not run concurrently; calls on one stream are always safe.  The first
 *    call on a device that needs scratch allocates it, and a later call that
 *    needs more allocates a larger area.  No scratch area is ever freed
 *    before the process ends, so HIP graphs captured earlier stay valid.  A
 *    call that would have to grow the scratch while its stream is being
 *    captured returns MHC_ECAPTURE: make one call of the largest size before
 *    capturing (or use a workspace, which never allocates).
 *  - Supported shapes: 1 <= S <= 8, H >= 4 with H % 4 == 0, T >= 0
 *    (T == 0 is a no-op), iters >= 1, eps > 0 and finite, T*S*H < 2^31.
 *  - Numeric domain: finite inputs with |scale*m + base| below about 80, so
 *    that exp() stays finite in fp32; outside it results are unspecified.
 */
#ifndef MHC_H
#define MHC_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes. */
enum {
  MHC_OK = 0,
  MHC_EINVAL = 1,      /* bad size, count, eps, iteration count or NULL pointer */
  MHC_EALIGN = 2,      /* H % 4 != 0 or a pointer not 16-byte aligned            */
  MHC_EUNSUPPORTED = 3,/* valid arguments the library does not handle (S > 8, sizes too large) */
  MHC_EHIP = 4,        /* the HIP runtime reported an error (launch, allocation) */
  MHC_EOVERLAP = 5,    /* an output buffer overlaps an input buffer              */
  MHC_ECAPTURE = 6     /* the scratch would have to grow while the stream is captured */
};

/*
 * mhc_site_pre -- the pre half of one site, for T tokens.
 *
 * Per token t (hyper.rs module doc, arithmetic contract, first four lines):
 *   ss      = sum_i x[t,i]^2 over the whole S*H slab;  rinv = 1/sqrt(ss/(S*H) + eps)
 *   m[r]    = rinv * sum_i fn_w[r,i] * x[t,i]                         r < R
 *   z[r]    = scale[g] * m[r] + base[r]   g = 0 for rows [0,S), 1 for [S,2S),
 *                                         2 for the S*S comb rows [2S,R)
 *   pre[t,c]   = 1/(1+exp(-z[c]))
 *   post[t,k]  = 2/(1+exp(-z[S+k]))
 *   comb[t,j,k]= Sinkhorn of exp(z[2S + j*S + k]) over `iters` rounds
 *                (j = source stream, k = target stream)
 *   y[t,i]     = sum_c pre[t,c] * x[t,c,i]
 *
 * Arguments:
 *   x      [T][S][H]  stream state (read only)
 *   fn_w   [R][S*H]   mixes weight, row-major (read only)
 *   scale  [3]        pre, post and comb scales (read only)
 *   base   [R]        per-row bias (read only)
 *   T, streams (=S), hidden (=H), iters, eps   as above
 *   pre    [T][S]     out
 *   post   [T][S]     out
 *   comb   [T][S][S]  out
 *   y      [T][H]     out (the branch input)
 *   stream            hipStream_t or NULL
 * Outputs must not overlap x, fn_w, scale, base or each other (MHC_EOVERLAP).
 * Returns MHC_OK or an error code above.
 */
int mhc_site_pre(const float* x, const float* fn_w, const float* scale, const float* base,
                 int T, int streams, int hidden, int iters, float eps,
                 float* pre, float* post, float* comb, float* y, void* stream);

/*
 * mhc_site_pre_scratch_bytes -- bytes of library scratch that
 * mhc_site_pre needs for T tokens of this shape: the packed weight where the
 * large-batch kernel runs, else the split reduction's partial sums.  0 for
 * T < 1 or a shape the call rejects.  Host only: no HIP call, safe without a
 * GPU.  A caller that captures HIP graphs can make one eager call at its
 * largest T first, or compare this figure across the shapes it will capture.
 */
size_t mhc_site_pre_scratch_bytes(int T, int streams, int hidden);

/*
 * mhc_site_pre_static -- mhc_site_pre for callers that cannot allocate device
 * memory (code under HIP graph capture, serving loops, harnesses that forbid
 * hipMalloc): the same arguments, checks, kernels and results, but the kernel
 * scratch is a fixed device array inside the library, 16 MiB on each GPU the
 * process uses, held until the process ends.  The call allocates, frees and
 * clears nothing.  A shape whose scratch (mhc_site_pre_scratch_bytes) exceeds
 * 16 MiB returns MHC_EUNSUPPORTED before anything is enqueued (large batches
 * of short slabs can need more; the decode, verify, prefill and wide sites
 * need at most 10.7 MB).  Every call on a GPU shares that GPU's array
 * (the last call's contents stay in it): two calls that overlap in time on one
 * GPU (different streams, or concurrent graph replays) race on it and must be
 * ordered by the caller.
 */
int mhc_site_pre_static(const float* x, const float* fn_w, const float* scale, const float* base,
                        int T, int streams, int hidden, int iters, float eps, float* pre,
                        float* post, float* comb, float* y, void* stream);

/*
 * mhc_site_post -- the post half of one site (hyper.rs, doc comment of `post`):
 *   x_out[t,k,i] = post[t,k] * f[t,i] + sum_j comb[t,j,k] * x[t,j,i]
 * where x is the SITE's input state (the same x given to mhc_site_pre) and f the
 * branch output for the site.
 *
 * Arguments:
 *   x      [T][S][H]  site input state (read only)
 *   f      [T][H]     branch output (read only)
 *   post   [T][S]     post gates (read only)
 *   comb   [T][S][S]  combination matrices, comb[t][j][k] (read only)
 *   T, streams (=S), hidden (=H)
 *   x_out  [T][S][H]  out; must not overlap any input (MHC_EOVERLAP)
 *   stream            hipStream_t or NULL
 * Returns MHC_OK or an error code above.
 */
int mhc_site_post(const float* x, const float* f, const float* post, const float* comb,
                  int T, int streams, int hidden, float* x_out, void* stream);

/*
 * Pre-packed mixes weight.  A site's weight fn_w is a fixed parameter (the
 * hyper.rs page's module doc: the mixes weight of a site, [R][S*H]), while the
 * large-batch pre kernel reads it in its own MFMA operand order, which
 * mhc_site_pre produces by packing fn_w into the library scratch on every
 * call.  A caller that keeps a site's weight can pack it once instead:
 *
 * mhc_packed_weight_bytes(streams, hidden): bytes of the packed form, or 0 for
 *   a shape the large-batch kernel does not serve (then no packed form exists
 *   and mhc_site_pre_packed takes packed == NULL).
 * mhc_pack_weight(fn_w, streams, hidden, packed, stream): writes the packed
 *   form of fn_w [R][S*H] into packed (mhc_packed_weight_bytes bytes, caller
 *   owned, 16-byte aligned, not overlapping fn_w).  MHC_EUNSUPPORTED for a
 *   shape with no packed form; asynchronous on `stream`.
 * mhc_site_pre_packed(x, fn_w, packed, scale, base, ...): mhc_site_pre with
 *   the weight read from `packed` wherever the large-batch kernel runs (fn_w
 *   is still read on the small-batch path).  packed must hold
 *   mhc_pack_weight's output for this fn_w and shape, and must not overlap the
 *   outputs (MHC_EOVERLAP); NULL is MHC_EINVAL for a shape with a packed form.
 *   The results are bit-identical to mhc_site_pre's.  Nothing is written to
 *   the library scratch on the large-batch path.
 */
size_t mhc_packed_weight_bytes(int streams, int hidden);
int mhc_pack_weight(const float* fn_w, int streams, int hidden, float* packed, void* stream);
int mhc_site_pre_packed(const float* x, const float* fn_w, const float* packed,
                        const float* scale, const float* base, int T, int streams, int hidden,
                        int iters, float eps, float* pre, float* post, float* comb, float* y,
                        void* stream);
/* mhc_site_post_pre with the next site's weight read from `packed` wherever the
 * fused kernel runs: same arguments as mhc_site_post_pre plus `packed`, with the
 * conditions of mhc_site_pre_packed (packed must not overlap x_out or the
 * outputs either); bit-identical results. */
int mhc_site_post_pre_packed(const float* x, const float* f, const float* post_in,
                             const float* comb_in, const float* fn_w, const float* packed,
                             const float* scale, const float* base, int T, int streams,
                             int hidden, int iters, float eps, float* x_out, float* pre,
                             float* post, float* comb, float* y, void* stream);

/*
 * mhc_site_pre_exact -- mhc_site_pre with decode-exact batching: every token's
 * pre, post, comb and y are bit-identical to those of a call of mhc_site_pre on
 * that token alone (T = 1), whatever T is and whatever else is in the batch
 * (the hyper.rs page, doc comment of pre_exact: a batched decode row must equal
 * the session's solo step, so the mixes of every row are reduced in the order
 * of a solo token).  Same arguments, checks and return codes as mhc_site_pre.
 * mhc_site_pre itself already has this property for T < 256 when S <= 4 and
 * for T <= 64 when S > 4 (there the two calls run the same kernels); above
 * that this call keeps the solo K-split instead of the faster large-batch
 * schedules, and reads x twice.
 */
int mhc_site_pre_exact(const float* x, const float* fn_w, const float* scale, const float* base,
                       int T, int streams, int hidden, int iters, float eps, float* pre,
                       float* post, float* comb, float* y, void* stream);

/*
 * mhc_site_pre_zq8 -- mhc_site_pre followed by the branch-input epilogue: the
 * RMS norm of y with weight nw and its int8 q8 encoding (the norm-and-q8 step
 * that the fused "v4z" pre kernel of the hc_fused_gate.rs page folds into the
 * pre chain; epsilon 1e-5 there).  Per token t, after y[t,:] as above:
 *   z[t,i] = y[t,i] * nw[i] / sqrt(mean_i(y[t,i]^2) + norm_eps)
 *   per block of 32 consecutive i:  d[t,b] = max|z| / 127,
 *   q[t,i] = z[t,i] * (1/d[t,b]) rounded to nearest, ties away from zero
 *   (an all-zero block gives d = 0 and q = 0).  d and 1/d are IEEE fp32
 *   divisions, so q and d are a function of the fp32 z written.
 *
 * Arguments: as mhc_site_pre, plus
 *   nw        [H]         norm weight (read only)
 *   norm_eps              > 0 and finite
 *   z         [T][H]      out (fp32)
 *   q         [T][H]      out (int8)
 *   d         [T][H/32]   out (fp32)
 * hidden must be a multiple of 32 and at most 8192 (MHC_EALIGN / MHC_EUNSUPPORTED).
 * Outputs must not overlap any input or each other (MHC_EOVERLAP).
 */
int mhc_site_pre_zq8(const float* x, const float* fn_w, const float* scale, const float* base,
                     const float* nw, int T, int streams, int hidden, int iters, float eps,
                     float norm_eps, float* pre, float* post, float* comb, float* y, float* z,
                     signed char* q, float* d, void* stream);

/*
 * mhc_site_post_pre -- the post half of one site followed by the pre half of the
 * next site on its output, the order in which a trunk runs them (hyper.rs page,
 * module doc: per site, attention then MLP, each site's output state is the
 * next site's input).  Equivalent to
 *     mhc_site_post(x, f, post_in, comb_in, ..., x_out);
 *     mhc_site_pre(x_out, fn_w, scale, base, ..., pre, post, comb, y);
 * and bit-identical to that pair.  Where the token-tiled pre kernel serves the
 * shape (S <= 4, T >= 256) one kernel does both and the new state is not read
 * back from memory.  The _zq8 form adds the branch-input epilogue of the second
 * site, as mhc_site_pre_zq8.
 *
 * Arguments: x, f, post_in, comb_in as mhc_site_post (the first site);
 * fn_w, scale, base, iters, eps as mhc_site_pre (the second site); x_out is the
 * first site's output and the second site's input; pre, post, comb, y (and
 * z, q, d) the second site's outputs.  An output that overlaps an input or
 * another output is MHC_EOVERLAP (a walk alternates two sets of gate buffers).
 */
int mhc_site_post_pre(const float* x, const float* f, const float* post_in, const float* comb_in,
                      const float* fn_w, const float* scale, const float* base, int T,
                      int streams, int hidden, int iters, float eps, float* x_out, float* pre,
                      float* post, float* comb, float* y, void* stream);
int mhc_site_post_pre_zq8(const float* x, const float* f, const float* post_in,
                          const float* comb_in, const float* fn_w, const float* scale,
                          const float* base, const float* nw, int T, int streams, int hidden,
                          int iters, float eps, float norm_eps, float* x_out, float* pre,
                          float* post, float* comb, float* y, float* z, signed char* q, float* d,
                          void* stream);
int mhc_site_post_pre_check(const float* x, const float* f, const float* post_in,
                            const float* comb_in, const float* fn_w, const float* scale,
                            const float* base, int T, int streams, int hidden, int iters,
                            float eps, const float* x_out, const float* pre, const float* post,
                            const float* comb, const float* y);

/*
 * Trunk entry and exit (hyper.rs page: doc comments of `expand`,
 * `contract_mean` and `collapse`; the HyperHead loader sizes the head).
 *
 * mhc_expand: x_out[t,k,i] = e[t,i] for every stream k.
 *   e [T][H] (read only) -> x_out [T][S][H]; x_out must not overlap e.
 * mhc_mean: y_out[t,i] = (sum_k x[t,k,i]) / S, streams summed in ascending
 *   order in fp32, then one IEEE division.  x [T][S][H] -> y_out [T][H].
 * mhc_head: the gated-head exit, the pre half of a site with the head's own
 *   weight fn_w [S][S*H], one scale [1] and biases base [S]:
 *     rinv = 1/sqrt(sum_i x[t,i]^2 / (S*H) + eps)         (over the slab)
 *     gates[t,c] = 1/(1+exp(-(scale * rinv * (fn_w[c,:] . x[t,:]) + base[c])))
 *     y[t,i] = sum_c gates[t,c] * x[t,c,i]
 *   gates [T][S] and y [T][H] are outputs; they must not overlap the inputs or
 *   each other.  Uses the library's per-device scratch (as mhc_site_pre).
 * Same size, pointer and return-code conventions as the site calls (hidden % 4
 * == 0, 16-byte aligned pointers, 1 <= streams <= 8, eps > 0 and finite;
 * T = 0 does nothing).  mhc_head_check is the host-side check alone.
 */
int mhc_expand(const float* e, int T, int streams, int hidden, float* x_out, void* stream);
int mhc_mean(const float* x, int T, int streams, int hidden, float* y_out, void* stream);
int mhc_head(const float* x, const float* fn_w, const float* scale, const float* base, int T,
             int streams, int hidden, float eps, float* gates, float* y, void* stream);
int mhc_head_check(const float* x, const float* fn_w, const float* scale, const float* base,
                   int T, int streams, int hidden, float eps, const float* gates,
                   const float* y);

/*
 * Persistent site workspace (the hyper.rs page, doc comment of HyperDecodeWs:
 * one set of buffers per engine, every buffer fully overwritten before it is
 * read, the stream state ping-ponged with one spare slot, so that a decode
 * token makes no allocation).  Here the caller provides the memory and the
 * library never allocates on the workspace path, so a walk over sites can be
 * captured in a HIP graph.
 *
 * mhc_workspace_bytes(max_tokens, streams, hidden) is the device memory a
 * workspace needs (0 for an invalid shape; 1 <= max_tokens <= 8192).
 * mhc_workspace_init carves `mem` (device memory, 256-byte aligned, at least
 * that many bytes, owned by the caller and kept alive while the workspace is
 * used) into the regions below and fills *ws (host memory of the caller); it
 * makes no HIP call and enqueues nothing.  Returns MHC_EINVAL / MHC_EALIGN /
 * MHC_EUNSUPPORTED.
 *
 * The fields are read-only for the caller except that the current stream state
 * state[cur] may be written (e.g. the trunk's entry state) and read at any
 * time.  All outputs have max_tokens rows; a call with T tokens writes the
 * first T.  z, q and d are meaningful only when hidden % 32 == 0.
 *
 * mhc_ws_site_pre / mhc_ws_site_pre_zq8: mhc_site_pre / mhc_site_pre_zq8 on
 * x = state[cur] with the workspace's outputs and its own scratch (so two
 * workspaces may run concurrently on different streams; one workspace must not).
 * mhc_ws_site_post: mhc_site_post from state[cur] with the workspace's post and
 * comb into state[cur ^ 1], then flips cur on the host.  A captured graph bakes
 * the slots in: capture an even number of posts (the two sites of a layer) so
 * that every replay starts and ends in the same slot.  0 <= T <= max_tokens; a
 * call with T = 0 does nothing and does not flip.  Errors as the plain calls.
 */
typedef struct mhc_workspace {
  int max_tokens, streams, hidden;
  int cur;              /* index of the current stream state: 0 or 1 */
  float* state[2];      /* [max_tokens][S][H] each */
  float* pre;           /* [max_tokens][S] */
  float* post;          /* [max_tokens][S] */
  float* comb;          /* [max_tokens][S][S] */
  float* y;             /* [max_tokens][H] */
  float* z;             /* [max_tokens][H] */
  signed char* q;       /* [max_tokens][H] */
  float* d;             /* [max_tokens][ceil(H/32)] */
  void* scratch;        /* kernel scratch: partials / packed weight */
  size_t scratch_bytes; /* bytes of scratch */
} mhc_workspace;

size_t mhc_workspace_bytes(int max_tokens, int streams, int hidden);
size_t mhc_workspace_struct_bytes(void); /* sizeof(mhc_workspace), for bindings */
int mhc_workspace_init(mhc_workspace* ws, void* mem, size_t bytes, int max_tokens, int streams,
                       int hidden);
int mhc_ws_site_pre(mhc_workspace* ws, const float* fn_w, const float* scale, const float* base,
                    int T, int iters, float eps, void* stream);
int mhc_ws_site_pre_zq8(mhc_workspace* ws, const float* fn_w, const float* scale,
                        const float* base, const float* nw, int T, int iters, float eps,
                        float norm_eps, void* stream);
int mhc_ws_site_post(mhc_workspace* ws, const float* f, int T, void* stream);

/*
 * Argument checks alone: return exactly the code mhc_site_pre / mhc_site_post
 * would return for these arguments before enqueuing any work (MHC_OK if the
 * call would go ahead).  They make no HIP call and are safe without a GPU.
 */
int mhc_site_pre_check(const float* x, const float* fn_w, const float* scale, const float* base,
                       int T, int streams, int hidden, int iters, float eps,
                       const float* pre, const float* post, const float* comb, const float* y);
int mhc_site_post_check(const float* x, const float* f, const float* post, const float* comb,
                        int T, int streams, int hidden, const float* x_out);
int mhc_site_pre_zq8_check(const float* x, const float* fn_w, const float* scale,
                           const float* base, const float* nw, int T, int streams, int hidden,
                           int iters, float eps, float norm_eps, const float* pre,
                           const float* post, const float* comb, const float* y, const float* z,
                           const signed char* q, const float* d);

/*
 * 8-bit blocks: activation checkpoints, and the operands of the 8-bit product.
 *
 * An encoded matrix of `rows` x `cols` is
 *   codes  [rows][P]      e4m3 (4 exponent bits of bias 7, 3 mantissa bits, no
 *                         infinity), P = cols rounded up to 128, zero past cols
 *   scales [rows][P/128]  one byte per block of 128 consecutive columns: e + 127,
 *                         the block's values being code * 2^e
 * or, in its SQUARE form, the same codes with one scale per 128 x 128 square:
 *   scales [ceil(rows/128)][P/128].
 * Of a block with largest finite magnitude a, e is the least integer >= -126
 * with a <= 448 * 2^e (0 where a = 0), and code = x * 2^-e rounded to nearest,
 * ties to even; an infinity or a NaN encodes as NaN.  A power of two moves only
 * exponents, so every code has the relative rounding of e4m3 itself, and decoded
 * values are exact in fp32 (but that an entry above 248 * 2^120 = 3.296e38
 * rounds to 2^128, which fp32 holds as an infinity).  The calls take scale bytes
 * as encode writes them (1 .. 247).
 *
 * mhc_f8_encode: x [rows][cols] (MHC_F32 or MHC_BF16) into codes / scales and, in
 *   the same pass, its transpose into codes_t [cols][Pt], scales_t
 *   [cols][Pt/128], Pt = rows rounded up to 128 (blocks along the rows of x; the
 *   form a product needs that sums over rows).  Either pair may be NULL, not
 *   both.  With square != 0 both use one scale per square (scales_t
 *   [P/128][Pt/128]), so codes_t is the exact transpose of codes: the form for
 *   weights.
 * mhc_f8_repack: the transpose of an encoded (not square) matrix, decoded and
 *   encoded again along the other axis: what mhc_f8_encode of the decoded
 *   matrix writes to codes_t, scales_t.
 * mhc_f8_decode: the values, fp32 [rows][cols].
 * mhc_f8_matmul: out[m][n] = sum_k A[m][k] * B[n][k], fp32 sums, out [M][N] of
 *   out_type MHC_F32 or MHC_BF16 (rounded to nearest even).  a, a_scales: M rows
 *   of K codes; b, b_scales: N rows, in the square form if b_square != 0.  K is
 *   a multiple of 128 (the padded width of both; K = 0 gives zeros).  Products
 *   are exact and the k blocks are summed in an order fixed by the shape; an
 *   operand value under 2^-126 may count as zero.
 * Training uses: forward z W^T: b = W.  Input gradient df W: a = df,
 *   b = codes_t of W.  Weight gradient df^T z: a = codes_t of df, b = codes_t of
 *   z (from mhc_f8_repack of the kept codes).
 *
 * cols % 4 == 0 and N % 4 == 0 (MHC_EALIGN), K % 128 == 0 (MHC_EALIGN); at most
 * 2^28 columns, 2^28 blocks in all, M * N < 2^31 and K <= 2^28
 * (MHC_EUNSUPPORTED); rows = 0 or M = 0 does nothing.  Pointers are 16-byte
 * aligned; outputs must not overlap inputs or each other.  No scratch.
 */
enum { MHC_F32 = 0, MHC_BF16 = 1 };

int mhc_f8_encode(const void* x, int x_type, int rows, int cols, int square,
                  unsigned char* codes, unsigned char* scales, unsigned char* codes_t,
                  unsigned char* scales_t, void* stream);
int mhc_f8_repack(const unsigned char* codes, const unsigned char* scales, int rows, int cols,
                  unsigned char* codes_t, unsigned char* scales_t, void* stream);
int mhc_f8_decode(const unsigned char* codes, const unsigned char* scales, int rows, int cols,
                  float* out, void* stream);
int mhc_f8_matmul(const unsigned char* a, const unsigned char* a_scales, const unsigned char* b,
                  const unsigned char* b_scales, int b_square, int M, int N, int K, void* out,
                  int out_type, void* stream);

/*
 * mhc_site_post_bwd -- the gradient of mhc_site_post.  With g = dL/dx_out:
 *   dx[t,j,i]    = sum_k comb[t,j,k] * g[t,k,i]
 *   df[t,i]      = sum_k post[t,k] * g[t,k,i]
 *   dpost[t,k]   = sum_i g[t,k,i] * f[t,i]
 *   dcomb[t,j,k] = sum_i x[t,j,i] * g[t,k,i]
 *
 * Arguments:
 *   g         [T][S][H]  gradient of the site's output state (read only)
 *   x         [T][S][H]  the site's input state: fp32 with x_scales NULL, or the
 *   x_scales             codes and scales of its 8-bit checkpoint (mhc_f8_encode
 *                        of the matrix [T*S][H])
 *   f         [T][H]     the branch output, fp32 with f_scales NULL, or its
 *   f_scales             8-bit checkpoint
 *   post [T][S], comb [T][S][S]  the gates of the forward pass (read only)
 *   dx [T][S][H], df [T][H], dpost [T][S], dcomb [T][S][S]   out
 * dx is the gradient through the post mix alone: pass it to mhc_site_pre_bwd as
 * dx_in, which adds the part that came through the pre half.
 */
int mhc_site_post_bwd(const float* g, const void* x, const unsigned char* x_scales,
                      const void* f, const unsigned char* f_scales, const float* post,
                      const float* comb, int T, int streams, int hidden, float* dx, float* df,
                      float* dpost, float* dcomb, void* stream);

/*
 * mhc_site_pre_bwd -- the gradient of mhc_site_pre, recomputed from its input x
 * (the gates and every Sinkhorn round; nothing else of the forward pass is
 * kept).  With an 8-bit checkpoint of x it is the gradient at the decoded x.
 *
 * Arguments:
 *   x, x_scales          as mhc_site_post_bwd
 *   fn_w, scale, base, T, streams, hidden, iters, eps   as mhc_site_pre;
 *                        iters at most 120 (MHC_EUNSUPPORTED above)
 *   dy    [T][H]         gradient of y (read only)
 *   dpre  [T][S]         further gradient of pre, beside the one through y, or NULL
 *   dpost [T][S], dcomb [T][S][S]   gradients of post and comb (read only)
 *   dx_in [T][S][H]      added to dx, or NULL (read only; may be dx itself)
 *   dx    [T][S][H]      out
 *   dfn_w [R][S*H], dscale [3], dbase [R]   out: sums over the T tokens, zeros
 *                        for T = 0
 *   work, work_bytes     device scratch of the caller, at least
 *                        mhc_site_pre_bwd_work_bytes bytes (MHC_EINVAL if less);
 *                        in use until the call's work is done
 * What comb adds to the gradients of z passes through differences
 * (dc' - sum dc' c') in each of its passes: it is accurate to fp32's rounding of
 * dcomb, not of itself where it is far smaller (comb next to a permutation).
 * Sums over tokens are added in an order fixed by the shape: equal inputs give
 * equal bits.  streams * hidden <= 2^24 (MHC_EUNSUPPORTED above).
 *
 * mhc_site_pre_bwd_work_bytes: 0 for T < 1 or a shape the call rejects.
 */
size_t mhc_site_pre_bwd_work_bytes(int T, int streams, int hidden);
int mhc_site_pre_bwd(const void* x, const unsigned char* x_scales, const float* fn_w,
                     const float* scale, const float* base, int T, int streams, int hidden,
                     int iters, float eps, const float* dy, const float* dpre,
                     const float* dpost, const float* dcomb, const float* dx_in, float* dx,
                     float* dfn_w, float* dscale, float* dbase, void* work, size_t work_bytes,
                     void* stream);

/*
 * The norms around a branch, and their gradients.
 *
 * mhc_branch_norm: the norm before a branch, for branches that take fp32 or bf16
 *   (mhc_site_pre_zq8 has it with int8 codes):
 *     z[t,i] = y[t,i] * nw[i] / sqrt(mean_i y[t,i]^2 + norm_eps)
 * mhc_site_post_norm: mhc_site_post with the norm behind the branch, its gate and the
 *   residual scale in front of the mix:
 *     n[t,i]       = f[t,i] / sqrt(mean_i f[t,i]^2 + norm_eps)
 *     h[t,i]       = alpha * a(gate[t,i]) * n[t,i] * nw[i]
 *     x_out[t,k,i] = post[t,k] * h[t,i] + sum_j comb[t,j,k] * x[t,j,i]
 *   a(v) = v (MHC_GATE_PLAIN), 1/(1+exp(-v)) (MHC_GATE_SIGMOID) or v/(1+exp(-v))
 *   (MHC_GATE_SILU); without a gate, a = 1.
 * mhc_branch_norm_bwd: from dz = dL/dz, with n = y / sqrt(mean y^2 + norm_eps) = y r:
 *     dy[t,i] = r (dz nw - n mean_i(dz nw n));  dnw[i] = sum_t dz n
 * mhc_site_post_norm_bwd: from g = dL/dx_out, with e[t,i] = sum_k post[t,k] g[t,k,i]:
 *     dx[t,j,i] = sum_k comb[t,j,k] g[t,k,i];  dcomb[t,j,k] = sum_i x[t,j,i] g[t,k,i]
 *     dpost[t,k] = sum_i g[t,k,i] h[t,i]
 *     df: as dy above with dz = alpha e a(gate);  dnw[i] = sum_t alpha e a(gate) n
 *     dgate[t,i] = alpha e a'(gate) n nw, summed over t where the gate has one row
 *
 * Arguments:
 *   y [T][H] fp32; in the gradient fp32 with y_scales NULL, or the codes and scales of
 *     its 8-bit checkpoint (mhc_f8_encode)
 *   nw [H]; norm_eps at least 2^-126 and finite (MHC_EINVAL)
 *   z, z_type and dz, dz_type   MHC_F32 or MHC_BF16 (z rounded to nearest even)
 *   x, post, comb, T, streams, hidden   as mhc_site_post; in the gradient x as in
 *     mhc_site_post_bwd
 *   f, f_type   [T][H], MHC_F32 or MHC_BF16; in the gradient, where f_scales is given,
 *     its 8-bit checkpoint (f_type is not read then)
 *   gate, gate_type, gate_rows, gate_act   [gate_rows][H] of MHC_F32 or MHC_BF16, one row
 *     for all tokens (gate_rows = 1) or one a token (gate_rows = T); NULL for none (the
 *     other three are not read then)
 *   alpha   any finite number
 *   dy, dx, df, dpost, dcomb, dnw [H]   out, fp32
 *   dgate   [gate_rows][H] fp32 out, NULL without a gate
 *   work, work_bytes   device scratch of the caller, at least mhc_norm_bwd_work_bytes
 *     bytes (MHC_EINVAL if less); in use until the call's work is done
 * hidden <= 8192 (MHC_EUNSUPPORTED above).  T = 0 does nothing but to zero the sums over
 * tokens.  Sums are fp32, those over tokens added in an order fixed by the shape: equal
 * inputs give equal bits.  A token's squares must stay within fp32.
 *
 * mhc_norm_bwd_work_bytes: 0 for T < 1 or a hidden that the calls reject, and where the
 *   calls need none (a few short rows; work may be NULL then).
 */
enum { MHC_GATE_PLAIN = 0, MHC_GATE_SIGMOID = 1, MHC_GATE_SILU = 2 };

int mhc_branch_norm(const float* y, const float* nw, int T, int hidden, float norm_eps, void* z,
                    int z_type, void* stream);
int mhc_site_post_norm(const float* x, const void* f, int f_type, const float* nw,
                       const void* gate, int gate_type, int gate_rows, int gate_act, float alpha,
                       const float* post, const float* comb, int T, int streams, int hidden,
                       float norm_eps, float* x_out, void* stream);
size_t mhc_norm_bwd_work_bytes(int T, int hidden);
int mhc_branch_norm_bwd(const void* dz, int dz_type, const void* y,
                        const unsigned char* y_scales, const float* nw, int T, int hidden,
                        float norm_eps, float* dy, float* dnw, void* work, size_t work_bytes,
                        void* stream);
int mhc_site_post_norm_bwd(const float* g, const void* x, const unsigned char* x_scales,
                           const void* f, int f_type, const unsigned char* f_scales,
                           const float* nw, const void* gate, int gate_type, int gate_rows,
                           int gate_act, float alpha, const float* post, const float* comb, int T,
                           int streams, int hidden, float norm_eps, float* dx, float* df,
                           float* dpost, float* dcomb, float* dnw, float* dgate, void* work,
                           size_t work_bytes, void* stream);

/*
 * 4-bit groups: the weights of a branch's products for decoding.
 *
 * A weight w [N][K], K a multiple of 32, in groups of G = 32, 64 or 128 consecutive
 * columns of a row, KG = ceil(K/G) of them (the last may be short):
 *   w[n][k] = scale[n][k/G] * (code[n][k] - zero[n][k/G])
 *   scales [N][KG]   MHC_BF16 or MHC_F16
 *   zeros  [N][KG]   one byte, 0 .. 15; NULL: 8 everywhere
 *   codes  [N][K/2]  0 .. 15.  Of the 16 bytes of 32 columns, byte j holds column j in its
 *                    low half and column 16 + j in its high half
 *
 * mhc_q4_encode: w (MHC_F32 or MHC_BF16) into codes and bf16 scales.  With zeros NULL
 *   scale = max|w| / 7 of the group and the codes are 1 .. 15; else, with lo = min(w, 0)
 *   and hi = max(w, 0), scale = hi/15 - lo/15 and zero = -lo/scale, rounded.  The scale
 *   is rounded to bf16 first (at least 2^-126), then code = w/scale + zero, each
 *   rounded to nearest even, within the codes' range: what is off by rounding is at most
 *   half a scale (but at a group's ends, where a scale rounded down may cut off up to
 *   2^-9 of the range).  Infinities and NaN set no scale; an infinity takes the code at
 *   its end of the range, a NaN the zero point.
 * mhc_q4_decode: the values, fp32 [N][K] (exact).
 * mhc_q4_matmul: out[m][n] = sum_k a[m][k] * w[n][k], out [M][N] of out_type MHC_F32 or
 *   MHC_BF16 (rounded to nearest even).
 *   a [M][K], a_type   MHC_F32 or MHC_BF16 with a_scales NULL; or MHC_I8 with a_scales
 *     [M][K/32], value a * a_scales: the q and d of mhc_site_pre_zq8
 *   Products with the codes are exact and summed in fp32 in an order fixed by the shape
 *   (int8: exactly within 32 columns for M <= 16, else of a * a_scales rounded to fp32); the
 *   scale is applied to a group's sum, so that 15 times the sum of |a| over a group must
 *   stay within fp32 (it does for |a| up to 2^117), also where the scale is small.  A value
 *   of a, or a part of one in fp32, that is under 2^-126 may count as zero.  A row of a with
 *   an infinity or a NaN gives a row that is not finite; other rows do not see it.
 *
 * N <= 2^24, K <= 2^20, M <= 2^20, M * N < 2^31 (MHC_EUNSUPPORTED); K % 32 == 0
 * (MHC_EALIGN); M = 0 does nothing.  Pointers are 16-byte aligned; outputs must not
 * overlap inputs or each other.  No scratch.
 */
enum { MHC_F16 = 2, MHC_I8 = 3 }; /* beside MHC_F32 and MHC_BF16 */

int mhc_q4_encode(const void* w, int w_type, int N, int K, int group, unsigned char* codes,
                  void* scales, unsigned char* zeros, void* stream);
int mhc_q4_decode(const unsigned char* codes, const void* scales, int scale_type,
                  const unsigned char* zeros, int N, int K, int group, float* out,
                  void* stream);
int mhc_q4_matmul(const void* a, int a_type, const float* a_scales, const unsigned char* codes,
                  const void* scales, int scale_type, const unsigned char* zeros, int M, int N,
                  int K, int group, void* out, int out_type, void* stream);

/* The argument checks of the calls above alone (no HIP call). */
int mhc_f8_encode_check(const void* x, int x_type, int rows, int cols, int square,
                        const unsigned char* codes, const unsigned char* scales,
                        const unsigned char* codes_t, const unsigned char* scales_t);
int mhc_f8_matmul_check(const unsigned char* a, const unsigned char* a_scales,
                        const unsigned char* b, const unsigned char* b_scales, int b_square,
                        int M, int N, int K, const void* out, int out_type);
int mhc_site_post_bwd_check(const float* g, const void* x, const unsigned char* x_scales,
                            const void* f, const unsigned char* f_scales, const float* post,
                            const float* comb, int T, int streams, int hidden, const float* dx,
                            const float* df, const float* dpost, const float* dcomb);
int mhc_site_pre_bwd_check(const void* x, const unsigned char* x_scales, const float* fn_w,
                           const float* scale, const float* base, int T, int streams, int hidden,
                           int iters, float eps, const float* dy, const float* dpre,
                           const float* dpost, const float* dcomb, const float* dx_in,
                           const float* dx, const float* dfn_w, const float* dscale,
                           const float* dbase, const void* work, size_t work_bytes);

int mhc_branch_norm_check(const float* y, const float* nw, int T, int hidden, float norm_eps,
                          const void* z, int z_type);
int mhc_branch_norm_bwd_check(const void* dz, int dz_type, const void* y,
                              const unsigned char* y_scales, const float* nw, int T, int hidden,
                              float norm_eps, const float* dy, const float* dnw,
                              const void* work, size_t work_bytes);
int mhc_site_post_norm_check(const float* x, const void* f, int f_type, const float* nw,
                             const void* gate, int gate_type, int gate_rows, int gate_act,
                             float alpha, const float* post, const float* comb, int T,
                             int streams, int hidden, float norm_eps, const float* x_out);
int mhc_site_post_norm_bwd_check(const float* g, const void* x, const unsigned char* x_scales,
                                 const void* f, int f_type, const unsigned char* f_scales,
                                 const float* nw, const void* gate, int gate_type, int gate_rows,
                                 int gate_act, float alpha, const float* post, const float* comb,
                                 int T, int streams, int hidden, float norm_eps, const float* dx,
                                 const float* df, const float* dpost, const float* dcomb,
                                 const float* dnw, const float* dgate, const void* work,
                                 size_t work_bytes);
int mhc_q4_encode_check(const void* w, int w_type, int N, int K, int group,
                        const unsigned char* codes, const void* scales,
                        const unsigned char* zeros);
int mhc_q4_matmul_check(const void* a, int a_type, const float* a_scales,
                        const unsigned char* codes, const void* scales, int scale_type,
                        const unsigned char* zeros, int M, int N, int K, int group,
                        const void* out, int out_type);

/* Static text for a return code (never NULL). */
const char* mhc_status_string(int status);

/*
 * Bandwidth probe (a measurement aid, not part of the site program).  The
 * hc_fused_gate.rs page's gate carries a bandwidth probe of its own, a pure
 * streamer reporting read and read + write GB/s; this one gives the same two
 * rates on this part, and the site kernels' rates are read against them.
 *
 * mhc_bandwidth_probe: with copy != 0, copies `bytes` from src to dst (both
 *   `bytes` long, not overlapping); with copy == 0, reads `bytes` from src and
 *   writes mhc_probe_sink_floats(bytes) block sums (one per 4 KiB of src) to
 *   dst.  Streaming 16-byte loads (and stores), one quad per thread.
 *   bytes % 16 == 0 and 16-byte aligned pointers (MHC_EALIGN otherwise); NULL
 *   pointers are MHC_EINVAL; overlapping buffers MHC_EOVERLAP; more than 2^43
 *   bytes MHC_EUNSUPPORTED; bytes == 0 does nothing.  Asynchronous on
 *   `stream` like the site calls.
 */
size_t mhc_probe_sink_floats(size_t bytes);
int mhc_bandwidth_probe(const float* src, float* dst, size_t bytes, int copy, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MHC_H */
