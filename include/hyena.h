/*
 * hyena.h -- C ABI of the MI355X (gfx950) Hyena order-N forward library.
 *
 * The operator (Hyena Hierarchy explainer, abeam-guide-lp.pages.dev, section
 * "Hyena 演算子の形"; paper digest, irregular6612.github.io, section
 * "방법 (Method)", framework figure):
 *
 *     z_1 = v,   z_{n+1} = x_n * (h_n conv z_n)  (n = 1..N),   y = z_{N+1}
 *
 * where "*" is the elementwise product and "conv" the causal long
 * convolution c[t] = sum_{k<=t} h[k] z[t-k] over the full length L
 * (homemade-llm "02. 3つの Hyena 演算子", section 4, causal FIR equation).
 * The convolution is evaluated by FFT with zero padding to at least 2L
 * (jisaku.com glossary "Hyena（ハイエナ）", section "計算効率"; gist.science
 * HyenaND summary, section "手法: HyenaND", boundary handling).  The filters
 * are generated implicitly as Window(t) * FFN(t/L, sin, cos) (jisaku.com
 * glossary, section "暗黙的畳み込みフィルタ").
 *
 * Conventions shared by every call:
 *   - Device pointers point to memory of the current HIP device; the caller
 *     allocates and frees all of it.  The library never allocates device
 *     memory and is reentrant; the only state it keeps across calls is the
 *     resident-workgroup count of a kernel, looked up once.
 *   - Every call only enqueues work on `stream` (a hipStream_t; NULL = the
 *     default stream) and returns; results are ready after the stream syncs.
 *     No call allocates, clears memory or synchronises, so the calls can be
 *     captured into a HIP graph and replayed.
 *   - Argument errors are detected on the host before anything is enqueued
 *     and returned as a status; nothing is written in that case.  A failed
 *     kernel launch returns HYENA_ERR_HIP.  Device faults surface at the
 *     caller's next synchronisation.  No C++ exception crosses this ABI.
 *   - Activations v, x_n and y are contiguous [B][D][L] arrays (time
 *     fastest) in the I/O dtype; device pointers must be 16-byte aligned.
 *   - Test hook: the environment variable HYENA_FORCE_PATH ("single" or
 *     "fourstep") and HYENA_FOURSTEP_N1 (a power of two) override the
 *     planner.  Both the spectrum and the forward read them at each call,
 *     so set them identically for both.
 */
#ifndef HYENA_MI355X_H
#define HYENA_MI355X_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  HYENA_OK = 0,
  HYENA_ERR_NULL = 1,        /* a required pointer is NULL                       */
  HYENA_ERR_SHAPE = 2,       /* a size is <= 0 or out of the supported range     */
  HYENA_ERR_UNSUPPORTED = 3, /* a valid request the library does not implement   */
  HYENA_ERR_ALIGN = 4,       /* a device pointer is not 16-byte aligned          */
  HYENA_ERR_WORKSPACE = 5,   /* workspace missing or smaller than required       */
  HYENA_ERR_ALIAS = 6,       /* the output overlaps an input                     */
  HYENA_ERR_HIP = 7          /* a HIP runtime call or kernel launch failed       */
} hyena_status;

typedef enum { HYENA_FP32 = 0, HYENA_BF16 = 1 } hyena_dtype;

typedef enum { HYENA_PATH_SINGLE = 1, HYENA_PATH_FOURSTEP = 2 } hyena_path;

/* Limits of the library. */
#define HYENA_MAX_ORDER 8          /* N in 1..8                                 */
#define HYENA_MAX_L (1LL << 22)    /* L in 1..2^22                              */
#define HYENA_MAX_FREQ 16          /* K in 0..16 (positional features 1+2K)     */

/*
 * Implicit filter generator weights (jisaku.com glossary, section
 * "暗黙的畳み込みフィルタ"; paper digest figure, HyenaFilter node).  All device
 * pointers, fp32, row-major [out][in]:
 *   W1 [H][1+2K], b1 [H]; W2 [H][H], b2 [H]; W3 [N*D][H], b3 [N*D]; alpha [D].
 * b1, b2, b3 may be NULL (zero bias).  H must be one of 8, 16, 32, 64, 128.
 */
typedef struct {
  int32_t D;      /* channels                                   */
  int32_t N;      /* order (number of filters per channel)      */
  int32_t K;      /* sin/cos frequencies; feature dim is 1+2K   */
  int32_t H;      /* FFN hidden width                           */
  const float* W1;
  const float* b1;
  const float* W2;
  const float* b2;
  const float* W3;
  const float* b3;
  const float* alpha;
} hyena_filter_params;

/* Planner result for a sequence length (host only, no GPU needed). */
typedef struct {
  int64_t L;            /* sequence length                                          */
  int64_t M;            /* real FFT length of a zero-padded row, M >= 2L; each row   */
                        /* is transformed as a complex signal of N = M/2 points     */
  int32_t path;         /* hyena_path                                               */
  int32_t n1;           /* four-step: column FFT length, n1*n2 = N (0 single path)  */
  int32_t n2;           /* four-step: row FFT length (0 on the single path)         */
  int32_t reserved;
  int64_t spec_stride;  /* complex64 elements per (n, d) filter in the spectrum     */
} hyena_plan_info;

/* Fill *out with the plan the library uses for length L.
 * Errors: NULL out -> HYENA_ERR_NULL; L outside 1..HYENA_MAX_L -> HYENA_ERR_SHAPE. */
hyena_status hyena_plan(int64_t L, hyena_plan_info* out);

/*
 * hyena_filter_gen: h[n][d][t] = exp(-alpha_d * t / L) * o_{n*D+d}(t),
 *   o(t) = W3 sin(W2 sin(W1 e(t) + b1) + b2) + b3,
 *   e(t) = [t/L, sin(2 pi k t/L) (k=1..K), cos(2 pi k t/L) (k=1..K)].
 * Output h: device fp32 [N][D][L], written completely.
 * Errors: NULL p/h/weights -> NULL; bad D, N, K, H or L -> SHAPE / UNSUPPORTED.
 */
hyena_status hyena_filter_gen(const hyena_filter_params* p, int64_t L, float* h, void* stream);

/* Bytes of the spectrum buffer for (D, N, L): N*D*spec_stride*8. -1 on bad sizes. */
int64_t hyena_spectrum_bytes(int32_t D, int32_t N, int64_t L);

/* Bytes of scratch hyena_filter_spectrum needs (0 on the single path). -1 on bad sizes. */
int64_t hyena_spectrum_workspace_bytes(int32_t D, int32_t N, int64_t L);

/*
 * hyena_filter_spectrum: the DFT of each filter zero-padded to M points
 * (first step of the FFT convolution applied to h; jisaku.com glossary,
 * section "計算効率"), computed once and reused for any batch.
 * In: h, device fp32 [N][D][L].  Out: spec, device, hyena_spectrum_bytes()
 * bytes, in a library-defined order and scale (read it back in natural order
 * with hyena_spectrum_export).  workspace: device scratch of at least
 * hyena_spectrum_workspace_bytes() bytes (may be NULL when that is 0).
 * Errors: NULL -> NULL; sizes -> SHAPE; alignment -> ALIGN; small workspace
 * -> WORKSPACE; spec overlapping h -> ALIAS.
 */
hyena_status hyena_filter_spectrum(const float* h, int32_t D, int32_t N, int64_t L, void* spec,
                                   void* workspace, int64_t workspace_bytes, void* stream);

/* Natural-order copy of the spectrum: out[n][d][k][re,im] = sum_{t<L} h[n][d][t]
 * exp(-2 pi i k t / M) for k = 0..M/2 (device fp32, N*D*(M/2+1)*2 floats).  For tests. */
hyena_status hyena_spectrum_export(const void* spec, int32_t D, int32_t N, int64_t L, float* out,
                                   void* stream);

/* Bytes of scratch hyena_forward needs for this shape (0 on the single path). -1 on bad sizes. */
int64_t hyena_forward_workspace_bytes(int64_t B, int32_t D, int32_t N, int64_t L, hyena_dtype io);

/*
 * hyena_forward: y = z_{N+1} of the order-N recurrence above.
 *   v        device [B][D][L], I/O dtype
 *   x        HOST array of N device pointers, each [B][D][L], I/O dtype
 *   spec     the spectrum hyena_filter_spectrum wrote for the same (D, N, L)
 *   y        device [B][D][L], I/O dtype; must not overlap v, any x_n or spec
 *   io       HYENA_FP32, or HYENA_BF16 (bf16 loads widened exactly, all
 *            arithmetic fp32, y rounded to nearest even; on the four-step
 *            path (long rows, see hyena_plan) with N <= 2 the transform
 *            between its passes is also kept as bf16 pairs, rounded to
 *            nearest even: half the intermediate traffic and workspace)
 *   workspace device scratch of hyena_forward_workspace_bytes() bytes
 * Errors: NULL -> NULL; sizes -> SHAPE; N > HYENA_MAX_ORDER -> UNSUPPORTED;
 * alignment -> ALIGN; workspace -> WORKSPACE; y overlapping an input -> ALIAS.
 */
hyena_status hyena_forward(const void* v, const void* const* x, const void* spec, void* y,
                           int64_t B, int32_t D, int32_t N, int64_t L, hyena_dtype io,
                           void* workspace, int64_t workspace_bytes, void* stream);

/*
 * hyena_forward_static: hyena_forward for callers that cannot allocate device
 * memory -- code under HIP graph capture, tight serving loops, harnesses that
 * forbid allocation.  Same arguments, checks, kernels and results as
 * hyena_forward (linear mode), without the workspace: the four-step
 * intermediate lives in one static device buffer of the library,
 * HYENA_STATIC_SCRATCH_BYTES (128 MiB) per GPU, held from the library's load
 * until the process ends; pass groups are sized to it (at most 256 rows of
 * 512 KiB for L = 64K, 16 rows of 8 MiB for L = 1M).  The buffer needs no
 * clearing: each pass group writes its intermediate before reading it.  The
 * call allocates nothing (no hipMalloc, no hipFree); its first call on a
 * device looks the buffer's address up there, once.  All calls on one GPU
 * share that buffer: calls that may overlap in time on one GPU (different
 * streams, threads) race and must be serialised by the caller, e.g. by
 * issuing them on one stream.
 * Errors as hyena_forward; WORKSPACE if one row's intermediate (8 * M / 2
 * bytes) exceeded the buffer, which no supported L reaches (L = 2^22 needs
 * 32 MiB); HIP if the buffer's address cannot be obtained.
 */
#define HYENA_STATIC_SCRATCH_BYTES (128LL << 20)
hyena_status hyena_forward_static(const void* v, const void* const* x, const void* spec, void* y,
                                  int64_t B, int32_t D, int32_t N, int64_t L, hyena_dtype io, void* stream);

/*
 * Other filter families (homemade-llm "02. 3つの Hyena 演算子", section 3).
 *
 * hyena_filter_gen_li -- Hyena-LI: each filter is a sum of S real
 * exponentials, h[f][t] = sum_s R[f][s] * lambda[f][s]^t for t = 0..L-1
 * (0^0 = 1), f = n*D + d.  R, lambda: device fp32 [N*D][S]; h: device fp32
 * [N][D][L] (feed it to hyena_filter_spectrum like the FFN filters).
 * Errors: NULL -> NULL; D, N, L or S (1..64) out of range -> SHAPE.
 */
hyena_status hyena_filter_gen_li(const float* R, const float* lambda, int32_t D, int32_t N, int32_t S, int64_t L,
                                 float* h, void* stream);

/* hyena_filter_gen_mr -- Hyena-MR: explicit filters of Lh taps damped per
 * channel, h[n][d][t] = hhat[n][d][t] * exp(-alpha[d] * t), t < Lh.  hhat,
 * h: device fp32 [N][D][Lh]; alpha: [D].  Errors as above. */
hyena_status hyena_filter_gen_mr(const float* hhat, const float* alpha, int32_t D, int32_t N, int32_t Lh,
                                 float* h, void* stream);

/* hyena_forward_fir -- the order-N recurrence with explicit short filters
 * (Hyena-SE, or Hyena-MR after hyena_filter_gen_mr): h device fp32
 * [N][D][Lh], Lh in 1..HYENA_MAX_FIR, each convolution evaluated directly
 * (c[t] = sum_{k<Lh, k<=t} h[k] z[t-k]; no FFT, no spectrum, no workspace).
 * Other arguments and errors as hyena_forward. */
#define HYENA_MAX_FIR 256
hyena_status hyena_forward_fir(const void* v, const void* const* x, const float* h, int32_t Lh, void* y,
                               int64_t B, int32_t D, int32_t N, int64_t L, hyena_dtype io, void* stream);

/*
 * Backward of the recurrence (chain rule through the operator above; the
 * pages state no gradient formulas): for a scalar loss with dloss/dy = gy,
 *   gx_n = g_{n+1} * c_n,   gc_n = g_{n+1} * x_n,
 *   g_n[s] = sum_{t>=s} h_n[t-s] gc_n[t]        (adjoint of the causal conv),
 *   gh_n[k] = sum_b sum_{t>=k} gc_n[t] z_n[t-k]  (summed over the batch),
 * with c_n = h_n conv z_n, g_{N+1} = gy and gv = g_1.  The forward
 * intermediates are recomputed from v, x and the spectrum.
 *   gy, gv    device [B][D][L], I/O dtype;   gx  HOST array of N device
 *   pointers [B][D][L], I/O dtype;  gh  device fp32 [N][D][L].
 * L <= 8192 runs in one launch, one workgroup per channel; longer rows (up
 * to the forward's limit) express every convolution of the chain through
 * the forward's four-step causal convolution and a row reversal, with the
 * forward's c_n kept in the workspace (about (N + 1) * B * D * L * 4 bytes, N + 2 rows with B > 1,
 * plus per-row spectra; a spectrum built on the single path is rewritten
 * into the four-step layout there).  Errors as hyena_forward, plus ALIAS for an output overlapping an
 * input or another output.  hyena_backward_ex takes the convolution mode (see the circular mode below):
 * for circular rows (periodic convolution, c[t] = sum_k h[k] z[(t - k) mod L]) the adjoint and the
 * filter gradient are circular correlations; the one-launch kernel serves L <= 16384, longer rows the
 * four-step pipeline with the periodic reversal t -> -t mod L.
 */
int64_t hyena_backward_workspace_bytes(int64_t B, int32_t D, int32_t N, int64_t L, hyena_dtype io);

hyena_status hyena_backward(const void* v, const void* const* x, const void* spec, const void* gy, void* gv,
                            void* const* gx, float* gh, int64_t B, int32_t D, int32_t N, int64_t L,
                            hyena_dtype io, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * The block around the operator (paper digest, irregular6612.github.io,
 * section "방법 (Method)", framework figure: one projection of width (N+1)D
 * yields v and the gates; homemade-llm "02. 3つの Hyena 演算子", section 2:
 * every projected stream is featurised by a short convolution and the result
 * is mapped back by a dense matrix; Hyena Hierarchy explainer section
 * "計算方法": these projections are the D in O(NDL(log L + D))).
 *
 *   Z[b][t][c]  = sum_k u[b][t][k] W_in[c][k] + b_in[c]        c < (N+1)D
 *   S[b][c][t]  = sum_{j<T, j<=t} w_short[c][j] Z[b][t-j][c]    (causal, depthwise)
 *   v = S[:, 0:D],  x_n = S[:, nD:(n+1)D]                       ([B][D][L] each)
 *   y = hyena_forward(v, x, spec)
 *   out[b][t][e] = sum_d W_out[e][d] y[b][d][t] + b_out[e]      ([B][L][D])
 *
 * Device pointers; W_in, W_out and the activations u, out are in the I/O
 * dtype (bf16: fp32 accumulation on the matrix cores, stored values rounded
 * to nearest even), biases and short filters fp32.  b_in / b_out may be NULL.
 */
#define HYENA_MAX_SHORT 16         /* T in 1..16                                */

typedef struct {
  int32_t D;             /* width                                             */
  int32_t N;             /* order                                             */
  int32_t T;             /* short-filter taps                                 */
  int32_t reserved;      /* 0                                                 */
  const void* W_in;      /* [(N+1)*D][D], I/O dtype                           */
  const float* b_in;     /* [(N+1)*D] or NULL                                 */
  const float* w_short;  /* [(N+1)*D][T]                                      */
  const void* W_out;     /* [D][D], I/O dtype                                 */
  const float* b_out;    /* [D] or NULL                                       */
} hyena_block_params;

/* In-projection + short convolution: u [B][L][D] -> streams[0] = v,
 * streams[n] = x_n (HOST array of N+1 device pointers, each [B][D][L], I/O
 * dtype).  Uses W_in, b_in, w_short.  Errors: NULL -> NULL; sizes (incl. T
 * outside 1..HYENA_MAX_SHORT) -> SHAPE; alignment -> ALIGN; a stream
 * overlapping u or W_in -> ALIAS. */
hyena_status hyena_in_projection(const void* u, const hyena_block_params* p, void* const* streams,
                                 int64_t B, int64_t L, hyena_dtype io, void* stream);

/* Output projection: y [B][D][L] -> out [B][L][D] (I/O dtype).  Uses W_out,
 * b_out.  Errors as above; out overlapping y or W_out -> ALIAS. */
hyena_status hyena_out_projection(const void* y, const hyena_block_params* p, void* out, int64_t B,
                                  int64_t L, hyena_dtype io, void* stream);

/* Scratch of hyena_block_forward: v, x_1..x_N and y ([B][D][L] each, I/O
 * dtype, 256-byte aligned) plus the forward's own workspace.  -1 on bad sizes. */
int64_t hyena_block_workspace_bytes(int64_t B, int32_t D, int32_t N, int64_t L, hyena_dtype io);

/* The whole block: u [B][L][D] -> out [B][L][D] with the spectrum of the
 * block's filters (hyena_filter_spectrum for (D, N, L)).  workspace: at least
 * hyena_block_workspace_bytes() bytes.  Errors as the three calls it runs,
 * plus WORKSPACE for a small workspace and ALIAS for out overlapping u. */
hyena_status hyena_block_forward(const void* u, const hyena_block_params* p, const void* spec, void* out,
                                 int64_t B, int64_t L, hyena_dtype io, void* workspace,
                                 int64_t workspace_bytes, void* stream);

/*
 * Circular mode (gist.science HyenaND summary, section "手法: HyenaND",
 * boundary handling: periodic systems use circular convolution, other data
 * the zero-padded linear one).  c[t] = sum_{k<L} h[k] z[(t-k) mod L]: the
 * FFT length is M = L with no padding, so L must be a power of two >= 128
 * (HYENA_ERR_UNSUPPORTED otherwise).  The _ex calls take the mode; the calls
 * without the suffix are HYENA_CONV_LINEAR.  A spectrum is valid only for
 * the mode it was built with.
 */
typedef enum { HYENA_CONV_LINEAR = 0, HYENA_CONV_CIRCULAR = 1 } hyena_conv_mode;

hyena_status hyena_plan_ex(int64_t L, hyena_conv_mode mode, hyena_plan_info* out);
int64_t hyena_spectrum_bytes_ex(int32_t D, int32_t N, int64_t L, hyena_conv_mode mode);
int64_t hyena_spectrum_workspace_bytes_ex(int32_t D, int32_t N, int64_t L, hyena_conv_mode mode);
hyena_status hyena_filter_spectrum_ex(const float* h, int32_t D, int32_t N, int64_t L, hyena_conv_mode mode,
                                      void* spec, void* workspace, int64_t workspace_bytes, void* stream);
hyena_status hyena_spectrum_export_ex(const void* spec, int32_t D, int32_t N, int64_t L, hyena_conv_mode mode,
                                      float* out, void* stream);
int64_t hyena_forward_workspace_bytes_ex(int64_t B, int32_t D, int32_t N, int64_t L, hyena_dtype io,
                                         hyena_conv_mode mode);
hyena_status hyena_forward_ex(const void* v, const void* const* x, const void* spec, void* y, int64_t B,
                              int32_t D, int32_t N, int64_t L, hyena_dtype io, hyena_conv_mode mode,
                              void* workspace, int64_t workspace_bytes, void* stream);
int64_t hyena_backward_workspace_bytes_ex(int64_t B, int32_t D, int32_t N, int64_t L, hyena_dtype io,
                                          hyena_conv_mode mode);
hyena_status hyena_backward_ex(const void* v, const void* const* x, const void* spec, const void* gy, void* gv,
                               void* const* gx, float* gh, int64_t B, int32_t D, int32_t N, int64_t L,
                               hyena_dtype io, hyena_conv_mode mode, void* workspace, int64_t workspace_bytes,
                               void* stream);

/* ------------------------------------------------------------------------
 * Convolutions on 2-D and 3-D grids (gist.science HyenaND summary, "手法:
 * HyenaND": native N-D long convolution evaluated through the N-D FFT, with
 * circular boundaries for periodic systems and every axis zero-padded to
 * twice its size for images and volumes; "実装: nSubQ": the FFT, the
 * spectral product and the inverse FFT fused with the intermediate on chip).
 *
 * Grid of k = ndim in {2, 3} axes with sides dims[0..k-1] (row-major, the
 * last axis contiguous).  The same order-N recurrence as hyena_forward,
 * z_1 = v, z_{n+1} = x_n * (K_n conv z_n), y = z_{N+1}, with
 *   non-circular: c[t] = sum over grid points s of K[t - s] z[s]; the kernel
 *                 holds one value per offset o with |o_a| < dims[a], stored
 *                 row-major with extent 2*dims[a]-1 and index o_a+dims[a]-1
 *                 (a causal kernel is zero at negative offsets);
 *   circular:     c[t] = sum_s K[(t - s) mod dims] z[s]; the kernel has the
 *                 grid's shape.
 * Supported: the FFT grid is a cube of side P, a power of two with, per
 * dimension count, 16 <= P <= 1024 (2-D) or 8 <= P <= 128 (3-D).  Non-circular
 * grids take the smallest such P >= 2*max(dims)-1 (so sides up to 512 in
 * 2-D and 64 in 3-D); circular grids need every side equal to one such P.
 * Other shapes return HYENA_ERR_UNSUPPORTED (a side outside 1..4096: SHAPE).
 * Up to P = 128 (2-D) or 32 (3-D) one workgroup holds a grid for all orders
 * and no workspace is used; larger grids run as passes over the first axis
 * and over rows (2-D) or planes (3-D) through a workspace of
 * hyena_nd_workspace_bytes (at least one grid, P^k/2 complex64 values; a
 * smaller one than returned means more, smaller pass groups).
 *
 * hyena_nd_plan: writes P.
 * hyena_nd_spectrum_bytes: bytes of the spectrum of `rows` kernels (-1 for
 *   an invalid or unsupported shape).  The layout is private.
 * hyena_nd_filter_spectrum: kernel [rows][extent] fp32 (device) -> spec
 *   (device, hyena_nd_spectrum_bytes).  Row r is the kernel n*D + d for the
 *   shared form, (b*N + n)*D + d for per-sample kernels (the summary's
 *   input-dependent kernels, one per sample).
 * hyena_nd_workspace_bytes: workspace for `rows` grids (kernel rows for the
 *   spectrum, B*D for the forward); 0 on the single-pass shapes, -1 for an
 *   invalid or unsupported shape.
 * hyena_nd_forward: v, each x[n] (host array of N device pointers) and y are
 *   [B][D][dims...] in `io`; spec from hyena_nd_filter_spectrum with N*D
 *   rows (per_sample = 0) or B*N*D rows (per_sample = 1).  1 <= N <= 8.
 *   Pointers 16-byte aligned (HYENA_ERR_ALIGN); y and the workspace must not
 *   overlap v, any x[n], spec or each other (HYENA_ERR_ALIAS); a missing or
 *   too small workspace where one is needed is HYENA_ERR_WORKSPACE.  No
 *   allocation; the work is enqueued on `stream`.
 * ---------------------------------------------------------------------- */
hyena_status hyena_nd_plan(int32_t ndim, const int64_t* dims, int32_t circular, int64_t* padded_side);
int64_t hyena_nd_spectrum_bytes(int32_t rows, int32_t ndim, const int64_t* dims, int32_t circular);
int64_t hyena_nd_workspace_bytes(int64_t rows, int32_t ndim, const int64_t* dims, int32_t circular);
hyena_status hyena_nd_filter_spectrum(const float* kernel, int32_t rows, int32_t ndim, const int64_t* dims,
                                      int32_t circular, void* spec, void* workspace, int64_t workspace_bytes,
                                      void* stream);
hyena_status hyena_nd_forward(const void* v, const void* const* x, const void* spec, void* y, int64_t B,
                              int32_t D, int32_t N, int32_t ndim, const int64_t* dims, int32_t circular,
                              int32_t per_sample, hyena_dtype io, void* workspace, int64_t workspace_bytes,
                              void* stream);

/* ------------------------------------------------------------------------
 * The state-space block: operators that stand next to the long convolution
 * in a model of this kind -- a residual addition with a norm, a projection
 * by an 8-bit matrix product, a short causal convolution, and a selective
 * state-space scan, each with the form for single tokens of a serving loop
 * and the backward pass of a training step where it has one.
 *
 * Shared by all of them: the conventions at the top of this file; sizes
 * 1 <= B <= 2^20, 1 <= D <= 2^20, B*D <= 2^30, 1 <= L <= HYENA_MAX_L (SHAPE
 * outside, UNSUPPORTED from 2^24 workgroups
 * of a launch on); activations and
 * carried states 16-byte aligned (ALIGN), fp32 parameter vectors and lengths
 * 4-byte aligned; an output may overlap no input and no other output (ALIAS).
 * Arithmetic is fp32, bf16 values are widened exactly and rounded once, to
 * nearest even, where they are stored.  Sums have a fixed order: equal inputs
 * give equal bits.  A workspace serves one call at a time: calls, or replays
 * of captured ones, that may run at once need one each.
 *
 * lengths (device int32 [B], or NULL): sequence b holds min(max(lengths[b],
 * 0), L) steps.  Whatever stands behind them (NaN included) is not read into
 * any result; outputs of activation shape are zero there, and the state left
 * behind is the one at the sequence's own end.  A sequence of no steps hands
 * its state on, whatever it holds, and adds nothing to a parameter's gradient.
 * ---------------------------------------------------------------------- */

/*
 * Short causal depthwise convolution (the block's short filter by itself):
 *   p[b][c][t] = bias[c] + sum_{j<T} w[c][j] x[b][c][t-j],
 *   y = p, or p / (1 + exp(-p)) with silu,
 * x[b][c][-i] = state[b][c][T-1-i] for i = 1..T-1 (oldest first; zeros where
 * state is NULL).  state_out (NULL: not wanted) is the last T-1 inputs of
 * state and x together, the state of a call that continues the sequence.
 * With T = 1 there is no state: both must be NULL (SHAPE).
 * x, y [B][D][L], state, state_out [B][D][T-1], I/O dtype; w [D][T], bias [D]
 * (or NULL), fp32; T in 1..HYENA_MAX_SHORT.
 */
typedef struct {
  int64_t B;
  int64_t L;
  int32_t D;
  int32_t T;
  int32_t silu;            /* 0 or 1                     */
  int32_t reserved;        /* 0                          */
  const float* w;
  const float* bias;       /* or NULL                    */
  const void* state;       /* or NULL                    */
  const int32_t* lengths;  /* or NULL                    */
} hyena_short_conv_params;

hyena_status hyena_short_conv(const void* x, const hyena_short_conv_params* p, void* y, void* state_out,
                              hyena_dtype io, void* stream);

/* One token for each sequence: x, y [B][D]; state [B][D][T-1] is read and
 * moved on by one in place (NULL with T = 1).  p->L, p->state and p->lengths
 * are not used. */
hyena_status hyena_short_conv_step(const void* x, const hyena_short_conv_params* p, void* state, void* y,
                                   hyena_dtype io, void* stream);

/* Gradients of a loss with dloss/dy = gy and dloss/dstate_out = gstate_out
 * (NULL: zero): gx [B][D][L] and gstate [B][D][T-1] (NULL: not wanted) in the
 * I/O dtype, gw [D][T] and gbias [D] (NULL: not wanted) fp32, summed over
 * batch and time.  workspace: hyena_short_conv_backward_workspace_bytes(). */
int64_t hyena_short_conv_backward_workspace_bytes(int64_t B, int32_t D, int32_t T, int64_t L);
hyena_status hyena_short_conv_backward(const void* x, const hyena_short_conv_params* p, const void* gy,
                                       const void* gstate_out, void* gx, float* gw, float* gbias, void* gstate,
                                       hyena_dtype io, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Selective state-space scan.  Per sequence b, channel d of group g = d /
 * (D/G) and state n:
 *   dt[t]   = softplus(delta[b][d][t] + delta_bias[d])  (or the sum itself),
 *   h[t][n] = exp(dt[t] A[d][n]) h[t-1][n] + dt[t] u[b][d][t] Bm[b][g][n][t],
 *   y[t]    = sum_n Cm[b][g][n][t] h[t][n] + skip[d] u[b][d][t],
 * times z / (1 + exp(-z)) where z is given; h[-1] = state[b][d] (or zeros).
 * state_out (NULL: not wanted) is h at the sequence's end.
 * u, delta, z, y [B][D][L], Bm, Cm [B][G][N][L], I/O dtype; A [D][N], skip,
 * delta_bias [D] (or NULL), state, state_out [B][D][N], fp32.  N in
 * 1..HYENA_MAX_STATE; G divides D.  A is finite and, for a decaying state,
 * not positive: the factors exp(dt A) are multiplied up over 128 steps, which
 * must not overflow.
 * workspace: hyena_selective_scan_workspace_bytes() (0 where the time axis is
 * not split).
 */
#define HYENA_MAX_STATE 64

typedef struct {
  int64_t B;
  int64_t L;
  int32_t D;
  int32_t G;
  int32_t N;
  int32_t softplus;         /* 0 or 1                    */
  const void* u;
  const void* delta;
  const float* A;
  const void* Bm;
  const void* Cm;
  const float* skip;        /* or NULL                   */
  const void* z;            /* or NULL                   */
  const float* delta_bias;  /* or NULL                   */
  const float* state;       /* or NULL                   */
  const int32_t* lengths;   /* or NULL                   */
} hyena_selective_scan_params;

int64_t hyena_selective_scan_workspace_bytes(int64_t B, int32_t D, int32_t N, int64_t L);
hyena_status hyena_selective_scan(const hyena_selective_scan_params* p, void* y, float* state_out, hyena_dtype io,
                                  void* workspace, int64_t workspace_bytes, void* stream);

/* One token for each sequence: u, delta, z, y [B][D], Bm, Cm [B][G][N]; state
 * [B][D][N] fp32 is moved on by one in place.  p->L, p->state and p->lengths
 * are not used; A is 16-byte aligned as well. */
hyena_status hyena_selective_scan_step(const hyena_selective_scan_params* p, float* state, void* y, hyena_dtype io,
                                       void* stream);

/* Gradients of a loss with dloss/dy = gy and dloss/dstate_out = gstate_out
 * (NULL: zero).  gu, gdelta, gz as u; gB, gC as Bm, summed over the group's
 * channels; gA [D][N], gskip, gdelta_bias [D] fp32, summed over batch and
 * time; gstate [B][D][N] fp32.  gz is required with z and NULL without it;
 * gskip, gdelta_bias and gstate may be NULL (not wanted).  The states are
 * computed again from p.  workspace:
 * hyena_selective_scan_backward_workspace_bytes(). */
typedef struct {
  void* gu;
  void* gdelta;
  float* gA;
  void* gB;
  void* gC;
  float* gskip;
  void* gz;
  float* gdelta_bias;
  float* gstate;
} hyena_selective_scan_grads;

int64_t hyena_selective_scan_backward_workspace_bytes(int64_t B, int32_t D, int32_t G, int32_t N, int64_t L);
hyena_status hyena_selective_scan_backward(const hyena_selective_scan_params* p, const void* gy,
                                           const float* gstate_out, const hyena_selective_scan_grads* g,
                                           hyena_dtype io, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Residual addition and root-mean-square norm along D of `rows` rows:
 *   s = x + residual (stored in s_out, rounded to the I/O dtype, and normed
 *   as stored; s = x and s_out NULL where residual is NULL),
 *   y = s / sqrt(mean(s^2) + eps) * weight.
 * x, residual, s_out, y [rows][D] I/O dtype, weight [D] fp32; rows <= 2^31,
 * eps >= 0 (a row of zeros with eps = 0 gives NaN).  The squares are summed in
 * fp32, whose range they must not leave.
 *
 * hyena_rms_norm_quantized stores y in 8 bits instead: q [rows][D] e4m3 codes
 * (OCP, largest value 448) and scales [rows][ceil(D/128)] fp32, one for each
 * 128 values of a row: scale = max|y| / 448 (1 where all are 0, at least
 * 2^-126), q = e4m3(y / scale), rounded to nearest even from the fp32 y.  A
 * block that holds a NaN or an infinity is NaN as a whole.
 *
 * hyena_rms_norm_backward: from s (x, or what s_out holds) and gy the
 * gradient gx of s, and gw [D] fp32 of weight; gs (NULL: zero), the gradient
 * that reaches s past the norm, is added to gx.  The same gx is the gradient
 * of x and of residual.
 */
hyena_status hyena_rms_norm(const void* x, const void* residual, const float* weight, void* y, void* s_out,
                            int64_t rows, int32_t D, float eps, hyena_dtype io, void* stream);
hyena_status hyena_rms_norm_quantized(const void* x, const void* residual, const float* weight, void* q,
                                      float* scales, void* s_out, int64_t rows, int32_t D, float eps,
                                      hyena_dtype io, void* stream);
int64_t hyena_rms_norm_backward_workspace_bytes(int64_t rows, int32_t D);
hyena_status hyena_rms_norm_backward(const void* s, const float* weight, const void* gy, const void* gs, void* gx,
                                     float* gw, int64_t rows, int32_t D, float eps, hyena_dtype io, void* workspace,
                                     int64_t workspace_bytes, void* stream);

/*
 * Matrix product of 8-bit operands with block scales:
 *   out[m][n] = sum_k (q[m][k] scales[m][k/128]) (wq[n][k] wscales[n/128][k/128]) + bias[n]
 * q [M][K], wq [N][K] e4m3, scales [M][ceil(K/128)], wscales [ceil(N/128)]
 * [ceil(K/128)] fp32, bias [N] fp32 or NULL.  Each block of 128 is summed on
 * the matrix cores and scaled into an fp32 sum: in fp32 for an fp32 output and
 * for M <= 64; for a bf16 output of more rows by the 8-bit instructions, which
 * add up each 8 neighbouring products with less than 2^-13 of the largest one
 * lost of each of the others, cut towards zero (an fp32 output avoids it where
 * sums cancel).  A row's and a block's scales are multiplied in fp32, whose
 * normal range that product must not leave.  M = B * L rows of
 * tokens; out is [B][L][N], or with channel_major [B][N][L], the layout of
 * the operators above, in the I/O dtype.  M <= 2^31, whatever B and L are
 * unless channel_major; K a multiple of 16 (UNSUPPORTED
 * otherwise), K, N <= 2^20, out 16-byte aligned.  It serves a product's
 * forward, and the gradient of its left operand with the transposed weight's
 * codes.
 *
 * hyena_quantize: codes and scales as above of x [rows][K] (any K): blocks of
 * block_rows x 128 with block_rows 1 (the left operand) or 128 (the right
 * one; scales [ceil(rows/128)][ceil(K/128)]).
 */
hyena_status hyena_quantize(const void* x, void* q, float* scales, int64_t rows, int32_t K, int32_t block_rows,
                            hyena_dtype io, void* stream);
hyena_status hyena_scaled_matmul(const void* q, const float* scales, const void* wq, const float* wscales,
                                 const float* bias, void* out, int64_t B, int64_t L, int32_t N, int32_t K,
                                 int32_t channel_major, hyena_dtype io, void* stream);

/* ------------------------------------------------------------------------
 * The linear-attention block: the operators of a token mixer that stands in
 * the place of the selective scan -- rotary positions on queries and keys,
 * linear attention with a decay for each head, and a norm of each head's
 * outputs with a gate.  The conventions of the state-space block hold (sizes,
 * lengths, aliases, order of sums, workspaces), with activations token-major:
 * [B][L][heads][D], as a row-major projection leaves them.  Activations that
 * are read may be parts of wider rows: a stride[3] holds the elements between
 * sequences, tokens and heads (0 repeats one; each in 0..2^38; a head's D
 * values are contiguous), and their alignment is that of an element.
 * ---------------------------------------------------------------------- */

/*
 * Linear attention with a decay for each head.  Per sequence b and head h,
 * with lambda = exp(log_decay[h]) (1 where log_decay is NULL):
 *   S[t] = lambda S[t-1] + k[b][t][h] v[b][t][h]^T      (Dk x Dv, fp32),
 *   o[b][t][h] = scale S[t]^T q[b][t][h],
 * S[-1] = state[b][h] (or zeros).  state_out (NULL: not wanted) is S at the
 * sequence's end.  q has Hq heads, k Hk and v Hv, each a divisor of H: head h
 * reads head h / (H/Hq) of q, and so on.  q, k [B][L][..][Dk], v [B][L][Hv][Dv]
 * with strides, o [B][L][H][Dv] contiguous, I/O dtype; log_decay [H], state,
 * state_out [B][H][Dk][Dv], fp32; Dk, Dv in 1..HYENA_MAX_HEAD.
 *
 * Decays: log_decay is not positive (minus infinity: S[t] = k[t] v[t]^T); a
 * positive one grows the state, exp(log_decay t) not to overflow.  It is a
 * constant of the head: the backward forms no gradient of it.
 *
 * Sums and states are fp32.  With bf16 activations the state where q meets
 * it, the weight of a pair of tokens where v does, and the states and their
 * gradients in the backward's products are taken to 2^-17 of themselves: an
 * output is off by its own rounding and at most 2^-17 of the summed sizes of
 * its terms (states are kept, and handed on, in fp32).  A value that is
 * not finite reaches what the formulas say and no earlier token; an infinity
 * may become NaN on its way.
 * workspace: hyena_linear_attention_workspace_bytes() (0 where the time axis
 * is not split; this block's sizes of workspaces are -1 for sizes that the
 * call refuses).
 */
#define HYENA_MAX_HEAD 256

typedef struct {
  int64_t B;
  int64_t L;
  int32_t H;
  int32_t Hq;
  int32_t Hk;
  int32_t Hv;
  int32_t Dk;
  int32_t Dv;
  float scale;              /* finite                    */
  int32_t reserved;         /* 0                         */
  const void* q;
  const void* k;
  const void* v;
  int64_t q_stride[3];
  int64_t k_stride[3];
  int64_t v_stride[3];
  const float* log_decay;   /* or NULL                   */
  const float* state;       /* or NULL                   */
  const int32_t* lengths;   /* or NULL                   */
} hyena_linear_attention_params;

int64_t hyena_linear_attention_workspace_bytes(int64_t B, int64_t L, int32_t H, int32_t Dk, int32_t Dv);
hyena_status hyena_linear_attention(const hyena_linear_attention_params* p, void* o, float* state_out,
                                    hyena_dtype io, void* workspace, int64_t workspace_bytes, void* stream);

/* One token for each sequence: q, k, v [B][..][D] (the strides between tokens
 * move nothing, but are checked as the others are), o [B][H][Dv]; state [B][H][Dk][Dv] is moved on by one in
 * place.  p->L, p->state and p->lengths are not used. */
hyena_status hyena_linear_attention_step(const hyena_linear_attention_params* p, float* state, void* o,
                                         hyena_dtype io, void* stream);

/* Gradients of a loss with dloss/do = go ([B][L][H][Dv], contiguous) and
 * dloss/dstate_out = gstate_out (NULL: zero): gq [B][L][Hq][Dk], gk
 * [B][L][Hk][Dk], gv [B][L][Hv][Dv] contiguous, I/O dtype, summed in fp32
 * over the heads that share one; gstate [B][H][Dk][Dv] fp32 (NULL: not
 * wanted).  workspace: hyena_linear_attention_backward_workspace_bytes(). */
typedef struct {
  void* gq;
  void* gk;
  void* gv;
  float* gstate;
} hyena_linear_attention_grads;

int64_t hyena_linear_attention_backward_workspace_bytes(int64_t B, int64_t L, int32_t H, int32_t Hq, int32_t Hk,
                                                        int32_t Hv, int32_t Dk, int32_t Dv);
hyena_status hyena_linear_attention_backward(const hyena_linear_attention_params* p, const void* go,
                                             const float* gstate_out, const hyena_linear_attention_grads* g,
                                             hyena_dtype io, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Rotary positions: the first R values of each head are turned in pairs by
 * angles position * freq[i], i = 0..R/2-1, the others copied:
 *   (a, b) -> scale (a cos - b sin, a sin + b cos),
 * with (a, b) = values (i, i + R/2), or (2i, 2i + 1) with interleaved;
 * inverse turns the other way, which with the same scale is the gradient.
 * Angles are formed and reduced in double precision, so positions may be far
 * (any int32).  positions[b pos_stride[0] + t pos_stride[1]] (int32, or NULL:
 * t) is shared by the token's heads; freq [R/2] double, 8-byte aligned (radians a step, plain or
 * stretched for a longer context).  R even, 2 <= R <= D <= 2^16.
 * x [B][L][H][D] with strides; out is contiguous, or x itself: turned in
 * place, with x's strides, which then must keep its heads apart (ALIAS).
 */
typedef struct {
  int64_t B;
  int64_t L;
  int32_t H;
  int32_t D;
  int32_t R;
  int32_t interleaved;      /* 0 or 1                    */
  int32_t inverse;          /* 0 or 1                    */
  float scale;              /* finite                    */
  int64_t x_stride[3];
  const double* freq;
  const int32_t* positions; /* or NULL                   */
  int64_t pos_stride[2];    /* sequences, tokens         */
} hyena_rotary_params;

hyena_status hyena_rotary(const hyena_rotary_params* p, const void* x, void* out, hyena_dtype io, void* stream);

/*
 * Norm of groups of a row with an activation: each of the G groups of D/G
 * neighbouring values of a row (a head's output) is normed by itself,
 *   n = (x - mean) / sqrt(var + eps),   m = n weight + bias,
 *   y = m, with silu m / (1 + exp(-m)), or with z m z / (1 + exp(-z));
 * silu and z exclude each other (UNSUPPORTED).  x, z, y [rows][D] I/O dtype,
 * weight, bias [D] fp32 or NULL (1, 0); rows <= 2^31, eps >= 0 (a group of
 * equal values with eps = 0 gives NaN).  var is the mean of (x - mean)^2.
 *
 * hyena_group_norm_backward: from x and gy = dloss/dy the gradients gx, gz
 * (required with z, NULL without it) and gweight, gbias [D] fp32 (NULL: not
 * wanted), summed over the rows; mean and var are computed again.
 */
typedef struct {
  int64_t rows;
  int32_t D;
  int32_t G;
  int32_t silu;             /* 0 or 1                    */
  float eps;
  const void* x;
  const void* z;            /* or NULL                   */
  const float* weight;      /* or NULL                   */
  const float* bias;        /* or NULL                   */
} hyena_group_norm_params;

hyena_status hyena_group_norm(const hyena_group_norm_params* p, void* y, hyena_dtype io, void* stream);
int64_t hyena_group_norm_backward_workspace_bytes(int64_t rows, int32_t D, int32_t G);
hyena_status hyena_group_norm_backward(const hyena_group_norm_params* p, const void* gy, void* gx, float* gweight,
                                       float* gbias, void* gz, hyena_dtype io, void* workspace,
                                       int64_t workspace_bytes, void* stream);

/* Static description of a status code. */
const char* hyena_status_str(hyena_status s);

#ifdef __cplusplus
}
#endif

#endif /* HYENA_MI355X_H */
