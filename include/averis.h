/*
 * libaveris -- C ABI of the Averis mean-residual split FP4 linear on MI355X
 * (gfx950): split-quant, plain quant, and the quantized GEMMs of the forward
 * and dgrad passes, plus the vanilla-FP4 comparison arm.
 *
 * The method (from "The Curse and Blessing of Mean Bias in FP4-Quantized LLM
 * Training", as reviewed on the "Lighthouse" blog, §2.1-§2.2, and summarised
 * in the paper's arXiv abstract and the gist.science technical summary §2):
 *   mu_X   = (1/l) 1^T X                       column mean over the l tokens
 *   X_R    = X - 1 mu_X^T                      residual (unquantized mean)
 *   Y      = 1 (Q4(mu_X) Q4(W)) + Q4(X_R) Q4(W)          forward
 *   dX     = 1 (Q4(mu_D) Q4(W)^T) + Q4(D_R) Q4(W)^T      dgrad (D = dL/dY)
 * Q4 is NVFP4-style E2M1 with stochastic rounding by default (Lighthouse
 * §3.1; two-level "hierarchical" microscaling per "Dissecting Outlier
 * Dynamics in LLM NVFP4 Pretraining", abstract).
 *
 * Q4 as implemented (a reading; the pages give no bit-level recipe):
 *   blocks of 16 along the GEMM contraction axis (the tensor's columns);
 *   amax   = max |T| over the tensor (per segment for grouped calls)
 *   S_enc  = fp32(2688 / amax), or 1 when amax == 0 or the quotient is not
 *            finite;  S_dec = fp32(1 / S_enc)
 *   s_b    = fp32(fp32(amax_b / 6) * S_enc) capped at 448 -> E4M3FN (RNE,
 *            subnormals kept) = the block's scale byte, value d_b
 *   e_b    = fp32(S_enc / d_b) (0 if d_b == 0);  v = fp32(t * e_b)
 *   E2M1 code (sign << 3 | index into {0,.5,1,1.5,2,3,4,6}) by
 *     RN: nearest, ties to the even index, |v| >= 6 -> 6, or
 *     SR: with lo <= |v| < hi the neighbouring grid points and
 *         frac = (|v| - lo) / (hi - lo), up iff floor(2^22 frac) + 64 u >= 2^22,
 *         u the element's 16-bit
 *         draw from Philox4x32-10: key = seed, counter = (g lo, g hi,
 *         stream, 0), g = idx >> 3, word (idx >> 1) & 3, half idx & 1,
 *         idx = row * cols + col (global row for grouped tensors).
 *   SR streams: 0 residual and vanilla activations, 1 means, 2 weights,
 *   3 transposed residuals (wgrad).
 *   The mean is fp32(RN64(exact column sum) / l); the residual is
 *   fp32(x - mu) with the unquantized mean.
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers owned by the caller.  The
 *     library allocates nothing and keeps no state between calls beyond a
 *     per-device record that a kernel's LDS limit was raised (set once,
 *     atomically); calls may come from several threads.
 *   - Work is enqueued on `stream` (NULL = the default stream) and the call
 *     returns without synchronising.  Scales flow device to device.
 *   - Arguments are validated before any HIP call; a rejected call enqueues
 *     nothing and returns the status.  Nothing aborts.
 *   - The workspace `ws` (device, >= averis_workspace_bytes(...) bytes,
 *     256-byte aligned) holds intermediate results only; its contents on
 *     entry do not matter.  Calls that share a workspace must be ordered on
 *     one stream.
 *   - Values that are not finite in an input give unspecified codes.
 */
#ifndef AVERIS_H
#define AVERIS_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define AVERIS_ABI_VERSION 1

typedef enum {
  AVERIS_OK = 0,
  AVERIS_E_NULL = 1,       /* a required pointer is NULL                      */
  AVERIS_E_SHAPE = 2,      /* negative size, cols % 16 != 0, operand mismatch */
  AVERIS_E_DTYPE = 3,      /* unknown dtype                                   */
  AVERIS_E_ALIGN = 4,      /* pointer or leading dimension misaligned         */
  AVERIS_E_WORKSPACE = 5,  /* workspace missing or smaller than required      */
  AVERIS_E_ARG = 6,        /* other invalid argument (rounding, stream, nseg) */
  AVERIS_E_HIP = 7         /* a kernel launch failed                          */
} averis_status_t;

typedef enum { AVERIS_F32 = 0, AVERIS_BF16 = 1 } averis_dtype_t;
typedef enum { AVERIS_RN = 0, AVERIS_SR = 1 } averis_round_t;

/* Workspace queries, see averis_workspace_bytes. */
typedef enum {
  AVERIS_OP_SPLIT_QUANT = 0,  /* rows, cols, nseg (nseg = 0: not grouped)     */
  AVERIS_OP_QUANT = 1,        /* rows, cols, nseg (batch for batched quant)   */
  AVERIS_OP_GEMM = 2,         /* rows = M, cols = K, n = N, nseg              */
  AVERIS_OP_WGRAD = 3,        /* rows = m, cols = l (tokens), n               */
  AVERIS_OP_QUANT_PAIR_MULTI = 4, /* n = number of weights (rows, cols unused) */
  AVERIS_OP_MOE_SORT = 5,     /* rows = tokens * topk slots, n = experts (cols unused) */
  AVERIS_OP_GRAD_NORM = 6,    /* n = number of tensors (rows, cols unused)    */
  AVERIS_OP_FP8_GEMM = 7,     /* rows = m, cols = k, n, nseg (0: not grouped) */
  AVERIS_OP_FP8_WGRAD = 8,    /* rows = m, cols = tokens, n, nseg             */
  AVERIS_OP_RMSNORM_GRAD = 9, /* rows, cols                                   */
  AVERIS_OP_FP8_ACT_GRAD = 10 /* rows, cols, nseg (0: not grouped)            */
} averis_op_t;

/* An NVFP4-style tensor of rows x cols logical elements, 16-blocks along
 * cols.  codes: rows * cols/2 bytes, row-major, byte j of a row holds element
 * 2j in bits 3:0 and element 2j+1 in bits 7:4; 16-byte aligned.
 * scales: rows * cols/16 E4M3FN bytes, row-major; 16-byte aligned.
 * tscale: 2 floats [S_enc, S_dec] per tensor (per segment / batch entry for
 * grouped calls).
 * All three are device pointers. */
typedef struct {
  uint8_t* codes;
  uint8_t* scales;
  float*   tscale;
  int64_t  rows;
  int64_t  cols;
} averis_nvfp4_t;

/* ---------------------------------------------------------------------- */
/* Split-quant (Lighthouse §2.1 column mean; §2.2 X_R = X - 1 mu, separate */
/* quantization of mean and residual; gist.science summary §2).            */
/* ---------------------------------------------------------------------- */

/* a: rows x cols activation or output gradient (dtype F32 or BF16), row
 * stride lda elements (lda >= cols, lda * element size a multiple of 16
 * bytes, a 16-byte aligned).  Writes
 *   residual: rows x cols, Q4(a - 1 mu) with SR stream 0 (or RN),
 *   mean:     1 x cols,    Q4(mu) with SR stream 1 (or RN),
 *   mean_f32: the fp32 mean (optional, may be NULL), cols floats.
 * rows == 0 gives mu = 0 and an all-zero mean tensor with S_enc = 1.
 * Workspace: averis_workspace_bytes(AVERIS_OP_SPLIT_QUANT, rows, cols, 0, 0). */
averis_status_t averis_split_quant(const void* a, averis_dtype_t dtype, int64_t rows, int64_t cols,
                                   int64_t lda, uint64_t seed, averis_round_t rnd,
                                   const averis_nvfp4_t* residual, const averis_nvfp4_t* mean,
                                   float* mean_f32, void* ws, size_t ws_bytes, hipStream_t stream);

/* Grouped split-quant over expert segments (the paper's MoE runs, arXiv
 * abstract): rows seg_offsets[s] .. seg_offsets[s+1]-1 form segment s, each
 * with its own mean (row s of `mean`, nseg x cols, SR index s*cols + col)
 * and its own residual tensor scale (residual->tscale holds 2*nseg floats,
 * as does mean->tscale).  seg_offsets: DEVICE int64[nseg+1], non-decreasing,
 * seg_offsets[0] = 0, seg_offsets[nseg] = rows (the kernels clamp values
 * outside [0, rows]).  mean_f32 (optional): nseg x cols.  An empty segment
 * has mean 0.  Workspace: AVERIS_OP_SPLIT_QUANT with nseg. */
averis_status_t averis_split_quant_grouped(const void* a, averis_dtype_t dtype, int64_t rows,
                                           int64_t cols, int64_t lda, const int64_t* seg_offsets,
                                           int nseg, uint64_t seed, averis_round_t rnd,
                                           const averis_nvfp4_t* residual,
                                           const averis_nvfp4_t* mean, float* mean_f32, void* ws,
                                           size_t ws_bytes, hipStream_t stream);

/* Split-quant with the mean-energy ratio ([Lighthouse] §7 recommends
 * monitoring R = ||mu||_2 / sqrt(E||X||^2 / N) as a free stability signal).
 * Reading: E||X||^2 is the operand's sum of squares ||A||_F^2 and N its row
 * count l, so R = ||mu||_2 / sqrt(||A||_F^2 / l) in [0, 1] (1 when every row
 * equals mu), computed from fp64 column sums and sums of squares gathered in
 * the statistics pass; R = 0 for an empty segment or an all-zero one.
 * seg_offsets = NULL with nseg = 1 is averis_split_quant, otherwise
 * averis_split_quant_grouped; the quantized outputs are bit for bit those of
 * that call.  ratio: device float[nseg] (4-byte aligned), required.
 * Workspace: AVERIS_OP_SPLIT_QUANT as for the call it extends. */
averis_status_t averis_split_quant_ratio(const void* a, averis_dtype_t dtype, int64_t rows,
                                         int64_t cols, int64_t lda, const int64_t* seg_offsets,
                                         int nseg, uint64_t seed, averis_round_t rnd,
                                         const averis_nvfp4_t* residual,
                                         const averis_nvfp4_t* mean, float* mean_f32, float* ratio,
                                         void* ws, size_t ws_bytes, hipStream_t stream);

/* ---------------------------------------------------------------------- */
/* Plain quant: the vanilla-FP4 arm (arXiv abstract: "vanilla NVFP4") and  */
/* the weight operand W (Lighthouse §2.2, both equations).                 */
/* ---------------------------------------------------------------------- */

/* Q4 of the logical rows x cols tensor T, blocks along cols, one tensor
 * scale.  transpose = 0: T[r][c] = a[r*lda + c]; transpose = 1:
 * T[r][c] = a[c*lda + r] (a stored cols x rows; used for the forward copy
 * of W, Q4(W^T)).  sr_stream: 0 for activations, 2 for weights.
 * Workspace: AVERIS_OP_QUANT (rows, cols, 0). */
averis_status_t averis_quant(const void* a, averis_dtype_t dtype, int64_t rows, int64_t cols,
                             int64_t lda, int transpose, uint64_t seed, averis_round_t rnd,
                             uint32_t sr_stream, const averis_nvfp4_t* out, void* ws,
                             size_t ws_bytes, hipStream_t stream);

/* Batched plain quant: `batch` independent rows x cols tensors (matrix b at
 * a + b*batch_stride elements), each with its own tensor scale
 * (out->tscale: 2*batch floats); out is (batch*rows) x cols and the SR index
 * uses the global row b*rows + r.  Used for per-expert weights.
 * Workspace: AVERIS_OP_QUANT (rows, cols, batch). */
averis_status_t averis_quant_batched(const void* a, averis_dtype_t dtype, int batch, int64_t rows,
                                     int64_t cols, int64_t lda, int64_t batch_stride,
                                     int transpose, uint64_t seed, averis_round_t rnd,
                                     uint32_t sr_stream, const averis_nvfp4_t* out, void* ws,
                                     size_t ws_bytes, hipStream_t stream);

/* Both quantized copies of a weight in one call (Lighthouse §2.2: the
 * forward product takes Q4(W^T) with blocks along m, the dgrad product Q4(W)
 * with blocks along n).  a holds `batch` stored rows x cols matrices W_b
 * (row stride lda, matrix b at a + b*batch_stride elements).  Writes
 *   out   = Q4(W_b),   (batch*rows) x cols, blocks along cols, and
 *   out_t = Q4(W_b^T), (batch*cols) x rows, blocks along rows,
 * with one tensor scale per matrix (max |W_b|, shared by both copies).
 * Codes, scales and tensor scales are those of averis_quant_batched with
 * transpose = 0 (out) and transpose = 1 (out_t), the same seed and stream,
 * bit for bit.  Needs rows % 16 == 0, cols % 16 == 0, both > 0, 16-byte
 * aligned a and lda * element size % 16 == 0.
 * Workspace: AVERIS_OP_QUANT (rows, cols, batch). */
averis_status_t averis_quant_pair(const void* a, averis_dtype_t dtype, int batch, int64_t rows,
                                  int64_t cols, int64_t lda, int64_t batch_stride, uint64_t seed,
                                  averis_round_t rnd, uint32_t sr_stream,
                                  const averis_nvfp4_t* out, const averis_nvfp4_t* out_t,
                                  void* ws, size_t ws_bytes, hipStream_t stream);

/* Both GEMM copies of a weight from ONE quantization in 16 x 16 tiles (the
 * shared weight that Lighthouse §2.2 implies by writing the dgrad operand as
 * the transpose of the forward one).  Same arguments, shapes, layouts and
 * workspace as averis_quant_pair; the difference: each 16 x 16 tile of W_b
 * has one E4M3 scale, from the tile's largest magnitude, and the codes are
 * encoded once (SR draw of element (r, c) of W_b: index (b*rows + r) * cols
 * + c, stream sr_stream) and written in both layouts, so that
 * deq(out_t) = deq(out)^T exactly.  Every 16-run of out and of out_t carries
 * its tile's scale byte; the GEMM calls take both copies unchanged.
 * Errors as averis_quant_pair. */
averis_status_t averis_quant_pair_2d(const void* a, averis_dtype_t dtype, int batch, int64_t rows,
                                     int64_t cols, int64_t lda, int64_t batch_stride,
                                     uint64_t seed, averis_round_t rnd, uint32_t sr_stream,
                                     const averis_nvfp4_t* out, const averis_nvfp4_t* out_t,
                                     void* ws, size_t ws_bytes, hipStream_t stream);

/* One weight of averis_quant_pair_multi: the stored rows x cols matrix W at
 * a (device, row stride lda elements), its seed and its two outputs (host
 * pointers to descriptors of device buffers): out = Q4(W), rows x cols, and
 * out_t = Q4(W^T), cols x rows, as averis_quant_pair writes them with
 * batch 1. */
typedef struct {
  const void* a;
  int64_t rows;
  int64_t cols;
  int64_t lda;
  uint64_t seed;
  const averis_nvfp4_t* out;
  const averis_nvfp4_t* out_t;
} averis_weight_t;

#define AVERIS_MAX_WEIGHTS 16

/* Both quantized copies of each of n weights of their own shapes (Lighthouse
 * §2.2, as averis_quant_pair; e.g. the seven linears of a transformer block,
 * all known when a step starts) in two launches instead of two per weight.
 * For every i the codes, scales and tensor scales are those of
 * averis_quant_pair(w[i].a, dtype, 1, w[i].rows, w[i].cols, w[i].lda, 0,
 * w[i].seed, rnd, sr_stream, w[i].out, w[i].out_t, ...), bit for bit.
 * w: host array of n entries (1 <= n <= AVERIS_MAX_WEIGHTS), read during the
 * call only; every entry must meet averis_quant_pair's requirements (else
 * that call's status, nothing launched).  The outputs of different entries
 * must not overlap.  Workspace: AVERIS_OP_QUANT_PAIR_MULTI with n. */
averis_status_t averis_quant_pair_multi(int n, const averis_weight_t* w, averis_dtype_t dtype,
                                        averis_round_t rnd, uint32_t sr_stream, void* ws,
                                        size_t ws_bytes, hipStream_t stream);

/* Grouped plain quant of activations: one tensor scale per segment
 * (vanilla arm of the grouped case).  Workspace: AVERIS_OP_QUANT with nseg. */
averis_status_t averis_quant_grouped(const void* a, averis_dtype_t dtype, int64_t rows,
                                     int64_t cols, int64_t lda, const int64_t* seg_offsets,
                                     int nseg, uint64_t seed, averis_round_t rnd,
                                     uint32_t sr_stream, const averis_nvfp4_t* out, void* ws,
                                     size_t ws_bytes, hipStream_t stream);

/* ---------------------------------------------------------------------- */
/* Quantized GEMMs (Lighthouse §2.2; gist.science summary §2).             */
/* C = deq(A) deq(B)^T (+ 1 deq(mean) deq(B)^T), FP32 accumulation.        */
/* ---------------------------------------------------------------------- */

/* Forward: y (xr->rows x wt->rows) = 1 (mean W) + X_R W with
 *   xr:   Q4(X - 1 mu), l x m
 *   mean: Q4(mu), 1 x m
 *   wt:   Q4(W^T), n x m (blocks along m)
 * y: F32 or BF16, row stride ldy >= n elements.  Workspace: AVERIS_OP_GEMM
 * (l, m, n, 0). */
averis_status_t averis_gemm_fwd(const averis_nvfp4_t* xr, const averis_nvfp4_t* mean,
                                const averis_nvfp4_t* wt, void* y, averis_dtype_t ydtype,
                                int64_t ldy, void* ws, size_t ws_bytes, hipStream_t stream);

/* Dgrad: dx (dr->rows x w->rows) = 1 (mean_d W^T) + D_R W^T with
 *   dr:     Q4(D - 1 mu_D), l x n
 *   mean_d: Q4(mu_D), 1 x n
 *   w:      Q4(W), m x n (blocks along n)
 * Same kernel as the forward; only the quantized copy of W differs. */
averis_status_t averis_gemm_dgrad(const averis_nvfp4_t* dr, const averis_nvfp4_t* mean_d,
                                  const averis_nvfp4_t* w, void* dx, averis_dtype_t dxdtype,
                                  int64_t lddx, void* ws, size_t ws_bytes, hipStream_t stream);

/* The rank-one row formed once, by the split ([Lighthouse] §2.2: the term
 * 1(mu_bar W_bar) is a row vector added to every output row).
 * averis_split_quant_rank1 is averis_split_quant (bit for bit the same
 * residual, mean and mean_f32) that also writes
 *   rho[j] = deq(mean) . deq(b_j),  j < b->rows,
 * for the B operand of the GEMM that will take this split (wt for the
 * forward, w for dgrad: b->cols == cols), fp32 accumulation of exact
 * products, times the two tensor scales.  rho: device float[b->rows], 4-byte
 * aligned.  cols <= 32768 (the dequantized mean is staged in on-chip memory).
 * Workspace: AVERIS_OP_SPLIT_QUANT (rows, cols, 0, 0).
 * averis_gemm_rank1 then computes c = deq(a) deq(b)^T + 1 rho^T (a: the
 * residual, b as above) with no mean row of its own; it equals averis_gemm_fwd
 * / averis_gemm_dgrad of the same operands up to fp32 summation order.  No
 * workspace. */
averis_status_t averis_split_quant_rank1(const void* a, averis_dtype_t dtype, int64_t rows,
                                         int64_t cols, int64_t lda, uint64_t seed,
                                         averis_round_t rnd, const averis_nvfp4_t* residual,
                                         const averis_nvfp4_t* mean, float* mean_f32,
                                         const averis_nvfp4_t* b, float* rho, void* ws,
                                         size_t ws_bytes, hipStream_t stream);
averis_status_t averis_gemm_rank1(const averis_nvfp4_t* a, const float* rho,
                                  const averis_nvfp4_t* b, void* c, averis_dtype_t cdtype,
                                  int64_t ldc, hipStream_t stream);

/* The rank-one rows of several GEMMs that take the same split (the
 * projections that read one input, e.g. q, k and v of a transformer block;
 * [Lighthouse] §2.2 as above): averis_split_quant_rank1 with nb B operands
 * (1 <= nb <= AVERIS_MAX_RANK1), b[i]->cols == cols, writing
 *   rho[i][j] = deq(mean) . deq(b[i]_j),  j < b[i]->rows,
 * each bit for bit the row averis_split_quant_rank1 with b[i] alone writes,
 * and the same residual, mean and mean_f32.  b, rho: host arrays of nb
 * pointers (descriptors of device tensors; device float[b[i]->rows], 4-byte
 * aligned), read during the call only.  Workspace as averis_split_quant_rank1.
 * Errors as averis_split_quant_rank1, for any entry. */
#define AVERIS_MAX_RANK1 4
averis_status_t averis_split_quant_rank1_multi(const void* a, averis_dtype_t dtype, int64_t rows,
                                               int64_t cols, int64_t lda, uint64_t seed,
                                               averis_round_t rnd, const averis_nvfp4_t* residual,
                                               const averis_nvfp4_t* mean, float* mean_f32,
                                               int nb, const averis_nvfp4_t* const* b,
                                               float* const* rho, void* ws, size_t ws_bytes,
                                               hipStream_t stream);

/* Grouped forms (expert segments, as averis_split_quant_grouped and
 * averis_gemm_grouped): b holds nseg stacked N x cols matrices (expert s =
 * rows s*N .. s*N+N-1, its own tensor scale b->tscale[2s..2s+1]) and
 *   rho[s*N + j] = deq(mean_s) . deq(b_s,j)   (device float[nseg*N]);
 * an empty segment has mean 0 and so rho_s = 0.  averis_gemm_grouped_rank1:
 * c[rows of s] = deq(a_s) deq(b_s)^T + 1 rho_s^T. */
averis_status_t averis_split_quant_grouped_rank1(const void* a, averis_dtype_t dtype,
                                                 int64_t rows, int64_t cols, int64_t lda,
                                                 const int64_t* seg_offsets, int nseg,
                                                 uint64_t seed, averis_round_t rnd,
                                                 const averis_nvfp4_t* residual,
                                                 const averis_nvfp4_t* mean, float* mean_f32,
                                                 const averis_nvfp4_t* b, float* rho, void* ws,
                                                 size_t ws_bytes, hipStream_t stream);
averis_status_t averis_gemm_grouped_rank1(const averis_nvfp4_t* a, const float* rho,
                                          const averis_nvfp4_t* b, const int64_t* seg_offsets,
                                          int nseg, void* c, averis_dtype_t cdtype, int64_t ldc,
                                          hipStream_t stream);

/* Vanilla arm: c = deq(a) deq(b)^T, no mean term. */
averis_status_t averis_gemm_vanilla(const averis_nvfp4_t* a, const averis_nvfp4_t* b, void* c,
                                    averis_dtype_t cdtype, int64_t ldc, void* ws, size_t ws_bytes,
                                    hipStream_t stream);

/* Grouped GEMM: for each segment s (rows seg_offsets[s] .. [s+1]-1 of a),
 * c[rows of s] = deq(a_s) deq(b_s)^T (+ 1 deq(mean_s) deq(b_s)^T), where
 * b is (nseg * N) x K (expert s = rows s*N .. s*N+N-1, its own tensor scale
 * b->tscale[2s..2s+1]), a->tscale and mean->tscale hold 2*nseg floats,
 * mean is nseg x K or NULL (vanilla).  Workspace: AVERIS_OP_GEMM with nseg. */
averis_status_t averis_gemm_grouped(const averis_nvfp4_t* a, const averis_nvfp4_t* mean,
                                    const averis_nvfp4_t* b, const int64_t* seg_offsets, int nseg,
                                    void* c, averis_dtype_t cdtype, int64_t ldc, void* ws,
                                    size_t ws_bytes, hipStream_t stream);

/* ---------------------------------------------------------------------- */
/* wgrad (the W4A4G4 setting of the arXiv abstract and Lighthouse §3.1    */
/* keeps weights, activations and gradients in FP4; §2.2 writes out only   */
/* the forward and dgrad products).  Reading: the split applied to both    */
/* operands of                                                             */
/* dW = X^T D.  The residuals' column sums vanish, so                      */
/*   dW = deq(Q4(X_R^T)) deq(Q4(D_R^T))^T + l mu_X mu_D^T,                 */
/* with the transposed residuals quantized in 16-blocks along the tokens   */
/* (the contraction axis of this product) and the outer product taken from */
/* the fp32 means (no contraction runs over them).                         */
/* ---------------------------------------------------------------------- */

/* out_t = Q4((a - 1 mu)^T): cols x rows, 16-blocks along the rows (tokens),
 * SR stream 3, element index col * rows + row.  a: rows x cols (F32 or BF16,
 * row stride lda, as for averis_split_quant); rows % 16 == 0 (rows may be 0).
 * mu: the fp32 column means averis_split_quant wrote for the same a (cols
 * floats, device, 16-byte aligned).  residual_tscale: the residual tensor's
 * [S_enc, S_dec] from that call (device, 2 floats); the transposed residual
 * holds the same values and takes the same tensor scale, copied to
 * out_t->tscale.  No workspace.  Other arguments as for averis_split_quant. */
averis_status_t averis_residual_t_quant(const void* a, averis_dtype_t dtype, int64_t rows,
                                        int64_t cols, int64_t lda, const float* mu,
                                        const float* residual_tscale, uint64_t seed,
                                        averis_round_t rnd, const averis_nvfp4_t* out_t,
                                        hipStream_t stream);

/* dw (m x n, F32 or BF16, row stride lddw >= n) =
 *   deq(xt) deq(dt)^T + l mu_x mu_d^T
 * with xt = Q4(X_R^T) (m x l) and dt = Q4(D_R^T) (n x l) from
 * averis_residual_t_quant, mu_x (m floats) and mu_d (n floats) the fp32
 * means of X and D (device, 16-byte aligned); m, n, l multiples of 16 (l may
 * be 0: dw = l mu_x mu_d^T = 0).  FP32 accumulation; the token axis is split
 * into fp32 partials that are summed in a fixed order, so repeated calls
 * give the same bits.  Workspace: averis_workspace_bytes(AVERIS_OP_WGRAD,
 * m, l, n, 0). */
averis_status_t averis_gemm_wgrad(const averis_nvfp4_t* xt, const averis_nvfp4_t* dt,
                                  const float* mu_x, const float* mu_d, void* dw,
                                  averis_dtype_t dwdtype, int64_t lddw, void* ws, size_t ws_bytes,
                                  hipStream_t stream);

/* ---------------------------------------------------------------------- */
/* Column statistics fused into the producer (Lighthouse §2.2 cost note:   */
/* the split adds two column reductions and two subtractions; §4.2: it     */
/* changes the quantization kernel's pre-processing).  The GEMM that makes */
/* the next split's input gathers that input's column statistics in its   */
/* epilogue, so the split reads its input once.                            */
/* ---------------------------------------------------------------------- */

/* averis_gemm_rank1 with bf16 output c (n = b->rows columns, row stride ldc)
 * that also writes the column statistics of c, as stored, into ws: per
 * 256-row tile and column, the fp64 sum, max, min and smallest nonzero
 * magnitude.  ws is the split-quant workspace of c:
 * averis_workspace_bytes(AVERIS_OP_SPLIT_QUANT, a->rows, n, 0, 0) bytes, to
 * be passed unchanged to averis_split_quant_from_stats for this c (nothing
 * else may use it in between).  Needs a->cols % 64 == 0, n % 16 == 0, c
 * 16-byte aligned and ldc * 2 % 16 == 0 (c is then a valid split input).
 * c equals averis_gemm_rank1's bf16 output bit for bit. */
averis_status_t averis_gemm_rank1_stats(const averis_nvfp4_t* a, const float* rho,
                                        const averis_nvfp4_t* b, void* c, int64_t ldc, void* ws,
                                        size_t ws_bytes, hipStream_t stream);

/* averis_split_quant of the bf16 rows x cols tensor a (row stride lda) from
 * the column statistics that averis_gemm_rank1_stats wrote into ws when it
 * produced a: the mean, the tensor scales and the quantized outputs are
 * averis_split_quant's bit for bit, and a is read once (by the quant pass;
 * a column whose sum is not certified exact is re-summed from its tiles'
 * partials and, for a tile not exact on its own, from its rows).  b and rho:
 * both NULL, or the rank-one row of the GEMM that takes this split, as for
 * averis_split_quant_rank1.  Order this call after that GEMM (same stream). */
averis_status_t averis_split_quant_from_stats(const void* a, int64_t rows, int64_t cols,
                                              int64_t lda, uint64_t seed, averis_round_t rnd,
                                              const averis_nvfp4_t* residual,
                                              const averis_nvfp4_t* mean, float* mean_f32,
                                              const averis_nvfp4_t* b, float* rho, void* ws,
                                              size_t ws_bytes, hipStream_t stream);

/* ---------------------------------------------------------------------- */
/* Allocation-free split-quant                                             */
/* ---------------------------------------------------------------------- */

/* Bytes of the device array that averis_split_quant_noalloc uses as its
 * workspace (one copy per device). */
#define AVERIS_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)

/* For callers that cannot allocate device memory or pass a workspace: code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc.  averis_split_quant with the same arguments and results, bit for
 * bit, whose workspace is a file-scope device array of
 * AVERIS_NOALLOC_SCRATCH_BYTES inside the library: the call allocates
 * nothing.  The array holds the split's intermediate results, which depend on
 * the shape: averis_workspace_bytes(AVERIS_OP_SPLIT_QUANT, rows, cols, 0, 0)
 * must not exceed AVERIS_NOALLOC_SCRATCH_BYTES (about rows / 128 * cols * 28
 * bytes: a 16384 x 3072 input fits), else the call returns
 * AVERIS_E_WORKSPACE, enqueues nothing, and averis_last_error() names both
 * sizes.  Every call on one device shares that device's array: calls that
 * overlap on one device (several streams or threads at once) race and give
 * wrong results; order them on one stream.  The first call on a device looks
 * up the array's address there (once; the lookup is not captured). */
averis_status_t averis_split_quant_noalloc(const void* a, averis_dtype_t dtype, int64_t rows,
                                           int64_t cols, int64_t lda, uint64_t seed,
                                           averis_round_t rnd, const averis_nvfp4_t* residual,
                                           const averis_nvfp4_t* mean, float* mean_f32,
                                           hipStream_t stream);

/* ---------------------------------------------------------------------- */
/* Mixture-of-experts routing and token exchange: from router logits to    */
/* the rows sorted by expert that every grouped call takes, and back, with */
/* the gradients.  A slot is one of a token's topk choices: slot t * topk  */
/* + j; tokens * topk < 2^31.  Matrices are F32 or BF16, any row stride    */
/* and element alignment; sums are fp32, rounded once on output.           */
/* ---------------------------------------------------------------------- */

#define AVERIS_MAX_EXPERTS 1024
#define AVERIS_MAX_TOPK 32

/* expert_ids[t][j], weights[t][j] (tokens x topk): the topk largest of token
 * t's logits in descending order and their softmax weights.  Ties go to the
 * lowest expert; a NaN logit counts as the largest; it and +inf make the
 * weights of the token's experts NaN.  A logit of -inf is masked: never chosen,
 * and a slot for which no open expert is left gets id -1 and weight 0 (every
 * slot of a token whose logits are all -inf).  renorm = 1: softmax over the chosen logits; 0: over
 * all of them.  logits: tokens x experts, row stride ld >= experts;
 * 1 <= topk <= min(experts, AVERIS_MAX_TOPK). */
averis_status_t averis_moe_route(const void* logits, averis_dtype_t dtype, int64_t tokens,
                                 int experts, int64_t ld, int topk, int renorm,
                                 int32_t* expert_ids, float* weights, hipStream_t stream);

/* dlogits (tokens x experts, the logits' type, row stride ldd >= experts)
 * from dweights (tokens x topk): the gradient of averis_moe_route's weights
 * with the choice held fixed.  expert_ids as that call wrote them (for the
 * same logits, topk and renorm); a slot with id -1 contributes nothing.
 * dlogits may be logits. */
averis_status_t averis_moe_route_grad(const void* logits, averis_dtype_t dtype, int64_t tokens,
                                      int experts, int64_t ld, int topk, int renorm,
                                      const int32_t* expert_ids, const float* dweights,
                                      void* dlogits, int64_t ldd, hipStream_t stream);

#define AVERIS_MAX_GROUPS 64

/* What a token's experts are chosen and weighted by: s_e = e^l_e / sum e^l
 * over the open experts, or 1 / (1 + e^-l_e). */
typedef enum { AVERIS_SCORE_SOFTMAX = 0, AVERIS_SCORE_SIGMOID = 1 } averis_score_t;

/* Routing by scores, with a bias that balances the experts' load and with
 * groups of experts.  Experts are chosen by c_e = s_e + bias[e] (bias:
 * `experts` floats, NULL: 0) and weighted by s_e:
 *   the experts divide in order into `groups` equal groups (at most
 *   AVERIS_MAX_GROUPS); where topk_groups < groups only the topk_groups with
 *   the largest scores stay, a group's score being the sum of its group_top
 *   (1 or 2) largest c_e (of its one open expert, c_e);
 *   of theirs, expert_ids[t][j] are the topk largest c_e in descending order,
 *   weights[t][j] = scale s_e, divided by the sum of the chosen s_e with renorm = 1.
 * The choice is by the values of c_e in fp64 (without a bias, and with
 * group_top = 1 or all groups, of l_e, which order alike), equal ones by the
 * lowest index first (sums of two different pairs that only fp64's own rounding
 * tells apart may go either way).  A logit of -inf, or c_e = -inf, is closed: never chosen, and a
 * slot for which none is left gets id -1 and weight 0; a group without an open
 * expert does not stay.  A NaN value counts as the largest.  A NaN logit makes its
 * weight NaN (with renorm or softmax scores all of the token's; so does +inf with
 * softmax: where the choice is by c_e, the lowest open indexes are then taken).
 * Other arguments as for averis_moe_route; topk <= topk_groups experts / groups. */
averis_status_t averis_moe_route_groups(const void* logits, averis_dtype_t dtype, int64_t tokens,
                                        int experts, int64_t ld, int topk, const float* bias,
                                        averis_score_t score, int groups, int topk_groups,
                                        int group_top, int renorm, float scale,
                                        int32_t* expert_ids, float* weights, hipStream_t stream);

/* dlogits from dweights: the gradient of averis_moe_route_groups' weights with
 * the choice held fixed (the bias has none).  expert_ids as that call wrote them for the
 * same logits, topk, score, renorm and scale; an id outside the experts
 * contributes nothing.  Zeros outside the chosen, but for softmax without
 * renorm.  dlogits (the logits' type, row stride ldd >= experts) may be
 * logits. */
averis_status_t averis_moe_route_groups_grad(const void* logits, averis_dtype_t dtype,
                                             int64_t tokens, int experts, int64_t ld, int topk,
                                             averis_score_t score, int renorm, float scale,
                                             const int32_t* expert_ids, const float* dweights,
                                             void* dlogits, int64_t ldd, hipStream_t stream);

/* The order of the slots by expert, stable (within an expert by slot):
 *   seg_offsets[experts + 1]: expert e owns rows seg_offsets[e] ..
 *                seg_offsets[e + 1] - 1 (the array the grouped calls take);
 *   pos[slot]:   the slot's row; for a dropped slot (id outside [0, experts))
 *                ~row, a negative number, its row in the tail
 *                seg_offsets[experts] .. tokens * topk - 1;
 *   src[row]:    the row's slot (optional, may be NULL), tail included.
 * Workspace: AVERIS_OP_MOE_SORT (0 bytes for short inputs). */
averis_status_t averis_moe_sort(const int32_t* expert_ids, int64_t tokens, int topk, int experts,
                                int64_t* seg_offsets, int32_t* pos, int32_t* src, void* ws,
                                size_t ws_bytes, hipStream_t stream);

/* rows[pos[t][j]] = x[t] for every slot; the tail rows are written as zeros.
 * x: tokens x cols, rows: (tokens * topk) x cols, pos from averis_moe_sort.
 * Its gradient, dx[t] = sum_j drows[pos[t][j]], is averis_moe_combine with
 * weights = NULL. */
averis_status_t averis_moe_dispatch(const void* x, averis_dtype_t dtype, int64_t tokens,
                                    int64_t cols, int64_t ldx, const int32_t* pos, int topk,
                                    void* rows, int64_t ldr, hipStream_t stream);

/* y[t] = sum_j weights[t][j] rows[pos[t][j]] over the slots that were not
 * dropped, in slot order (weights = NULL: all 1); a token without any gets
 * zeros.  Dropped slots' rows and weights are not read. */
averis_status_t averis_moe_combine(const void* rows, averis_dtype_t dtype, int64_t tokens,
                                   int64_t cols, int64_t ldr, const int32_t* pos,
                                   const float* weights, int topk, void* y, int64_t ldy,
                                   hipStream_t stream);

/* The gradients of averis_moe_combine: drows[pos[t][j]] = weights[t][j] dy[t]
 * (tail rows zero) and dweights[t][j] = <dy[t], rows[pos[t][j]]> (0 for a
 * dropped slot).  drows may be rows. */
averis_status_t averis_moe_combine_grad(const void* dy, averis_dtype_t dtype, int64_t tokens,
                                        int64_t cols, int64_t ldy, const void* rows, int64_t ldr,
                                        const int32_t* pos, const float* weights, int topk,
                                        void* drows, int64_t lddr, float* dweights,
                                        hipStream_t stream);

/* ---------------------------------------------------------------------- */
/* Linears in 8-bit floating point with one scale for a block of 128, for  */
/* the layers a recipe keeps out of FP4.                                   */
/*   E4M3FN codes; one E8M0 scale (2^(byte - 127)) for each run of 128     */
/*   along the contraction axis, or for each 128 x 128 tile of a weight:   */
/*   the smallest power of two with amax <= 448 scale, at least 2^-127.    */
/*   Dividing by it is exact; the code is rounded to nearest, ties to      */
/*   even.  A run (tile) with a value that is not finite gets NaN codes    */
/*   and scale 1.                                                          */
/* Products: fp32 accumulation.  The matrix instruction adds the products  */
/* of eight consecutive k with each term cut at 2^-13 of the largest of    */
/* them, so |error| <= 2^-10 sum |a b| at worst (1.5e-5 of the result's    */
/* norm on random operands), before the output's rounding: one BF16 value  */
/* in 90 is rounded to the neighbour of what an exact sum would give.      */
/* ---------------------------------------------------------------------- */

/* rows x cols logical elements.  codes: rows of cols rounded up to 128
 * bytes, 16-byte aligned; the bytes past cols are 0.  scales: rows of
 * ceil(cols / 128) bytes rounded up to 4, 4-byte aligned; the bytes past
 * ceil(cols / 128) are not used.  Device pointers. */
typedef struct {
  uint8_t* codes;
  uint8_t* scales;
  int64_t  rows;
  int64_t  cols;
} averis_fp8_t;

/* Columns of a grouped transposed copy: each segment's rows start at a
 * multiple of 128 (a run never straddles two segments), and there is room
 * for any division of `rows` rows into nseg segments.  -1 for a bad query. */
int64_t averis_fp8_seg_cols(int64_t rows, int64_t nseg);

/* a (rows x cols, F32 or BF16, row stride lda, element aligned) quantized in
 * runs along its columns into out (rows x cols: the operand of forward and
 * dgrad) and in runs along its rows into out_t (cols x rows, the transposed
 * copy: the operand of wgrad), from one read; either may be NULL.
 * seg_offsets (DEVICE int64[nseg + 1], as for the grouped calls) or NULL
 * with nseg = 1: with segments out_t is cols x averis_fp8_seg_cols(rows,
 * nseg), segment s from the multiple of 128 after those before it, the rest
 * of its last run 0; with out_t and segments, rows outside every segment are
 * not written to out.  rows, cols <= 2^30; with out_t fewer than 2^23 tiles of
 * 128 x 128 (with segments, for any division of the rows). */
averis_status_t averis_fp8_quant(const void* a, averis_dtype_t dtype, int64_t rows, int64_t cols,
                                 int64_t lda, const int64_t* seg_offsets, int nseg,
                                 const averis_fp8_t* out, const averis_fp8_t* out_t,
                                 hipStream_t stream);

/* Both copies of a weight (or of `batch` stacked ones, matrix b at w + b *
 * batch_stride elements) from one quantization in 128 x 128 tiles: out
 * ((batch * rows) x cols) and out_t ((batch * cols) x rows), exact transposes
 * of each other, every run carrying its tile's scale byte; either may be
 * NULL.  Needs rows, cols > 0. */
averis_status_t averis_fp8_quant_weight(const void* w, averis_dtype_t dtype, int batch,
                                        int64_t rows, int64_t cols, int64_t ldw,
                                        int64_t batch_stride, const averis_fp8_t* out,
                                        const averis_fp8_t* out_t, hipStream_t stream);

/* c = deq(a) deq(b)^T: a m x k, b n x k, c m x n (F32 or BF16, row stride
 * ldc).  With seg_offsets: rows of segment s times the s-th of nseg stacked n
 * x k matrices b (rows of a outside every segment give no output).  Forward:
 * a = Q(X), b = out_t of the weight; dgrad: a = Q(D), b = out of it.  m (from
 * one row, a token) and n <= 2^30, k <= 2^22, at most 2^30 tiles of 128 x 128.
 * Workspace: AVERIS_OP_FP8_GEMM (m, k, n, nseg or 0 without segments; may be 0
 * bytes). */
averis_status_t averis_fp8_gemm(const averis_fp8_t* a, const averis_fp8_t* b,
                                const int64_t* seg_offsets, int nseg, void* c,
                                averis_dtype_t cdtype, int64_t ldc, void* ws, size_t ws_bytes,
                                hipStream_t stream);

/* Activations: z, max(z, 0), z / (1 + e^-z), and the tanh form of gelu,
 * z / 2 (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))). */
typedef enum {
  AVERIS_ACT_NONE = 0,
  AVERIS_ACT_RELU = 1,
  AVERIS_ACT_SILU = 2,
  AVERIS_ACT_GELU = 3
} averis_act_t;

/* averis_fp8_gemm with an epilogue: z = deq(a) deq(b)^T + 1 bias^T, c = act(z) +
 * residual, in fp32 and rounded once to c's type.  bias: n values (F32 or BF16;
 * with segments n for each, nseg x n), or NULL.  residual: m x n of c's type, row
 * stride ldr, or NULL; it may be c.  z: also written, m x n of c's type, row stride
 * ldz, for averis_fp8_act_grad, or NULL; it overlaps neither c nor residual.  An
 * infinite z with a smooth activation gives what the formula gives (-inf: NaN).
 * Everything else, the workspace too, as for averis_fp8_gemm. */
averis_status_t averis_fp8_gemm_act(const averis_fp8_t* a, const averis_fp8_t* b, const void* bias,
                                    averis_dtype_t bias_dtype, averis_act_t act,
                                    const void* residual, int64_t ldr, const int64_t* seg_offsets,
                                    int nseg, void* c, averis_dtype_t cdtype, int64_t ldc, void* z,
                                    int64_t ldz, void* ws, size_t ws_bytes, hipStream_t stream);

/* dw = deq(xt) deq(dt)^T over the tokens: xt m x rows and dt n x rows from
 * averis_fp8_quant's out_t, dw m x n (F32 or BF16, row stride lddw).  With
 * seg_offsets (those of the quantization; xt and dt then have
 * averis_fp8_seg_cols(rows, nseg) columns): nseg matrices one after the
 * other, matrix s (at dw + s * m * lddw elements) over segment s's tokens;
 * zeros for a segment without any.  At most 2^22 rows (with segments,
 * averis_fp8_seg_cols of them: each segment's last run counts whole), which is
 * fewer than averis_fp8_quant takes: longer ones go in parts, added in F32.  m, n
 * <= 2^30, at most 2^30 tiles of 128 x 128 (with segments fewer than 2^24, of
 * all their matrices).  Workspace: AVERIS_OP_FP8_WGRAD (m, rows, n, nseg or
 * 0). */
averis_status_t averis_fp8_gemm_wgrad(const averis_fp8_t* xt, const averis_fp8_t* dt,
                                      int64_t rows, const int64_t* seg_offsets, int nseg,
                                      void* dw, averis_dtype_t dwdtype, int64_t lddw, void* ws,
                                      size_t ws_bytes, hipStream_t stream);

/* ---------------------------------------------------------------------- */
/* Around a block's linears: the norm before them, with the residual's     */
/* addition and its output in fp8, and the way back through the activation */
/* and bias after them.                                                    */
/* ---------------------------------------------------------------------- */

#define AVERIS_MAX_NORM_COLS 16384

/* h = x + residual (rounded to the type; x itself without a residual),
 * rstd[i] = 1 / sqrt(mean of row i's squares of h + eps) (the sum in fp64,
 * rstd rounded to fp32), y = h rstd weight (fp32, rounded to the type).  Each of y
 * (rows x cols, the type of x), out (rows x cols) and out_t (cols x rows, runs
 * along the rows) may be NULL, not all three; out and out_t are what
 * averis_fp8_quant gives of y, bit for bit, whether y is written or not.
 * x, residual, h, y: F32 or BF16, row strides ldx, ldres, ldh, ldy >= cols,
 * element aligned.  residual may be NULL, h is then NULL too and ldh unused;
 * else h is written (it may be x or residual; y overlaps none of the three).  weight:
 * cols elements, F32 or BF16.  rstd: rows floats.  cols <= AVERIS_MAX_NORM_COLS,
 * rows <= 2^30; with out_t fewer than 2^23 tiles of 128 x 128.  eps >= 0; a row
 * whose mean square + eps is 0 gives NaN, as one with a NaN does; one with an
 * infinity has rstd 0, NaN there and 0 elsewhere. */
averis_status_t averis_rmsnorm(const void* x, averis_dtype_t dtype, int64_t rows, int64_t cols,
                               int64_t ldx, const void* residual, int64_t ldres,
                               const void* weight, averis_dtype_t wdtype, double eps, void* h,
                               int64_t ldh, void* y, int64_t ldy, float* rstd,
                               const averis_fp8_t* out, const averis_fp8_t* out_t,
                               hipStream_t stream);

/* The gradients of averis_rmsnorm from dy (of y) and dres (of h, by what else
 * reads it; may be NULL): with v = h rstd (h, rstd as that call left them)
 *   dh = rstd (dy weight - v mean(dy weight v)) + dres: that of x and of residual,
 *   dweight[j] = sum over the rows of dy v (cols floats, may be NULL; a fixed
 *   order: the same bits on every call; zeros for no rows).
 * fp32, dh rounded once to the type; dh may be dy or dres.  Workspace:
 * AVERIS_OP_RMSNORM_GRAD (unused without dweight). */
averis_status_t averis_rmsnorm_grad(const void* dy, averis_dtype_t dtype, int64_t rows,
                                    int64_t cols, int64_t lddy, const void* h, int64_t ldh,
                                    const void* weight, averis_dtype_t wdtype, const float* rstd,
                                    const void* dres, int64_t lddres, void* dh, int64_t lddh,
                                    float* dweight, void* ws, size_t ws_bytes,
                                    hipStream_t stream);

/* dz = dy act'(z) (rows x cols; fp32, relu's slope at 0 is 0, and where it is 0 dz
 * is +0 whatever dy is; the smooth ones' at +-inf 1 and 0): rounded to the type of dy and z and quantized into out and
 * out_t as averis_fp8_quant does, segments included, from one read; dbias[s][j]
 * = sum of dz (before it is rounded) over segment s's rows, nseg x cols floats
 * in a fixed order, zeros for a segment without any.  Each of the three may be
 * NULL, not all.  z is not read (and may be NULL) for AVERIS_ACT_NONE.  With
 * segments, rows outside every one are not written to out.  cols <= 2^27,
 * rows <= 2^30, fewer than 2^23 tiles of 128 x 128 (with segments, for any division
 * of the rows).  Workspace: AVERIS_OP_FP8_ACT_GRAD (unused without dbias). */
averis_status_t averis_fp8_act_grad(const void* dy, averis_dtype_t dtype, int64_t rows,
                                    int64_t cols, int64_t lddy, const void* z, int64_t ldz,
                                    averis_act_t act, const int64_t* seg_offsets, int nseg,
                                    const averis_fp8_t* out, const averis_fp8_t* out_t,
                                    float* dbias, void* ws, size_t ws_bytes, hipStream_t stream);

/* ---------------------------------------------------------------------- */
/* The global gradient norm over many tensors, and clipping                */
/* ---------------------------------------------------------------------- */

/* One gradient: numel elements at grad (device, F32 or BF16, element
 * aligned), clipped into out (the same type; grad itself for in place, or a
 * buffer that overlaps no listed gradient). */
typedef struct {
  const void* grad;
  void* out;
  int64_t numel;
  averis_dtype_t dtype;
} averis_grad_t;

#define AVERIS_MAX_GRADS (1 << 20)

/* norm (device float): sqrt of the sum of squares of every element of the n
 * tensors (fp64 sums in a fixed order: the same bits on every call; 0 for
 * none).  grads: host array, read during the call only; out is not used.
 * Workspace: AVERIS_OP_GRAD_NORM with n. */
averis_status_t averis_grad_norm(int n, const averis_grad_t* grads, float* norm, void* ws,
                                 size_t ws_bytes, hipStream_t stream);

/* averis_grad_norm, and out = grad * min(1, max_norm / (norm + eps)) for each
 * tensor: the factor rounded to fp32's 24 bits, the product rounded to fp32
 * and, for BF16, from there.  A norm that is not finite is not hidden: an infinite
 * one scales by 0 (which leaves NaN in place of infinite elements; by NaN if
 * max_norm is infinite too), NaN scales by NaN.  max_norm, eps >= 0; with
 * norm + eps = 0 the gradients, all zero, stay so. */
averis_status_t averis_grad_clip(int n, const averis_grad_t* grads, double max_norm, double eps,
                                 float* norm, void* ws, size_t ws_bytes, hipStream_t stream);

/* ---------------------------------------------------------------------- */
/* Utilities                                                               */
/* ---------------------------------------------------------------------- */

/* Bytes of workspace an entry point needs (0 if none); a bad query returns
 * 0 and the entry point then rejects the call with AVERIS_E_SHAPE. */
size_t averis_workspace_bytes(averis_op_t op, int64_t rows, int64_t cols, int64_t n, int64_t nseg);

/* Static string for a status code. */
const char* averis_status_str(averis_status_t status);

/* AVERIS_ABI_VERSION of the built library. */
int averis_abi_version(void);

/* Text of the last HIP error an entry point on the calling thread returned
 * AVERIS_E_HIP for, or of the size check averis_split_quant_noalloc returned
 * AVERIS_E_WORKSPACE for ("" if none).  The string is owned by the library and is
 * valid until the next call on the same thread. */
const char* averis_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* AVERIS_H */
