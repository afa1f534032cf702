/*
 * mcemu_ops.h -- C ABI of the 8-bit layer operators of libmcemu.so: what stands
 * around the 8-bit matrix products of a language-model layer, on the GPU's own
 * arithmetic (the emulated units of mcemu.h take the same operands).
 *
 *   mcemu_rmsnorm            residual addition, root-mean-square norm, output in
 *                            8 bits with a scale for each token
 *   mcemu_int8_linear        product of 8-bit integers, a scale for each token
 *                            and each channel
 *   mcemu_act8_compress      activation checkpoint: int8 codes, a power-of-two
 *   mcemu_act8_expand        scale for each MCEMU_ACT8_BLOCK elements of a row
 *   mcemu_act8_wgrad         a linear layer's weight gradient from a checkpoint
 *   mcemu_rmsnorm_backward   the norm's gradients, from its input or a checkpoint
 *
 * Conventions are those of mcemu.h: every function returns an mcemu_status;
 * buffers, workspaces and the stream belong to the caller; calls are enqueued
 * on `stream` and return before the work finishes; argument checks are
 * synchronous and nothing is launched when one fails.  Matrices are row-major
 * with leading dimensions in elements, at least the row length; elements of a
 * row are contiguous.  Element pointers must be aligned to their element
 * (MCEMU_ERR_ALIGNMENT); rows that start on 16-byte boundaries take the widest
 * loads, others are read in the aligned units of 16 bytes that hold them, so
 * that up to 15 bytes before a buffer may be read (and are not used: they lie in
 * the same allocation).  Buffers do not overlap unless a function says so.  Sizes are at most
 * 2^31 - 65536, and the product's operands what 32 bits count in rows of 64
 * (MCEMU_ERR_UNSUPPORTED).  No result depends on the order in which blocks
 * run: the same call gives the same bits.
 */
#ifndef MCEMU_OPS_H
#define MCEMU_OPS_H
#include "mcemu.h"

#ifdef __cplusplus
extern "C" {
#endif

/* int32 sums as an output type (mcemu_int8_linear), beside mcemu.h's formats. */
enum { MCEMU_INT32 = 8 };

/* ---- root-mean-square norm ------------------------------------------------ */
/* For each of T rows of H elements:
 *
 *     h    = x + res, rounded to fmt (h = x without res)
 *     rstd = 1 / sqrt(mean(h^2) + eps)                       in fp32
 *     v    = h * w                                           in fp32
 *     out_fmt == fmt:   y = v * rstd, rounded to fmt
 *     INT8/E4M3/E5M2:   A = max(max|v|, 2^-100), P = 127 / 448 / 57344,
 *                       y = round(v * (P / A)), scale = A * rstd / P
 *
 * so that y * scale is the norm's output.  rstd cancels in y, which therefore
 * depends on no summation order: v, A, P / A and the product are single fp32
 * operations (round to nearest, ties to even, as is the rounding to 8 bits).
 * The norm acts on h as it is stored.  A row that holds a NaN or an infinity
 * (or meets one in w) gets a scale that is not finite, or NaN in y; so does a
 * row of zeros with eps = 0, whose rstd is infinite.  Every other row has its
 * rstd: where the squares or their sum leave fp32's range they are added up
 * in fp64.  What is left are results that fp32 does not hold: an rstd above
 * 2^128 is infinite, and so is a v beyond fp32; and 8-bit values of a row
 * whose v lie below 2^-100 lose digits, to zeros at last.
 * fmt: FP16, BF16 or FP32 (x, res, h); wfmt: fmt or FP32; out_fmt: fmt, INT8,
 * E4M3 or E5M2 (the OCP encodings).  res and h are given together or not at
 * all; h may be x or res (same leading dimension).  scale [T] is required for
 * 8-bit outputs and not touched otherwise; rstd [T] may be NULL.  eps >= 0.
 * T = 0 is a no-op; H >= 1. */
int mcemu_rmsnorm(int fmt, int wfmt, int out_fmt, int T, int H, const void *x, int64_t ldx, const void *res,
                  int64_t ldr, const void *w, float eps, void *h, int64_t ldh, void *y, int64_t ldy, float *scale,
                  float *rstd, void *stream);

/* Gradients of y = h * rstd * w (the rounding to 8 bits counts as the identity):
 *
 *     z  = h * rstd,  g = dy * w
 *     dx = rstd * (g - z * mean(g * z)) + dres, rounded to fmt
 *     dw = sum over the rows of dy * z                       fp32 [H]
 *
 * dx is the gradient of x and of res alike; dres, the gradient that reaches h
 * along the residual path, may be NULL.  h is given either in fmt (h, ldh) or as
 * a checkpoint (q, ldq, e, lde of mcemu_act8_compress), the other being NULL.
 * rstd [T] is mcemu_rmsnorm's.  dx may be dy or dres (same leading dimension).
 * workspace: mcemu_rmsnorm_backward_workspace(T, H) bytes, 16-byte aligned. */
int mcemu_rmsnorm_backward(int fmt, int wfmt, int T, int H, const void *dy, int64_t lddy, const void *dres,
                           int64_t lddr, const void *h, int64_t ldh, const int8_t *q, int64_t ldq, const int8_t *e,
                           int64_t lde, const float *rstd, const void *w, void *dx, int64_t lddx, float *dw,
                           void *workspace, size_t ws_bytes, void *stream);
size_t mcemu_rmsnorm_backward_workspace(int T, int H);

/* ---- product of 8-bit integers ---------------------------------------------- */
/* y[m][n] = ((float)acc * sx[m]) * sw[n] + bias[n], acc = sum_k x[m][k] * w[n][k]
 *
 * acc is the exact int32 sum (the integers that mcemu_tile_gemm gives for an
 * INT8 model with C = 0); its conversion, the two products and the addition are
 * each rounded to fp32, and the result to out_fmt (FP16, BF16 or FP32; to
 * nearest, ties to even).  bias (fp32) may be NULL.  out_fmt MCEMU_INT32 gives
 * acc itself; sx, sw and bias are then NULL.  x [M][K] (a token a row), w [N][K]
 * (a channel a row), sx [M], sw [N], y [M][N].  K <= 131071, so that no sum
 * overflows (else UNSUPPORTED); K = 0 gives sums of 0.
 * workspace: mcemu_int8_linear_workspace(M, N, K, rows_aligned) bytes, 16-byte
 * aligned; may be NULL where that is 0.  rows_aligned: 1 when every row of x and
 * of w starts on a 16-byte boundary (both pointers and leading dimensions are
 * multiples of 16), which needs less. */
int mcemu_int8_linear(int M, int N, int K, const int8_t *x, int64_t ldx, const float *sx, const int8_t *w,
                      int64_t ldw, const float *sw, const float *bias, int out_fmt, void *y, int64_t ldy,
                      void *workspace, size_t ws_bytes, void *stream);
size_t mcemu_int8_linear_workspace(int M, int N, int K, int rows_aligned);

/* ---- activation checkpoints ------------------------------------------------- */
/* Elements of a row that share one exponent; a row of H has ceil(H / 128). */
#define MCEMU_ACT8_BLOCK 128
/* Exponent of a block that holds a NaN or an infinity: reads back as NaN. */
#define MCEMU_ACT8_NAN (-128)
/* For each block of a row: e = the least integer >= -120 with
 * max|x| <= 127 * 2^e, and q = x * 2^-e rounded to the nearest integer (ties to
 * even).  A block of zeros has e = -7.  e is at most 121 (FP16: 9) and q at most
 * 127 in magnitude, so that the largest finite inputs stay finite.  q * 2^e has
 * seven significant bits: exact in bfloat16 and fp32.
 * x [T][H] in fmt (FP16, BF16 or FP32); q [T][H]; e [T][ceil(H/128)]. */
int mcemu_act8_compress(int fmt, int T, int H, const void *x, int64_t ldx, int8_t *q, int64_t ldq, int8_t *e,
                        int64_t lde, void *stream);
/* x = q * 2^e, rounded to fmt. */
int mcemu_act8_expand(int fmt, int T, int H, const int8_t *q, int64_t ldq, const int8_t *e, int64_t lde, void *x,
                      int64_t ldx, void *stream);
/* dW[n][k] = sum_t dy[t][n] * (q[t][k] * 2^e[t][k / 128])  (+ dW[n][k] when
 * accumulate = 1, FP32 only), for a linear layer y = x W^T with W [N][K] whose
 * input x [T][K] was kept as a checkpoint.  dy is BF16 [T][N]; dW is FP32 or BF16
 * [N][K].  Products are exact, sums are held in fp32, the result is rounded once.
 * workspace: mcemu_act8_wgrad_workspace(T, N, K, dy_rows_aligned) bytes, 16-byte
 * aligned; may be NULL where that is 0.  dy_rows_aligned: 1 when every row of dy
 * starts on a 16-byte boundary (the pointer is a multiple of 16, lddy of 8),
 * which needs less. */
int mcemu_act8_wgrad(int T, int N, int K, const uint16_t *dy, int64_t lddy, const int8_t *q, int64_t ldq,
                     const int8_t *e, int64_t lde, int out_fmt, int accumulate, void *dW, int64_t lddw,
                     void *workspace, size_t ws_bytes, void *stream);
size_t mcemu_act8_wgrad_workspace(int T, int N, int K, int dy_rows_aligned);

/* Waits for `stream`.  MCEMU_ERR_TIMEOUT when a wait inside one of the product
 * kernels gave up on the current device since the last call of this function
 * (each wait is bounded by two seconds; the results of that launch are not
 * valid), MCEMU_OK otherwise.  Synchronous; not needed for ordering. */
int mcemu_ops_check(void *stream);

#ifdef __cplusplus
}
#endif
#endif /* MCEMU_OPS_H */
