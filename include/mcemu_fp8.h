/*
 * mcemu_fp8.h -- C ABI of the FP8 layer operators of libmcemu.so: matrix products
 * of 8-bit floating-point numbers that carry a scale, a power of two, for each
 * block of 128, for serving and for training, dense and grouped by expert.  They
 * run on the GPU's own matrix units (the emulated units of mcemu.h take the same
 * codes).
 *
 *   mcemu_fp8_quantize          operands from activations and gradients: blocks of
 *                               128 along a row, blocks of 128 rows of a column
 *   mcemu_fp8_quantize_weight   operands from weights: blocks of 128 x 128
 *   mcemu_fp8_linear            product of two operands
 *   mcemu_fp8_grouped_linear    rows grouped by expert, a weight for each group
 *   mcemu_fp8_grouped_wgrad     the groups' weight gradients
 *
 * A number is code * 2^e, e the exponent of its block (int8).  The scale is a
 * power of two because a floating code loses nothing by it and the matrix unit
 * applies it by itself.  e = MCEMU_FP8_NAN makes every number of the block NaN.
 *
 * Formats are MCEMU_E4M3 and MCEMU_E5M2 (the OCP encodings), for either operand
 * of a product.  Conventions are those of mcemu_ops.h: an mcemu_status from every
 * function, buffers and stream of the caller, row-major matrices with leading
 * dimensions in elements, synchronous argument checks, nothing launched when one
 * fails.  Sizes are at most 2^31 - 65536, and what a function says.  Results do
 * not depend on the order in which blocks run: the same call gives the same bits.
 *
 * Groups: offsets [E + 1] (int32, on the device) say where each group's rows
 * begin; group g has the rows offsets[g] to offsets[g + 1] - 1, none where they
 * are equal.  Offsets ascend within 0 .. T; one that does not counts as the
 * largest so far, one beyond T as T (nothing outside the buffers is read or
 * written).  1 <= E <= MCEMU_FP8_MAX_GROUPS.
 */
#ifndef MCEMU_FP8_H
#define MCEMU_FP8_H
#include "mcemu_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MCEMU_FP8_BLOCK 128
#define MCEMU_FP8_NAN (-128)
#define MCEMU_FP8_MAX_GROUPS 1024

/* ---- operands ----------------------------------------------------------------- */
/* For each block: e = the least integer >= -120 with max|x| <= P * 2^e, P = 448
 * (E4M3) or 57344 (E5M2); q = x * 2^-e rounded to the format (to nearest, ties to
 * even).  A block of zeros has e = -120.  A block that holds a NaN or an infinity
 * has e = MCEMU_FP8_NAN and codes 0x7F (NaN).
 *
 * x [T][H] in fmt (FP16, BF16 or FP32), H >= 1.
 * Rows (q and e, both NULL when not wanted): q [T][H], e [T][ceil(H / 128)], blocks
 * of 128 along a row.
 * Columns (qt and et, both NULL when not wanted): the transposed matrix qt [H][P],
 * et [H][P / 128], blocks of 128 rows of a column, P = mcemu_fp8_columns(T, E).
 * offsets NULL (E = 0): all rows are one group.  Each group begins a block: its rows
 * follow the ceil(n / 128) * 128 places of each group before it.  Places that no
 * row fills hold zeros (e = -120 where a block has no row at all); rows outside all
 * groups are left out.  This is what mcemu_fp8_grouped_wgrad takes, and for one
 * group mcemu_fp8_linear. */
int mcemu_fp8_quantize(int fmt, int out_fmt, int T, int H, const void *x, int64_t ldx, uint8_t *q, int64_t ldq,
                       int8_t *e, int64_t lde, uint8_t *qt, int64_t ldqt, int8_t *et, int64_t ldet, int E,
                       const int32_t *offsets, void *stream);
/* (T + 127 * max(E, 1)) / 128 * 128: room for T rows in any E groups. */
int64_t mcemu_fp8_columns(int T, int E);

/* The same for weights w [E][N][K], w_stride elements between matrices, in blocks of
 * 128 x 128: q [E][N][K] (q_stride between matrices) and e [E][ceil(N/128)][ceil(K/128)];
 * qt [E][K][N] and et [E][ceil(K/128)][ceil(N/128)], the same numbers transposed, both
 * NULL when not wanted.  e and et are dense. */
int mcemu_fp8_quantize_weight(int fmt, int out_fmt, int E, int N, int K, const void *w, int64_t ldw, int64_t w_stride,
                              uint8_t *q, int64_t ldq, int64_t q_stride, int8_t *e, uint8_t *qt, int64_t ldqt,
                              int64_t qt_stride, int8_t *et, void *stream);

/* ---- products ------------------------------------------------------------------ */
/* y[m][n] = sum_k (x[m][k] 2^ex[m][k/128]) (w[n][k] 2^ew[.][k/128]) + bias[n]
 *
 * x [M][K] and ex [M][ceil(K/128)].  w [N][K]; ew [ceil(N/128)][ceil(K/128)] with
 * w_tiles = 1 (ew[n/128][k/128]), [N][ceil(K/128)] with 0 (ew[n][k/128]).  Products
 * are exact; the matrix unit adds up runs of whole blocks, at most 512 along k (few
 * rows) or 1024 (many), with the sums of the emulated unit MCEMU_PRESET_B200_FP8, bit for
 * bit where the exponents are 0; the runs are added in fp32, then bias (fp32, may be
 * NULL), and the result is rounded once to out_fmt (FP16, BF16 or FP32).  How K is cut
 * into runs, and their order, go by the sizes, the width of the results, whether rows
 * are grouped and the device's number of multiprocessors, and by nothing else: a
 * 16-bit result need not be the fp32 call's, rounded.  accumulate = 1: the sum is added
 * to y (FP32 only, without bias; where the copy engine adds, numbers below 2^-126 count
 * as zeros).  K = 0 gives sums of 0.
 *   forward            x = activations' rows, w = weight's blocks
 *   input's gradient   x = dY's rows, w = the weight's transposed blocks
 *   weight's gradient  x = dY's columns, w = the activations' columns, w_tiles = 0
 * workspace: mcemu_fp8_linear_workspace(M, N, K, x_rows, w_rows) bytes, 16-byte
 * aligned; may be NULL where that is 0.  x_rows, w_rows: 1 when every row of the
 * operand starts on a 16-byte boundary (of a single row the pointer decides); an operand
 * of other rows is copied there. */
int mcemu_fp8_linear(int M, int N, int K, int x_fmt, const uint8_t *x, int64_t ldx, const int8_t *ex, int64_t ldex,
                     int w_fmt, const uint8_t *w, int64_t ldw, const int8_t *ew, int64_t ldew, int w_tiles,
                     const float *bias, int out_fmt, int accumulate, void *y, int64_t ldy, void *workspace,
                     size_t ws_bytes, void *stream);
size_t mcemu_fp8_linear_workspace(int M, int N, int K, int x_rows, int w_rows);

/* y[t][n] = sum_k (x[t][k] 2^ex[t][k/128]) (w[g][n][k] 2^ew[g][n/128][k/128]) for the
 * rows t of each group g; rows outside all groups are left as they are.  x [T][K], w
 * [E][N][K] (w_stride elements between matrices), ew dense [E][ceil(N/128)][ceil(K/128)].
 * w_rows: every row of every matrix starts on a 16-byte boundary. */
int mcemu_fp8_grouped_linear(int T, int E, int N, int K, int x_fmt, const uint8_t *x, int64_t ldx, const int8_t *ex,
                             int64_t ldex, int w_fmt, const uint8_t *w, int64_t ldw, int64_t w_stride, const int8_t *ew,
                             const int32_t *offsets, int out_fmt, void *y, int64_t ldy, void *workspace,
                             size_t ws_bytes, void *stream);
size_t mcemu_fp8_grouped_linear_workspace(int T, int E, int N, int K, int x_rows, int w_rows);

/* dW[g][n][k] = sum over the rows t of group g of dy[t][n] x[t][k]  (+ dW[g][n][k] when
 * accumulate = 1, FP32 only).  dy and x are the columns that mcemu_fp8_quantize gives
 * with the same T, E and offsets: dyt [N][P], edyt [N][P/128], xt [K][P], ext [K][P/128],
 * P a multiple of 128.  dW [E][N][K] in FP32, FP16 or BF16, dw_stride elements between
 * matrices; a group without rows gets zeros (accumulate = 1: keeps dW, bit for bit).  dy_rows, x_rows as above. */
int mcemu_fp8_grouped_wgrad(int P, int E, int N, int K, int dy_fmt, const uint8_t *dyt, int64_t lddyt,
                            const int8_t *edyt, int64_t ldedyt, int x_fmt, const uint8_t *xt, int64_t ldxt,
                            const int8_t *ext, int64_t ldext, const int32_t *offsets, int out_fmt, int accumulate,
                            void *dW, int64_t lddw, int64_t dw_stride, void *workspace, size_t ws_bytes, void *stream);
size_t mcemu_fp8_grouped_wgrad_workspace(int P, int E, int N, int K, int dy_rows, int x_rows);

/* Waits for `stream`.  MCEMU_ERR_TIMEOUT when a wait inside one of these products'
 * kernels gave up on the current device since the last call (see mcemu_ops_check). */
int mcemu_fp8_check(void *stream);

#ifdef __cplusplus
}
#endif
#endif /* MCEMU_FP8_H */
