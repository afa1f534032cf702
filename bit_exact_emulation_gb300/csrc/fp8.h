// fp8.h -- host-side launchers of the FP8 layer operators, called by the C ABI (fp8_api.cu)
// after its argument checks.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/mcemu_fp8.h"

namespace mcemu {

struct QuantArgs {
  int T, H, E;               // E: groups of rows, 1 without offsets
  const void *x;
  int64_t ldx;
  uint8_t *q, *qt;
  int8_t *e, *et;
  int64_t ldq, lde, ldqt, ldet;
  const int32_t *offsets;
  int out_fmt;
};
int launch_fp8_quantize(int fmt, const QuantArgs &a, void *stream);

struct QuantWeightArgs {
  int E, N, K;
  const void *w;
  int64_t ldw, w_stride;
  uint8_t *q, *qt;
  int64_t ldq, q_stride, ldqt, qt_stride;
  int8_t *e, *et;
  int out_fmt;
};
int launch_fp8_quantize_weight(int fmt, const QuantWeightArgs &a, void *stream);

// One operand of a product: `rows` rows (of each of its matrices) of K codes, exponents e[.][k / 128]
// for every row or (tile = 7) every 128 rows.
struct Fp8Operand {
  const uint8_t *q;
  const int8_t *e;
  int64_t ld, stride, lde, stride_e;
  int rows, tile, fmt;       // tile: a row's exponents are those of row >> tile
};

// y = a b^T: rows of a by rows of b.  Groups: of a's rows (by_k = 0; b has a matrix for each), or of
// blocks along k (by_k = 1; y has a matrix for each).  Without offsets all is one group.
struct Fp8Product {
  Fp8Operand a, b;
  int K, E, by_k;
  const int32_t *offsets;
  int T;                     // what offsets end at: a's rows, or by_k the columns (K too)
  const float *bias;
  void *y;
  int64_t ldy, stride_y;
  int out_fmt, accumulate;
  bool turned;               // a and b have changed places: y = b a^T, and the groups and `T` are b's
};
// a_rows, b_rows: every row of the operand starts on a 16-byte boundary (no copy of it is needed).
size_t fp8_product_workspace(int rows_a, int rows_b, int matrices_b, int K, bool a_rows, bool b_rows);
int launch_fp8_product(const Fp8Product &p, bool a_rows, bool b_rows, void *ws, void *stream);

// Whether a bounded device wait of the products' kernels gave up since the last question.
int fp8_pair_timeouts(cudaStream_t st, unsigned int *got);
int fp8_few_timeouts(cudaStream_t st, unsigned int *got);

}  // namespace mcemu
