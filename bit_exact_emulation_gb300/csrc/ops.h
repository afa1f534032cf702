// ops.h -- host-side launchers of the 8-bit layer operators, called by the C ABI
// (ops_api.cu) after its argument checks.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/mcemu_ops.h"

namespace mcemu {

struct NormArgs {
  int T, H;
  const void *x, *res, *w;
  void *h, *y;
  int64_t ldx, ldr, ldh, ldy;
  float *scale, *rstd;
  float eps;
  int w32;      // weights in fp32 (else in the elements' type)
  int out_fmt;  // MCEMU_INT8, MCEMU_E4M3, MCEMU_E5M2, or the elements' type
};
int launch_rmsnorm(int fmt, const NormArgs &a, void *stream);

struct NormGradArgs {
  int T, H;
  const void *dy, *dres, *h, *w;
  const int8_t *q, *e;
  const float *rstd;
  void *dx;
  float *dw;
  int64_t lddy, lddr, ldh, ldq, lde, lddx;
  int w32;
};
size_t rmsnorm_backward_workspace(int T, int H);
int launch_rmsnorm_backward(int fmt, const NormGradArgs &a, void *ws, void *stream);

int launch_act8_compress(int fmt, int T, int H, const void *x, int64_t ldx, int8_t *q, int64_t ldq, int8_t *e,
                         int64_t lde, void *stream);
int launch_act8_expand(int fmt, int T, int H, const int8_t *q, int64_t ldq, const int8_t *e, int64_t lde, void *x,
                       int64_t ldx, void *stream);

struct LinearArgs {
  int M, N, K;
  const int8_t *x, *w;
  int64_t ldx, ldw, ldy;
  const float *sx, *sw, *bias;
  void *y;
  int out_fmt;
};
// Whether a bounded device wait of these kernels gave up since the last question.
int int8_linear_timeouts(cudaStream_t st, unsigned int *got);
// rows: every row of x and w starts on a 16-byte boundary.
size_t int8_linear_workspace(int M, int N, int K, bool rows);
int launch_int8_linear(const LinearArgs &a, bool rows, void *ws, void *stream);

struct WgradArgs {
  int T, N, K;
  const uint16_t *dy;
  const int8_t *q, *e;
  int64_t lddy, ldq, lde, lddw;
  void *dW;
  int out_fmt, accumulate;
};
int act8_wgrad_timeouts(cudaStream_t st, unsigned int *got);
// direct: every row of dy starts on a 16-byte boundary.
size_t act8_wgrad_workspace(int T, int N, int K, bool direct);
int launch_act8_wgrad(const WgradArgs &a, bool direct, void *ws, void *stream);

}  // namespace mcemu
