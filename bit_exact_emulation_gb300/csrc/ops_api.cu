// ops_api.cu -- the C ABI of the 8-bit layer operators (include/mcemu_ops.h): argument
// checks and dispatch into the kernels.  No function here computes a result on the host.
#include <cuda_runtime.h>

#include <cmath>

#include "ops.h"

using namespace mcemu;

namespace {

int bytes_of(int fmt) {
  return fmt == MCEMU_FP32 ? 4 : (fmt == MCEMU_FP16 || fmt == MCEMU_BF16) ? 2 : 1;
}
bool float_fmt(int fmt) { return fmt == MCEMU_FP16 || fmt == MCEMU_BF16 || fmt == MCEMU_FP32; }
bool known_fmt(int fmt) { return fmt >= MCEMU_FP16 && fmt <= MCEMU_INT32; }
// Sizes and what they are rounded up to are counted in 32 bits.
constexpr int kMost = INT32_MAX - 65535;
bool too_large(int a, int b, int c = 0) { return a > kMost || b > kMost || c > kMost; }
bool aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
int blocks_of(int h) { return h / MCEMU_ACT8_BLOCK + (h % MCEMU_ACT8_BLOCK != 0); }

// A caller's workspace against what the call needs.
int check_ws(const void *ws, size_t have, size_t need) {
  if (need == 0) return MCEMU_OK;
  if (have < need) return MCEMU_ERR_WORKSPACE;
  if (!ws) return MCEMU_ERR_INVALID_ARG;
  return aligned(ws, 16) ? MCEMU_OK : MCEMU_ERR_ALIGNMENT;
}

// A call's status; a CUDA error that it reports is taken from the runtime, where the next call's
// question after its own launches would find it.
int collected(int st) {
  if (st == MCEMU_ERR_CUDA) cudaGetLastError();
  return st;
}

}  // namespace

extern "C" int mcemu_rmsnorm(int fmt, int wfmt, int out_fmt, int T, int H, const void *x, int64_t ldx,
                             const void *res, int64_t ldr, const void *w, float eps, void *h, int64_t ldh, void *y,
                             int64_t ldy, float *scale, float *rstd, void *stream) {
  if (!known_fmt(fmt) || !known_fmt(wfmt) || !known_fmt(out_fmt)) return MCEMU_ERR_INVALID_ARG;
  const bool narrow = out_fmt == MCEMU_INT8 || out_fmt == MCEMU_E4M3 || out_fmt == MCEMU_E5M2;
  if (!float_fmt(fmt) || (wfmt != fmt && wfmt != MCEMU_FP32) || (!narrow && out_fmt != fmt))
    return MCEMU_ERR_UNSUPPORTED;
  if (T < 0 || H < 1 || !(eps >= 0.f) || std::isinf(eps)) return MCEMU_ERR_INVALID_ARG;
  if (too_large(T, H)) return MCEMU_ERR_UNSUPPORTED;
  if (T == 0) return MCEMU_OK;
  if (!x || !w || !y || (narrow && !scale) || !res != !h) return MCEMU_ERR_INVALID_ARG;
  if (ldx < H || ldy < H || (res && (ldr < H || ldh < H))) return MCEMU_ERR_INVALID_ARG;
  const size_t s = bytes_of(fmt);
  if (!aligned(x, s) || !aligned(res, s) || !aligned(h, s) || !aligned(w, bytes_of(wfmt)) ||
      !aligned(y, bytes_of(out_fmt)) || !aligned(scale, 4) || !aligned(rstd, 4))
    return MCEMU_ERR_ALIGNMENT;
  NormArgs a{T, H, x, res, w, h, y, ldx, ldr, ldh, ldy, scale, rstd, eps, wfmt == MCEMU_FP32, out_fmt};
  return collected(launch_rmsnorm(fmt, a, stream));
}

extern "C" size_t mcemu_rmsnorm_backward_workspace(int T, int H) {
  return T < 1 || H < 1 || too_large(T, H) ? 0 : rmsnorm_backward_workspace(T, H);
}

extern "C" int mcemu_rmsnorm_backward(int fmt, int wfmt, int T, int H, const void *dy, int64_t lddy,
                                      const void *dres, int64_t lddr, const void *h, int64_t ldh, const int8_t *q,
                                      int64_t ldq, const int8_t *e, int64_t lde, const float *rstd, const void *w,
                                      void *dx, int64_t lddx, float *dw, void *workspace, size_t ws_bytes,
                                      void *stream) {
  if (!known_fmt(fmt) || !known_fmt(wfmt)) return MCEMU_ERR_INVALID_ARG;
  if (!float_fmt(fmt) || (wfmt != fmt && wfmt != MCEMU_FP32)) return MCEMU_ERR_UNSUPPORTED;
  if (T < 0 || H < 1 || !dw) return MCEMU_ERR_INVALID_ARG;
  if (too_large(T, H)) return MCEMU_ERR_UNSUPPORTED;
  if (!aligned(dw, 4)) return MCEMU_ERR_ALIGNMENT;
  if (T == 0)
    return collected(cudaMemsetAsync(dw, 0, (size_t)H * 4, (cudaStream_t)stream) == cudaSuccess ? MCEMU_OK : MCEMU_ERR_CUDA);
  if (!dy || !w || !dx || !rstd || !q != !e || !h == !q) return MCEMU_ERR_INVALID_ARG;
  if (lddy < H || lddx < H || (dres && lddr < H) || (h && ldh < H) || (q && (ldq < H || lde < blocks_of(H))))
    return MCEMU_ERR_INVALID_ARG;
  const size_t s = bytes_of(fmt);
  if (!aligned(dy, s) || !aligned(dres, s) || !aligned(h, s) || !aligned(dx, s) || !aligned(w, bytes_of(wfmt)) ||
      !aligned(rstd, 4))
    return MCEMU_ERR_ALIGNMENT;
  const int st = check_ws(workspace, ws_bytes, rmsnorm_backward_workspace(T, H));
  if (st != MCEMU_OK) return st;
  NormGradArgs a{T, H, dy, dres, h, w, q, e, rstd, dx, dw, lddy, lddr, ldh, ldq, lde, lddx, wfmt == MCEMU_FP32};
  return collected(launch_rmsnorm_backward(fmt, a, workspace, stream));
}

extern "C" int mcemu_act8_compress(int fmt, int T, int H, const void *x, int64_t ldx, int8_t *q, int64_t ldq,
                                   int8_t *e, int64_t lde, void *stream) {
  if (!known_fmt(fmt)) return MCEMU_ERR_INVALID_ARG;
  if (!float_fmt(fmt)) return MCEMU_ERR_UNSUPPORTED;
  if (T < 0 || H < 1) return MCEMU_ERR_INVALID_ARG;
  if (too_large(T, H)) return MCEMU_ERR_UNSUPPORTED;
  if (T == 0) return MCEMU_OK;
  if (!x || !q || !e || ldx < H || ldq < H || lde < blocks_of(H)) return MCEMU_ERR_INVALID_ARG;
  if (!aligned(x, bytes_of(fmt))) return MCEMU_ERR_ALIGNMENT;
  return collected(launch_act8_compress(fmt, T, H, x, ldx, q, ldq, e, lde, stream));
}

extern "C" int mcemu_act8_expand(int fmt, int T, int H, const int8_t *q, int64_t ldq, const int8_t *e, int64_t lde,
                                 void *x, int64_t ldx, void *stream) {
  if (!known_fmt(fmt)) return MCEMU_ERR_INVALID_ARG;
  if (!float_fmt(fmt)) return MCEMU_ERR_UNSUPPORTED;
  if (T < 0 || H < 1) return MCEMU_ERR_INVALID_ARG;
  if (too_large(T, H)) return MCEMU_ERR_UNSUPPORTED;
  if (T == 0) return MCEMU_OK;
  if (!x || !q || !e || ldx < H || ldq < H || lde < blocks_of(H)) return MCEMU_ERR_INVALID_ARG;
  if (!aligned(x, bytes_of(fmt))) return MCEMU_ERR_ALIGNMENT;
  return collected(launch_act8_expand(fmt, T, H, q, ldq, e, lde, x, ldx, stream));
}

extern "C" size_t mcemu_int8_linear_workspace(int M, int N, int K, int rows_aligned) {
  return M < 1 || N < 1 || K < 1 || K > 131071 || too_large(M, N) ? 0 : int8_linear_workspace(M, N, K, rows_aligned != 0);
}

extern "C" int mcemu_int8_linear(int M, int N, int K, const int8_t *x, int64_t ldx, const float *sx,
                                 const int8_t *w, int64_t ldw, const float *sw, const float *bias, int out_fmt,
                                 void *y, int64_t ldy, void *workspace, size_t ws_bytes, void *stream) {
  if (!known_fmt(out_fmt)) return MCEMU_ERR_INVALID_ARG;
  if (!float_fmt(out_fmt) && out_fmt != MCEMU_INT32) return MCEMU_ERR_UNSUPPORTED;
  if (M < 0 || N < 0 || K < 0) return MCEMU_ERR_INVALID_ARG;
  if (K > 131071 || too_large(M, N)) return MCEMU_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return MCEMU_OK;
  if ((K > 0 && (!x || !w)) || !y) return MCEMU_ERR_INVALID_ARG;
  if (out_fmt == MCEMU_INT32 ? (sx || sw || bias) : (!sx || !sw)) return MCEMU_ERR_INVALID_ARG;
  if (ldx < K || ldw < K || ldy < N) return MCEMU_ERR_INVALID_ARG;
  const size_t s = out_fmt == MCEMU_INT32 ? 4 : bytes_of(out_fmt);
  if (!aligned(y, s) || !aligned(sx, 4) || !aligned(sw, 4) || !aligned(bias, 4)) return MCEMU_ERR_ALIGNMENT;
  const bool rows = aligned(x, 16) && aligned(w, 16) && ldx % 16 == 0 && ldw % 16 == 0;
  const int st = check_ws(workspace, ws_bytes, mcemu_int8_linear_workspace(M, N, K, rows));
  if (st != MCEMU_OK) return st;
  LinearArgs a{M, N, K, x, w, ldx, ldw, ldy, sx, sw, bias, y, out_fmt};
  return collected(launch_int8_linear(a, rows, workspace, stream));
}

extern "C" size_t mcemu_act8_wgrad_workspace(int T, int N, int K, int dy_rows_aligned) {
  return T < 1 || N < 1 || K < 1 || too_large(T, N, K) ? 0 : act8_wgrad_workspace(T, N, K, dy_rows_aligned != 0);
}

extern "C" int mcemu_act8_wgrad(int T, int N, int K, const uint16_t *dy, int64_t lddy, const int8_t *q, int64_t ldq,
                                const int8_t *e, int64_t lde, int out_fmt, int accumulate, void *dW, int64_t lddw,
                                void *workspace, size_t ws_bytes, void *stream) {
  if (!known_fmt(out_fmt) || (accumulate != 0 && accumulate != 1)) return MCEMU_ERR_INVALID_ARG;
  if ((out_fmt != MCEMU_FP32 && out_fmt != MCEMU_BF16) || (accumulate && out_fmt != MCEMU_FP32))
    return MCEMU_ERR_UNSUPPORTED;
  if (T < 0 || N < 0 || K < 0) return MCEMU_ERR_INVALID_ARG;
  if (too_large(T, N, K)) return MCEMU_ERR_UNSUPPORTED;
  if (N == 0 || K == 0) return MCEMU_OK;
  if ((T > 0 && (!dy || !q || !e)) || !dW) return MCEMU_ERR_INVALID_ARG;
  if (lddy < N || ldq < K || lde < blocks_of(K) || lddw < K) return MCEMU_ERR_INVALID_ARG;
  if (!aligned(dy, 2) || !aligned(dW, bytes_of(out_fmt))) return MCEMU_ERR_ALIGNMENT;
  const bool direct = aligned(dy, 16) && lddy % 8 == 0;
  const int st = check_ws(workspace, ws_bytes, mcemu_act8_wgrad_workspace(T, N, K, direct));
  if (st != MCEMU_OK) return st;
  WgradArgs a{T, N, K, dy, q, e, lddy, ldq, lde, lddw, dW, out_fmt, accumulate};
  return collected(launch_act8_wgrad(a, direct, workspace, stream));
}

extern "C" int mcemu_ops_check(void *stream) {
  unsigned int linear = 0, wgrad = 0;
  if (int8_linear_timeouts((cudaStream_t)stream, &linear) != MCEMU_OK ||
      act8_wgrad_timeouts((cudaStream_t)stream, &wgrad) != MCEMU_OK)
    return collected(MCEMU_ERR_CUDA);
  return linear || wgrad ? MCEMU_ERR_TIMEOUT : MCEMU_OK;
}
