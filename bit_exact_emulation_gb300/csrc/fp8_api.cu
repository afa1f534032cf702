// fp8_api.cu -- the C ABI of the FP8 layer operators (include/mcemu_fp8.h): argument checks and
// dispatch into the kernels.  No function here computes a result on the host.
#include <cuda_runtime.h>

#include "fp8.h"

using namespace mcemu;

namespace {

int bytes_of(int fmt) { return fmt == MCEMU_FP32 ? 4 : 2; }
bool float_fmt(int fmt) { return fmt == MCEMU_FP16 || fmt == MCEMU_BF16 || fmt == MCEMU_FP32; }
bool code_fmt(int fmt) { return fmt == MCEMU_E4M3 || fmt == MCEMU_E5M2; }
bool known_fmt(int fmt) { return fmt >= MCEMU_FP16 && fmt <= MCEMU_INT32; }
// Sizes and what they are rounded up to are counted in 32 bits.
constexpr int kMost = INT32_MAX - 65535;
bool too_large(int a, int b, int c = 0) { return a > kMost || b > kMost || c > kMost; }
bool aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool rows_of(const void *p, int64_t ld, int64_t stride = 0) { return aligned(p, 16) && ld % 16 == 0 && stride % 16 == 0; }
// A single row has no next one, and the pitch that the copy engine wants.
int64_t pitch_of(int rows, int K, int64_t ld) { return rows == 1 ? ((int64_t)K + 15) & ~(int64_t)15 : ld; }
int blocks_of(int n) { return n / MCEMU_FP8_BLOCK + (n % MCEMU_FP8_BLOCK != 0); }
bool bad_groups(int E) { return E < 1 || E > MCEMU_FP8_MAX_GROUPS; }

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

extern "C" int64_t mcemu_fp8_columns(int T, int E) {
  if (T < 0 || T > kMost || E < 0 || E > MCEMU_FP8_MAX_GROUPS) return 0;
  return ((int64_t)T + 127 * (E > 1 ? E : 1)) / MCEMU_FP8_BLOCK * MCEMU_FP8_BLOCK;
}

extern "C" int mcemu_fp8_quantize(int fmt, int out_fmt, int T, int H, const void *x, int64_t ldx, uint8_t *q, int64_t ldq,
                                  int8_t *e, int64_t lde, uint8_t *qt, int64_t ldqt, int8_t *et, int64_t ldet, int E,
                                  const int32_t *offsets, void *stream) {
  if (!known_fmt(fmt) || !known_fmt(out_fmt)) return MCEMU_ERR_INVALID_ARG;
  if (!float_fmt(fmt) || !code_fmt(out_fmt)) return MCEMU_ERR_UNSUPPORTED;
  if (T < 0 || H < 1 || !q != !e || !qt != !et || (!q && !qt)) return MCEMU_ERR_INVALID_ARG;
  if (!offsets ? E != 0 : bad_groups(E)) return MCEMU_ERR_INVALID_ARG;
  const int64_t columns = mcemu_fp8_columns(T, E);
  if (too_large(T, H) || (qt && columns > kMost)) return MCEMU_ERR_UNSUPPORTED;
  if (T == 0 && (!qt || columns == 0)) return MCEMU_OK;
  if ((T > 0 && !x) || ldx < H || (q && (ldq < H || lde < blocks_of(H))) ||
      (qt && (ldqt < columns || ldet < columns / MCEMU_FP8_BLOCK)))
    return MCEMU_ERR_INVALID_ARG;
  if (!aligned(x, bytes_of(fmt)) || !aligned(offsets, 4)) return MCEMU_ERR_ALIGNMENT;
  QuantArgs a{T, H, offsets ? E : 1, x, ldx, q, qt, e, et, ldq, lde, ldqt, ldet, offsets, out_fmt};
  return collected(launch_fp8_quantize(fmt, a, stream));
}

extern "C" int mcemu_fp8_quantize_weight(int fmt, int out_fmt, int E, int N, int K, const void *w, int64_t ldw,
                                         int64_t w_stride, uint8_t *q, int64_t ldq, int64_t q_stride, int8_t *e,
                                         uint8_t *qt, int64_t ldqt, int64_t qt_stride, int8_t *et, void *stream) {
  if (!known_fmt(fmt) || !known_fmt(out_fmt)) return MCEMU_ERR_INVALID_ARG;
  if (!float_fmt(fmt) || !code_fmt(out_fmt)) return MCEMU_ERR_UNSUPPORTED;
  if (bad_groups(E) || N < 0 || K < 0 || !qt != !et) return MCEMU_ERR_INVALID_ARG;
  if (too_large(N, K)) return MCEMU_ERR_UNSUPPORTED;
  if (N == 0 || K == 0) return MCEMU_OK;
  if (!w || !q || !e || ldw < K || ldq < K || (qt && ldqt < N)) return MCEMU_ERR_INVALID_ARG;
  if (E > 1 && (w_stride < (N - 1) * ldw + K || q_stride < (N - 1) * ldq + K || (qt && qt_stride < (K - 1) * ldqt + N)))
    return MCEMU_ERR_INVALID_ARG;
  if (!aligned(w, bytes_of(fmt))) return MCEMU_ERR_ALIGNMENT;
  QuantWeightArgs a{E, N, K, w, ldw, w_stride, q, qt, ldq, q_stride, ldqt, qt_stride, e, et, out_fmt};
  return collected(launch_fp8_quantize_weight(fmt, a, stream));
}

extern "C" size_t mcemu_fp8_linear_workspace(int M, int N, int K, int x_rows, int w_rows) {
  return M < 1 || N < 1 || K < 1 || too_large(M, N, K) ? 0 : fp8_product_workspace(M, N, 1, K, x_rows != 0, w_rows != 0);
}

extern "C" int mcemu_fp8_linear(int M, int N, int K, int x_fmt, const uint8_t *x, int64_t ldx, const int8_t *ex,
                                int64_t ldex, int w_fmt, const uint8_t *w, int64_t ldw, const int8_t *ew, int64_t ldew,
                                int w_tiles, const float *bias, int out_fmt, int accumulate, void *y, int64_t ldy,
                                void *workspace, size_t ws_bytes, void *stream) {
  if (!known_fmt(x_fmt) || !known_fmt(w_fmt) || !known_fmt(out_fmt) || (w_tiles != 0 && w_tiles != 1) ||
      (accumulate != 0 && accumulate != 1))
    return MCEMU_ERR_INVALID_ARG;
  if (!code_fmt(x_fmt) || !code_fmt(w_fmt) || !float_fmt(out_fmt) || (accumulate && out_fmt != MCEMU_FP32))
    return MCEMU_ERR_UNSUPPORTED;
  if (M < 0 || N < 0 || K < 0 || (accumulate && bias)) return MCEMU_ERR_INVALID_ARG;
  if (too_large(M, N, K)) return MCEMU_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return MCEMU_OK;
  if ((K > 0 && (!x || !w || !ex || !ew)) || !y) return MCEMU_ERR_INVALID_ARG;
  if (ldx < K || ldw < K || ldy < N || ldex < blocks_of(K) || ldew < blocks_of(K)) return MCEMU_ERR_INVALID_ARG;
  if (!aligned(y, bytes_of(out_fmt)) || !aligned(bias, 4)) return MCEMU_ERR_ALIGNMENT;
  ldx = pitch_of(M, K, ldx);
  ldw = pitch_of(N, K, ldw);
  const bool xr = rows_of(x, ldx), wr = rows_of(w, ldw);
  const int st = check_ws(workspace, ws_bytes, mcemu_fp8_linear_workspace(M, N, K, xr, wr));
  if (st != MCEMU_OK) return st;
  Fp8Product p{{x, ex, ldx, 0, ldex, 0, M, 0, x_fmt}, {w, ew, ldw, 0, ldew, 0, N, w_tiles ? 7 : 0, w_fmt},
               K, 1, 0, nullptr, M, bias, y, ldy, 0, out_fmt, accumulate};
  return collected(launch_fp8_product(p, xr, wr, workspace, stream));
}

extern "C" size_t mcemu_fp8_grouped_linear_workspace(int T, int E, int N, int K, int x_rows, int w_rows) {
  return T < 1 || N < 1 || K < 1 || bad_groups(E) || too_large(T, N, K)
             ? 0
             : fp8_product_workspace(T, N, E, K, x_rows != 0, w_rows != 0);
}

extern "C" int mcemu_fp8_grouped_linear(int T, int E, int N, int K, int x_fmt, const uint8_t *x, int64_t ldx,
                                        const int8_t *ex, int64_t ldex, int w_fmt, const uint8_t *w, int64_t ldw,
                                        int64_t w_stride, const int8_t *ew, const int32_t *offsets, int out_fmt, void *y,
                                        int64_t ldy, void *workspace, size_t ws_bytes, void *stream) {
  if (!known_fmt(x_fmt) || !known_fmt(w_fmt) || !known_fmt(out_fmt)) return MCEMU_ERR_INVALID_ARG;
  if (!code_fmt(x_fmt) || !code_fmt(w_fmt) || !float_fmt(out_fmt)) return MCEMU_ERR_UNSUPPORTED;
  if (T < 0 || N < 0 || K < 0 || bad_groups(E)) return MCEMU_ERR_INVALID_ARG;
  if (too_large(T, N, K)) return MCEMU_ERR_UNSUPPORTED;
  if (T == 0 || N == 0) return MCEMU_OK;
  if ((K > 0 && (!x || !w || !ex || !ew)) || !y || !offsets) return MCEMU_ERR_INVALID_ARG;
  if (ldx < K || ldw < K || ldy < N || ldex < blocks_of(K) || (E > 1 && w_stride < (N - 1) * ldw + K)) return MCEMU_ERR_INVALID_ARG;
  if (!aligned(y, bytes_of(out_fmt)) || !aligned(offsets, 4)) return MCEMU_ERR_ALIGNMENT;
  ldx = pitch_of(T, K, ldx);
  ldw = pitch_of(N, K, ldw);
  const bool xr = rows_of(x, ldx), wr = rows_of(w, ldw, E > 1 ? w_stride : 0);
  const int st = check_ws(workspace, ws_bytes, mcemu_fp8_grouped_linear_workspace(T, E, N, K, xr, wr));
  if (st != MCEMU_OK) return st;
  const int64_t ldew = blocks_of(K);
  Fp8Product p{{x, ex, ldx, 0, ldex, 0, T, 0, x_fmt}, {w, ew, ldw, w_stride, ldew, blocks_of(N) * ldew, N, 7, w_fmt},
               K, E, 0, offsets, T, nullptr, y, ldy, 0, out_fmt, 0};
  return collected(launch_fp8_product(p, xr, wr, workspace, stream));
}

extern "C" size_t mcemu_fp8_grouped_wgrad_workspace(int P, int E, int N, int K, int dy_rows, int x_rows) {
  return P < 1 || N < 1 || K < 1 || bad_groups(E) || too_large(P, N, K)
             ? 0
             : fp8_product_workspace(N, K, 1, P, dy_rows != 0, x_rows != 0);
}

extern "C" int mcemu_fp8_grouped_wgrad(int P, int E, int N, int K, int dy_fmt, const uint8_t *dyt, int64_t lddyt,
                                       const int8_t *edyt, int64_t ldedyt, int x_fmt, const uint8_t *xt, int64_t ldxt,
                                       const int8_t *ext, int64_t ldext, const int32_t *offsets, int out_fmt,
                                       int accumulate, void *dW, int64_t lddw, int64_t dw_stride, void *workspace,
                                       size_t ws_bytes, void *stream) {
  if (!known_fmt(dy_fmt) || !known_fmt(x_fmt) || !known_fmt(out_fmt) || (accumulate != 0 && accumulate != 1))
    return MCEMU_ERR_INVALID_ARG;
  if (!code_fmt(dy_fmt) || !code_fmt(x_fmt) || !float_fmt(out_fmt) || (accumulate && out_fmt != MCEMU_FP32))
    return MCEMU_ERR_UNSUPPORTED;
  if (P < 0 || P % MCEMU_FP8_BLOCK || N < 0 || K < 0 || bad_groups(E)) return MCEMU_ERR_INVALID_ARG;
  if (too_large(P, N, K)) return MCEMU_ERR_UNSUPPORTED;
  if (N == 0 || K == 0) return MCEMU_OK;
  if ((P > 0 && (!dyt || !xt || !edyt || !ext || !offsets)) || !dW) return MCEMU_ERR_INVALID_ARG;
  const int blocks = P / MCEMU_FP8_BLOCK;
  if (lddyt < P || ldxt < P || ldedyt < blocks || ldext < blocks || lddw < K || (E > 1 && dw_stride < (N - 1) * lddw + K))
    return MCEMU_ERR_INVALID_ARG;
  if (!aligned(dW, bytes_of(out_fmt)) || !aligned(offsets, 4)) return MCEMU_ERR_ALIGNMENT;
  lddyt = pitch_of(N, P, lddyt);
  ldxt = pitch_of(K, P, ldxt);
  const bool dr = rows_of(dyt, lddyt), xr = rows_of(xt, ldxt);
  const int st = check_ws(workspace, ws_bytes, mcemu_fp8_grouped_wgrad_workspace(P, E, N, K, dr, xr));
  if (st != MCEMU_OK) return st;
  Fp8Product p{{dyt, edyt, lddyt, 0, ldedyt, 0, N, 0, dy_fmt}, {xt, ext, ldxt, 0, ldext, 0, K, 0, x_fmt},
               P, E, 1, offsets, P, nullptr, dW, lddw, dw_stride, out_fmt, accumulate};
  return collected(launch_fp8_product(p, dr, xr, workspace, stream));
}

extern "C" int mcemu_fp8_check(void *stream) {
  unsigned int pair = 0, few = 0;
  if (fp8_pair_timeouts((cudaStream_t)stream, &pair) != MCEMU_OK || fp8_few_timeouts((cudaStream_t)stream, &few) != MCEMU_OK)
    return collected(MCEMU_ERR_CUDA);
  return pair || few ? MCEMU_ERR_TIMEOUT : MCEMU_OK;
}
