// rmsnorm.cu -- root-mean-square norm with the residual's addition and an output in 8 bits
// with a scale for each token, and its gradients (include/mcemu_ops.h has the formulas).
//
// Both directions are bound by HBM: 7 bytes an element for bf16 rows with a residual,
// against some ten operations.  A row lives in the registers of its threads between the
// one pass over memory that reads it and the one that writes it.
#include "ops_common.cuh"

namespace mcemu {
namespace {

constexpr float kAmaxFloor = 7.88860905221011805e-31f;   // 2^-100
constexpr int kMaxThreads = 512, kMaxPerThread = 32;     // threads to a row, its elements a thread holds
constexpr int kMaxRow = kMaxThreads * kMaxPerThread;

template <class T, int VEC>
__device__ __forceinline__ void load_w(const void *w, int w32, int64_t i, float (&f)[VEC]) {
  if (w32) {
    if constexpr (VEC == 8) {
      const Vec<float, 4> lo = load_vec<float, 4>((const float *)w + i), hi = load_vec<float, 4>((const float *)w + i + 4);
#pragma unroll
      for (int j = 0; j < 4; j++) f[j] = lo.v[j], f[j + 4] = hi.v[j];
    } else {
      const Vec<float, VEC> x = load_vec<float, VEC>((const float *)w + i);
#pragma unroll
      for (int j = 0; j < VEC; j++) f[j] = x.v[j];
    }
  } else {
    const Vec<T, VEC> x = load_vec<T, VEC>((const T *)w + i);
#pragma unroll
    for (int j = 0; j < VEC; j++) f[j] = to_f(x.v[j]);
  }
}

// Sum and maximum over the threads of a row (blockDim.x of them, whole warps).
__device__ __forceinline__ void row_reduce(float &sum, float &mx, float2 *part) {
  sum = warp_sum(sum);
  mx = warp_max(mx);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  float2 *mine = part + threadIdx.y * warps;
  if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = make_float2(sum, mx);
  __syncthreads();
  sum = 0.f;
  mx = 0.f;
  for (int i = 0; i < warps; i++) {
    sum += mine[i].x;
    mx = max_nan(mx, mine[i].y);
  }
}

// One vector of v = h * w to the output type.
template <class T, int VEC>
__device__ __forceinline__ void put(int out_fmt, void *y, int64_t at, const float (&v)[VEC], float mul) {
  if (out_fmt == MCEMU_INT8) {
    Vec<int8_t, VEC> o;
#pragma unroll
    for (int j = 0; j < VEC; j++) o.v[j] = (int8_t)__float2int_rn(v[j] * mul);
    store_vec((int8_t *)y + at, o);
  } else if (out_fmt == MCEMU_E4M3 || out_fmt == MCEMU_E5M2) {
    Vec<uint8_t, VEC> o;
#pragma unroll
    for (int j = 0; j < VEC; j++)
      o.v[j] = __nv_cvt_float_to_fp8(v[j] * mul, __NV_SATFINITE, out_fmt == MCEMU_E4M3 ? __NV_E4M3 : __NV_E5M2);
    store_vec((uint8_t *)y + at, o);
  } else {
    Vec<T, VEC> o;
#pragma unroll
    for (int j = 0; j < VEC; j++) o.v[j] = from_f<T>(v[j] * mul);
    store_vec((T *)y + at, o);
  }
}

__device__ __forceinline__ float top_of(int out_fmt) {
  return out_fmt == MCEMU_INT8 ? 127.f : out_fmt == MCEMU_E4M3 ? 448.f : 57344.f;
}

__device__ __forceinline__ float finish_row(const NormArgs &a, int64_t row, float sum, float mx, bool lead) {
  const float rstd = 1.f / sqrtf(sum / (float)a.H + a.eps);
  const bool narrow = a.scale && (a.out_fmt == MCEMU_INT8 || a.out_fmt == MCEMU_E4M3 || a.out_fmt == MCEMU_E5M2);
  const float top = top_of(a.out_fmt), A = max_nan(mx, kAmaxFloor);
  if (lead) {
    if (a.rstd) a.rstd[row] = rstd;
    if (narrow) a.scale[row] = A * rstd / top;
  }
  return narrow ? top / A : rstd;
}

// A row in the registers of blockDim.x threads, PER vectors of VEC elements each;
// blockDim.y rows to a block.  All of a thread's loads are issued before its first store (h
// may lie on x or res, so the compiler would keep them in order).
template <class T, int VEC, int PER, bool RES>
__global__ void __launch_bounds__(kMaxThreads) rmsnorm_kernel(const NormArgs a) {
  __shared__ float2 part[kMaxThreads / 32];
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < a.T;
  float v[PER][VEC];
  float sum = 0.f, mx = 0.f;
  if (live) {
    Vec<T, VEC> x[PER], r[PER];
    const T *px = (const T *)a.x + row * a.ldx, *pr = (const T *)a.res + row * a.ldr;
#pragma unroll
    for (int p = 0; p < PER; p++) {
      const int i = (p * blockDim.x + threadIdx.x) * VEC;
      if (i < a.H) {
        x[p] = load_vec<T, VEC>(px + i);
        if constexpr (RES) r[p] = load_vec<T, VEC>(pr + i);
      }
    }
#pragma unroll
    for (int p = 0; p < PER; p++) {
      const int i = (p * blockDim.x + threadIdx.x) * VEC;
      if (i >= a.H) continue;
      if constexpr (RES) {
#pragma unroll
        for (int j = 0; j < VEC; j++) x[p].v[j] = from_f<T>(to_f(x[p].v[j]) + to_f(r[p].v[j]));
        store_vec((T *)a.h + row * a.ldh + i, x[p]);
      }
      float w[VEC];
      load_w<T, VEC>(a.w, a.w32, i, w);
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        const float h = to_f(x[p].v[j]);
        sum = fmaf(h, h, sum);
        v[p][j] = h * w[j];
        mx = max_nan(mx, fabsf(v[p][j]));
      }
    }
  }
  row_reduce(sum, mx, part);
  if (!live) return;
  const float mul = finish_row(a, row, sum, mx, threadIdx.x == 0);
#pragma unroll
  for (int p = 0; p < PER; p++) {
    const int i = (p * blockDim.x + threadIdx.x) * VEC;
    if (i < a.H) put<T, VEC>(a.out_fmt, a.y, row * a.ldy + i, v[p], mul);
  }
}

// Longer rows: a block to a row, h read a second time.
template <class T, int VEC>
__global__ void __launch_bounds__(kMaxThreads) rmsnorm_long_kernel(const NormArgs a) {
  __shared__ float2 part[kMaxThreads / 32];
  const int64_t row = blockIdx.x;
  float sum = 0.f, mx = 0.f;
  for (int i = threadIdx.x * VEC; i < a.H; i += blockDim.x * VEC) {
    Vec<T, VEC> x = load_vec<T, VEC>((const T *)a.x + row * a.ldx + i);
    if (a.res) {
      const Vec<T, VEC> r = load_vec<T, VEC>((const T *)a.res + row * a.ldr + i);
#pragma unroll
      for (int j = 0; j < VEC; j++) x.v[j] = from_f<T>(to_f(x.v[j]) + to_f(r.v[j]));
      store_vec((T *)a.h + row * a.ldh + i, x);
    }
    float w[VEC];
    load_w<T, VEC>(a.w, a.w32, i, w);
#pragma unroll
    for (int j = 0; j < VEC; j++) {
      const float h = to_f(x.v[j]);
      sum = fmaf(h, h, sum);
      mx = max_nan(mx, fabsf(h * w[j]));
    }
  }
  row_reduce(sum, mx, part);
  const float mul = finish_row(a, row, sum, mx, threadIdx.x == 0);
  const T *src = a.res ? (const T *)a.h + row * a.ldh : (const T *)a.x + row * a.ldx;
  for (int i = threadIdx.x * VEC; i < a.H; i += blockDim.x * VEC) {
    const Vec<T, VEC> x = load_vec<T, VEC>(src + i);
    float v[VEC], w[VEC];
    load_w<T, VEC>(a.w, a.w32, i, w);
#pragma unroll
    for (int j = 0; j < VEC; j++) v[j] = to_f(x.v[j]) * w[j];
    put<T, VEC>(a.out_fmt, a.y, row * a.ldy + i, v, mul);
  }
}

struct Shape {
  int per, threads, rows;
};
// Threads to a row and vectors to a thread.  Many rows: up to 32 elements a thread, so
// that a thread has several loads in flight; few rows: as many threads as the row feeds,
// for latency.
Shape shape_of(int T, int H, int vec, int max_per) {
  const int items = (H + vec - 1) / vec;
  const int want = T >= 2 * sm_count() ? max_per : 1;
  int per = 1;
  while (per < max_per && (per < want || (items + per - 1) / per > kMaxThreads)) per *= 2;
  while (per > 1 && (items + per / 2 - 1) / (per / 2) <= 32) per /= 2;      // a warp is enough
  const int threads = ((items + per - 1) / per + 31) / 32 * 32;
  int rows = threads < 256 ? 256 / threads : 1;
  if (T < rows * sm_count()) rows = 1;
  return {per, threads, rows};
}

template <class T, int VEC, int PER>
void go(const NormArgs &a, const Shape &s, cudaStream_t st) {
  const dim3 grid((a.T + s.rows - 1) / s.rows), block(s.threads, s.rows);
  if (a.res) rmsnorm_kernel<T, VEC, PER, true><<<grid, block, 0, st>>>(a);
  else rmsnorm_kernel<T, VEC, PER, false><<<grid, block, 0, st>>>(a);
}

template <class T>
int norm_typed(const NormArgs &a, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const int ob = a.out_fmt == MCEMU_INT8 || a.out_fmt == MCEMU_E4M3 || a.out_fmt == MCEMU_E5M2 ? 1 : (int)sizeof(T);
  const bool wide = a.H % V == 0 && rows16(a.x, a.ldx, sizeof(T)) && rows16(a.res, a.ldr, sizeof(T)) &&
                    rows16(a.h, a.ldh, sizeof(T)) && rows16(a.w, 0, 4) && rows_on(a.y, a.ldy, ob, V * ob);
  if (a.H > kMaxRow) {
    if (wide) rmsnorm_long_kernel<T, V><<<a.T, kMaxThreads, 0, st>>>(a);
    else rmsnorm_long_kernel<T, 1><<<a.T, kMaxThreads, 0, st>>>(a);
  } else if (wide) {
    const Shape s = shape_of(a.T, a.H, V, kMaxPerThread / V);
    if (s.per == 1) go<T, V, 1>(a, s, st);
    else if (s.per == 2) go<T, V, 2>(a, s, st);
    else if (s.per == 4 || V == 8) go<T, V, 4>(a, s, st);
    else go<T, V, 32 / V>(a, s, st);
  } else {
    const Shape s = shape_of(a.T, a.H, 1, kMaxPerThread);
    if (s.per <= 2) go<T, 1, 2>(a, s, st);
    else if (s.per <= 8) go<T, 1, 8>(a, s, st);
    else if (s.per == 16) go<T, 1, 16>(a, s, st);
    else go<T, 1, 32>(a, s, st);
  }
  return launch_status();
}

}  // namespace

int launch_rmsnorm(int fmt, const NormArgs &a, void *stream) {
  cudaStream_t st = (cudaStream_t)stream;
  return fmt == MCEMU_FP32 ? norm_typed<float>(a, st) : fmt == MCEMU_FP16 ? norm_typed<__half>(a, st)
                                                                          : norm_typed<__nv_bfloat16>(a, st);
}

}  // namespace mcemu
