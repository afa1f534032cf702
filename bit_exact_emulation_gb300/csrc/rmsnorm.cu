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
constexpr int kMaxThreads = 1024;             // to a row
// Vectors of a row that a thread holds: registers for two blocks of 512 threads at least.
template <int VEC> constexpr int kMaxPer = VEC == 1 ? 16 : 4;

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

// One vector of the output row: v * mul in its type.
template <class T, int VEC, bool SHIFT>
__device__ __forceinline__ void put(const NormArgs &a, int64_t row, int i, float (&v)[VEC], float mul) {
#pragma unroll
  for (int j = 0; j < VEC; j++) v[j] *= mul;
  if (a.out_fmt == MCEMU_INT8) {
    store_part<int8_t, VEC, SHIFT>((int8_t *)a.y + row * a.ldy, i, a.H, to_int8<VEC>(v));
  } else if (a.out_fmt == MCEMU_E4M3 || a.out_fmt == MCEMU_E5M2) {
    Vec<uint8_t, VEC> o;
    if constexpr (VEC == 1) {
      o.v[0] = __nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, a.out_fmt == MCEMU_E4M3 ? __NV_E4M3 : __NV_E5M2);
    } else if (a.out_fmt == MCEMU_E4M3) {
#pragma unroll
      for (int j = 0; j < VEC; j += 2)
        *(uint16_t *)&o.v[j] = __nv_cvt_float2_to_fp8x2(make_float2(v[j], v[j + 1]), __NV_SATFINITE, __NV_E4M3);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; j += 2)
        *(uint16_t *)&o.v[j] = __nv_cvt_float2_to_fp8x2(make_float2(v[j], v[j + 1]), __NV_SATFINITE, __NV_E5M2);
    }
    store_part<uint8_t, VEC, SHIFT>((uint8_t *)a.y + row * a.ldy, i, a.H, o);
  } else {
    store_part<T, VEC, SHIFT>((T *)a.y + row * a.ldy, i, a.H, pack<T, VEC>(v));
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
// blockDim.y rows to a block.  h is held in its own type and v = h * w computed twice: the
// registers of fp32 copies would halve the threads in flight, and with them the bandwidth (98 us
// in place of NORMNOW for 8192 x 8192 bf16 with a residual).  All of a thread's loads are issued before
// its first store (h may lie on x or res, so the compiler would keep them in order).
template <class T, int VEC, int PER, bool RES, bool SHIFT>
__global__ void __launch_bounds__(kMaxThreads) rmsnorm_kernel(const NormArgs a) {
  __shared__ float2 part[kMaxThreads / 32];
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < a.T;
  const T *px = (const T *)a.x + row * a.ldx, *pr = (const T *)a.res + row * a.ldr;
  const int back = SHIFT ? (int)(((uintptr_t)px / sizeof(T)) % VEC) : 0;     // of the first vector
  Vec<T, VEC> h[PER];
  float sum = 0.f, mx = 0.f;
  if (live) {
    Vec<T, VEC> r[PER];
#pragma unroll
    for (int p = 0; p < PER; p++) {
      const int i = (p * blockDim.x + threadIdx.x) * VEC - back;
      if (i < a.H) {
        h[p] = load_part<T, VEC, SHIFT>(px, i, a.H);
        if constexpr (RES) r[p] = load_part<T, VEC, SHIFT>(pr, i, a.H);
      }
    }
#pragma unroll
    for (int p = 0; p < PER; p++) {
      const int i = (p * blockDim.x + threadIdx.x) * VEC - back;
      if (i >= a.H) continue;
      if constexpr (RES) {
        h[p] = add_vec<T, VEC>(h[p], r[p]);
        store_part<T, VEC, SHIFT>((T *)a.h + row * a.ldh, i, a.H, h[p]);
      }
      float w[VEC], f[VEC];
      load_w_part<T, VEC, SHIFT>(a.w, a.w32, i, a.H, w);
      unpack<T, VEC>(h[p], f);
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        sum = fmaf(f[j], f[j], sum);
        mx = max_nan(mx, fabsf(f[j] * w[j]));
      }
    }
  }
  row_reduce(sum, mx, part);
  if (!live) return;
  const float mul = finish_row(a, row, sum, mx, threadIdx.x == 0);
#pragma unroll
  for (int p = 0; p < PER; p++) {
    const int i = (p * blockDim.x + threadIdx.x) * VEC - back;
    if (i >= a.H) continue;
    float w[VEC], f[VEC];
    load_w_part<T, VEC, SHIFT>(a.w, a.w32, i, a.H, w);
    unpack<T, VEC>(h[p], f);
#pragma unroll
    for (int j = 0; j < VEC; j++) w[j] *= f[j];
    put<T, VEC, SHIFT>(a, row, i, w, mul);
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
      x = add_vec<T, VEC>(x, load_vec<T, VEC>((const T *)a.res + row * a.ldr + i));
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
    put<T, VEC, false>(a, row, i, v, mul);
  }
}

struct Shape {
  int per, threads, rows;
};
// Threads to a row and vectors to a thread.  Many rows: as many vectors a thread as it can
// hold, so that it has several loads in flight; few rows: as many threads as the row feeds, for
// latency.
Shape shape_of(int T, int H, int vec, int max_per) {
  const int items = H / vec + (H % vec != 0);
  const int want = T >= 2 * sm_count() ? max_per : 1;
  int per = 1;
  while (per < max_per && (per < want || (items + per - 1) / per > kMaxThreads)) per *= 2;
  while (per > 1 && (items + per / 2 - 1) / (per / 2) <= 32) per /= 2;      // a warp is enough
  const int threads = ((items + per - 1) / per + 31) / 32 * 32;
  int rows = threads < 256 ? 256 / threads : 1;
  if (T < rows * sm_count()) rows = 1;
  return {per, threads, rows};
}

template <class T, int VEC, int PER, bool SHIFT>
void go(const NormArgs &a, const Shape &s, cudaStream_t st) {
  const dim3 grid((a.T + s.rows - 1) / s.rows), block(s.threads, s.rows);
  if (a.res) rmsnorm_kernel<T, VEC, PER, true, SHIFT><<<grid, block, 0, st>>>(a);
  else rmsnorm_kernel<T, VEC, PER, false, SHIFT><<<grid, block, 0, st>>>(a);
}

template <class T>
int norm_typed(const NormArgs &a, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const int ob = a.out_fmt == MCEMU_INT8 || a.out_fmt == MCEMU_E4M3 || a.out_fmt == MCEMU_E5M2 ? 1 : (int)sizeof(T);
  Walk walk{V};
  walk.add(a.x, a.ldx, sizeof(T));
  walk.add(a.res, a.ldr, sizeof(T));
  walk.add(a.h, a.ldh, sizeof(T));
  walk.add(a.y, a.ldy, ob);
  const bool wide = walk.ok && !walk.shifted() && a.H % V == 0 && rows16(a.w, 0, 4);
  // Vectors where every operand's rows lie alike against 16-byte boundaries (contiguous ones
  // do, whatever H); 8191 x 5003 bf16 with a residual: SHIFTNOW us, one element at a time 149.
  const bool shift = walk.ok && !wide && a.H >= 64;
  const int vec = wide || shift ? V : 1, max_per = wide || shift ? kMaxPer<V> : kMaxPer<1>;
  const int span = shift ? a.H + V - 1 : a.H;
  if ((int64_t)span > (int64_t)kMaxThreads * max_per * vec) {
    if (wide) rmsnorm_long_kernel<T, V><<<a.T, 512, 0, st>>>(a);
    else rmsnorm_long_kernel<T, 1><<<a.T, 512, 0, st>>>(a);
    return launch_status();
  }
  const Shape s = shape_of(a.T, span, vec, max_per);
  if (wide) {
    if (s.per == 1) go<T, V, 1, false>(a, s, st);
    else if (s.per == 2) go<T, V, 2, false>(a, s, st);
    else go<T, V, 4, false>(a, s, st);
  } else if (shift) {
    if (s.per <= 2) go<T, V, 2, true>(a, s, st);
    else go<T, V, 4, true>(a, s, st);
  } else {
    if (s.per <= 4) go<T, 1, 4, false>(a, s, st);
    else go<T, 1, 16, false>(a, s, st);
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
