// rmsnorm.cu -- root-mean-square norm with the residual's addition and an output in 8 bits
// with a scale for each token (include/mcemu_ops.h has the formulas).
//
// Bound by HBM: 7 bytes an element for bf16 rows with a residual, against some ten operations.
// A row lives in the registers of its threads between the one pass over memory that reads it
// and the one that writes it.
#include "norm_rows.cuh"
#include "ops_common.cuh"

namespace mcemu {
namespace {

constexpr float kAmaxFloor = 7.88860905221011805e-31f;   // 2^-100
constexpr int kMaxThreads = 1024;             // to a row
constexpr int kMaxPer = 4;                    // vectors of a row that a thread holds
constexpr int kSingles = 16;                  // elements a thread holds where no vector fits

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
template <class T, int VEC>
__device__ __forceinline__ void put(const NormArgs &a, int64_t row, int i, float (&v)[VEC], float mul) {
#pragma unroll
  for (int j = 0; j < VEC; j++) v[j] *= mul;
  if (a.out_fmt == MCEMU_INT8) {
    store_vec((int8_t *)a.y + row * a.ldy + i, to_int8<VEC>(v));
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
    store_vec((uint8_t *)a.y + row * a.ldy + i, o);
  } else {
    store_vec((T *)a.y + row * a.ldy + i, pack<T, VEC>(v));
  }
}

__device__ __forceinline__ float top_of(int out_fmt) {
  return out_fmt == MCEMU_INT8 ? 127.f : out_fmt == MCEMU_E4M3 ? 448.f : 57344.f;
}

// 1 / sqrt(mean(h^2) + eps) from sums in fp64, whose range holds the squares of all that fp32 holds and
// their sums.  Every warp goes through the whole row as it is stored, which its threads wrote
// before they joined their sums: no barrier is needed, and all warps have the same bits.  The sum s is
// brought to [1, 4) by 2^-2k, so that the root and the quotients are fp32's.
template <class T>
__device__ __forceinline__ float rstd_of_any_row(const T *h, int H, float eps) {
  double s = 0;
  __syncwarp();
#pragma unroll 1
  for (int i = threadIdx.x & 31; i < H; i += 32) {
    const double f = to_f(h[i]);
    s = fma(f, f, s);
  }
#pragma unroll 1
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  s = fma((double)eps, (double)H, s);
  const int k = max(-200, min(200, ((__double2hiint(s) >> 20 & 0x7FF) - 1023) >> 1));
  const float x = (float)(s * __hiloint2double((1023 - 2 * k) << 20, 0));
  return (float)(__hiloint2double((1023 - k) << 20, 0) * (double)(1.f / sqrtf(x / (float)H)));
}

// A call in place of the code itself costs nothing where a block takes one row, and the code itself
// nothing where it walks over rows: 300 x 777 fp32 2.44 us against 3.2, 8191 x 5003 bf16 90 against 71.
template <class T>
__device__ __noinline__ float rstd_of_any_row_apart(const T *h, int H, float eps) { return rstd_of_any_row(h, H, eps); }

// What fp32's sum of squares is good for: beyond it the sum overflows, and below (2^-100) the denormal
// numbers' steps of 2^-149 begin to count.  A row outside (which takes values beyond 10^18, or a tiny
// eps) or one that is not finite is added up again.  The vote says to the compiler what is true anyway,
// that a warp's threads agree.
template <class T, bool WALK>
__device__ __forceinline__ float rstd_of(const NormArgs &a, int64_t row, float sum) {
  const float mean = sum / (float)a.H + a.eps;
  if (__any_sync(0xFFFFFFFFu, !(mean >= kAmaxFloor && mean <= 3.4028235e38f))) {
    const T *h = a.res ? (const T *)a.h + row * a.ldh : (const T *)a.x + row * a.ldx;
    return WALK ? rstd_of_any_row(h, a.H, a.eps) : rstd_of_any_row_apart(h, a.H, a.eps);
  }
  return 1.f / sqrtf(mean);
}

// Writes a row's rstd and scale; what its v = h * w are multiplied by.  8-bit values do not depend on
// rstd, and only the row's first warp waits for it.
template <class T, bool WALK = false>
__device__ __forceinline__ float finish_row(const NormArgs &a, int64_t row, float sum, float mx) {
  if (a.scale && (a.out_fmt == MCEMU_INT8 || a.out_fmt == MCEMU_E4M3 || a.out_fmt == MCEMU_E5M2)) {
    const float top = top_of(a.out_fmt), A = max_nan(mx, kAmaxFloor);
    if (threadIdx.x < 32) {
      const float rstd = rstd_of<T, WALK>(a, row, sum);
      if (threadIdx.x == 0) {
        if (a.rstd) a.rstd[row] = rstd;
        a.scale[row] = A * rstd / top;
      }
    }
    return top / A;
  }
  const float rstd = rstd_of<T, WALK>(a, row, sum);
  if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
  return rstd;
}

// A row in the registers of blockDim.x threads, PER vectors of VEC elements each;
// blockDim.y rows to a block.  h is held in its own type and v = h * w computed twice: the
// registers of fp32 copies would halve the threads in flight, and with them the bandwidth (98 us
// in place of 72 for 8192 x 8192 bf16 with a residual).  All of a thread's loads are issued before
// its first store (h may lie on x or res, so the compiler would keep them in order).  MOST threads to a
// block: 256, five blocks of which are to fit, without a residual where a row takes so few (8192 x
// 4096 bf16 27.2 us; 64 registers in place of 48: 28.8), else kMaxThreads.
template <class T, int VEC, int PER, bool RES, int MOST>
__global__ void __launch_bounds__(MOST, MOST == 256 ? 5 : 0) rmsnorm_kernel(const NormArgs a) {
  __shared__ float2 part[kMaxThreads / 32];
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < a.T;
  const T *px = (const T *)a.x + row * a.ldx, *pr = (const T *)a.res + row * a.ldr;
  Vec<T, VEC> h[PER];
  float sum = 0.f, mx = 0.f;
  if (live) {
    Vec<T, VEC> r[PER];
#pragma unroll
    for (int p = 0; p < PER; p++) {
      const int i = (p * blockDim.x + threadIdx.x) * VEC;
      if (i < a.H) {
        h[p] = load_vec<T, VEC>(px + i);
        if constexpr (RES) r[p] = load_vec<T, VEC>(pr + i);
      }
    }
#pragma unroll
    for (int p = 0; p < PER; p++) {
      const int i = (p * blockDim.x + threadIdx.x) * VEC;
      if (i >= a.H) continue;
      if constexpr (RES) {
        h[p] = add_vec<T, VEC>(h[p], r[p]);
        store_vec((T *)a.h + row * a.ldh + i, h[p]);
      }
      float w[VEC], f[VEC];
      load_w<T, VEC>(a.w, a.w32, i, w);
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
  const float mul = finish_row<T>(a, row, sum, mx);
#pragma unroll
  for (int p = 0; p < PER; p++) {
    const int i = (p * blockDim.x + threadIdx.x) * VEC;
    if (i >= a.H) continue;
    float w[VEC], f[VEC];
    load_w<T, VEC>(a.w, a.w32, i, w);
    unpack<T, VEC>(h[p], f);
#pragma unroll
    for (int j = 0; j < VEC; j++) w[j] *= f[j];
    put<T, VEC>(a, row, i, w, mul);
  }
}

// Rows that no vector fits: one element of every TX to a thread, at distances that the compiler
// knows (with TX a variable the address of every access is computed anew: 8191 x 5003 bf16 with a
// residual 149 us in place of 85).
template <class T, int TX, bool RES>
__global__ void __launch_bounds__(TX < 256 ? 256 : TX) single_kernel(const NormArgs a) {
  __shared__ float2 part[kMaxThreads / 32];
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int left = row < a.T ? a.H - (int)threadIdx.x : 0;       // elements p with p * TX < left
  const int64_t i0 = threadIdx.x;
  const T *px = (const T *)a.x + row * a.ldx + i0, *pr = (const T *)a.res + row * a.ldr + i0;
  T h[kSingles], r[kSingles];
  float v[kSingles], sum = 0.f, mx = 0.f;
#pragma unroll
  for (int p = 0; p < kSingles; p++) {
    if (p * TX >= left) continue;
    h[p] = px[p * TX];
    if constexpr (RES) r[p] = pr[p * TX];
  }
#pragma unroll
  for (int p = 0; p < kSingles; p++)
    if (p * TX < left) v[p] = a.w32 ? ((const float *)a.w)[i0 + p * TX] : to_f(((const T *)a.w)[i0 + p * TX]);
  T *ph = (T *)a.h + row * a.ldh + i0;
#pragma unroll
  for (int p = 0; p < kSingles; p++) {
    if (p * TX >= left) continue;
    if constexpr (RES) {
      h[p] = from_f<T>(to_f(h[p]) + to_f(r[p]));
      ph[p * TX] = h[p];
    }
    const float f = to_f(h[p]);
    sum = fmaf(f, f, sum);
    v[p] *= f;
    mx = max_nan(mx, fabsf(v[p]));
  }
  row_reduce(sum, mx, part);
  if (row >= a.T) return;
  const float mul = finish_row<T>(a, row, sum, mx);
#pragma unroll
  for (int p = 0; p < kSingles; p++) {
    if (p * TX >= left) continue;
    float o[1] = {v[p]};
    put<T, 1>(a, row, (int)i0 + p * TX, o, mul);
  }
}

// The same for many rows (two to a multiprocessor at least; fewer are as fast the other way, 300 x 777
// fp32 2.7 us against 2.9): a block walks over rows, its columns' weights in registers, and copies
// the next row to shared memory meanwhile in whole units.  Columns beyond a row are zeros there.
// bf16 with a residual to int8, against one row to a block: 8191 x 5003 71 us, 84; 8191 x 4099 63,
// 79; 16384 x 1025 34, 47.
constexpr int kWalk = 8;                      // elements a thread holds

template <class T, int TX, bool RES>
__global__ void __launch_bounds__(TX) walk_kernel(const NormArgs a) {
  using R = Rows<TX, kWalk, (int)sizeof(T)>;
  constexpr int kStage = (RES ? 2 : 1) * R::kPitch;
  __shared__ float2 part[2][32];
  extern __shared__ __align__(16) uint8_t raw[];
  const int i0 = threadIdx.x, left = a.H - i0, lane = threadIdx.x & 31;
  float w[kWalk];
#pragma unroll
  for (int p = 0; p < kWalk; p++)
    w[p] = p * TX >= left ? 0.f : a.w32 ? ((const float *)a.w)[i0 + p * TX] : to_f(((const T *)a.w)[i0 + p * TX]);
  R xs(a.x, a.ldx, a.H), rs(a.res, a.ldr, a.H);
  const auto fetch = [&](uint8_t *to) {
    xs.fetch(to);
    if constexpr (RES) rs.fetch(to + R::kPitch);
  };
  int64_t row = blockIdx.x;
  if (row < a.T) fetch(raw);
  copy_commit();
  for (int s = 0; row < a.T; row += gridDim.x, s ^= 1) {
    const uint8_t *cur = raw + s * kStage;
    const T *x = (const T *)(cur + xs.off) + i0, *r = (const T *)(cur + R::kPitch + rs.off) + i0;
    copy_wait<0>();
    __syncthreads();                          // this row is there, and the one before is done with
    if (row + gridDim.x < a.T) fetch(raw + (s ^ 1) * kStage);
    copy_commit();
    T *ph = (T *)a.h + row * a.ldh + i0;
    float v[kWalk], sum = 0.f, mx = 0.f;
#pragma unroll
    for (int p = 0; p < kWalk; p++) {
      T h = x[p * TX];
      if constexpr (RES) {
        h = from_f<T>(to_f(h) + to_f(r[p * TX]));
        if (p * TX < left) ph[p * TX] = h;
      }
      const float f = to_f(h);
      sum = fmaf(f, f, sum);
      v[p] = f * w[p];
      mx = max_nan(mx, fabsf(v[p]));
    }
    sum = warp_sum(sum);
    mx = warp_max(mx);
    if constexpr (TX > 32) {
      if (lane == 0) part[s][threadIdx.x >> 5] = make_float2(sum, mx);
      __syncthreads();
      const float2 one = lane < TX / 32 ? part[s][lane] : make_float2(0.f, 0.f);
      sum = warp_sum(one.x);
      mx = warp_max(one.y);
    }
    const float mul = finish_row<T, true>(a, row, sum, mx);
    if (a.out_fmt == MCEMU_INT8) {
      int8_t *py = (int8_t *)a.y + row * a.ldy + i0;
#pragma unroll
      for (int p = 0; p < kWalk; p++)
        if (p * TX < left) {
          const float o[1] = {v[p] * mul};
          py[p * TX] = to_int8<1>(o).v[0];
        }
    } else {
#pragma unroll
      for (int p = 0; p < kWalk; p++) {
        float o[1] = {v[p]};
        if (p * TX < left) put<T, 1>(a, row, i0 + p * TX, o, mul);
      }
    }
  }
}

// Longer rows: a block of 1024 threads to a row, h read a second time.  A vector's squares are added up
// on their own, so that no thread adds more than H / 1024 numbers in a row.
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
    float w[VEC], some = 0.f;
    load_w<T, VEC>(a.w, a.w32, i, w);
#pragma unroll
    for (int j = 0; j < VEC; j++) {
      const float h = to_f(x.v[j]);
      some = fmaf(h, h, some);
      mx = max_nan(mx, fabsf(h * w[j]));
    }
    sum += some;
  }
  row_reduce(sum, mx, part);
  const float mul = finish_row<T>(a, row, sum, mx);
  const T *src = a.res ? (const T *)a.h + row * a.ldh : (const T *)a.x + row * a.ldx;
  for (int i = threadIdx.x * VEC; i < a.H; i += blockDim.x * VEC) {
    const Vec<T, VEC> x = load_vec<T, VEC>(src + i);
    float v[VEC], w[VEC];
    load_w<T, VEC>(a.w, a.w32, i, w);
#pragma unroll
    for (int j = 0; j < VEC; j++) v[j] = to_f(x.v[j]) * w[j];
    put<T, VEC>(a, row, i, v, mul);
  }
}

// Threads to a row and vectors to a thread.  Many rows: as many vectors a thread as it can
// hold, so that it has several loads in flight; few rows: as many threads as the row feeds, for
// latency.
template <class T, int VEC, int PER>
void go(const NormArgs &a, int items, cudaStream_t st) {
  const int threads = ((items + PER - 1) / PER + 31) / 32 * 32;
  int rows = threads < 256 ? 256 / threads : 1;
  if (a.T < rows * sm_count()) rows = 1;
  const dim3 grid((a.T + rows - 1) / rows), block(threads, rows);
  if constexpr (PER == kMaxPer)
    if (!a.res && threads * rows <= 256) {
      rmsnorm_kernel<T, VEC, PER, false, 256><<<grid, block, 0, st>>>(a);
      return;
    }
  if (a.res) rmsnorm_kernel<T, VEC, PER, true, kMaxThreads><<<grid, block, 0, st>>>(a);
  else rmsnorm_kernel<T, VEC, PER, false, kMaxThreads><<<grid, block, 0, st>>>(a);
}
template <class T, int VEC>
void go_vectors(const NormArgs &a, cudaStream_t st) {
  const int items = a.H / VEC;
  const bool many = a.T >= 2 * sm_count();
  if (items <= 32 || (items <= kMaxThreads && !many)) go<T, VEC, 1>(a, items, st);
  else if (items <= 64 || (items <= 2 * kMaxThreads && !many)) go<T, VEC, 2>(a, items, st);
  else go<T, VEC, kMaxPer>(a, items, st);
}

template <class T, int TX>
void go_single(const NormArgs &a, cudaStream_t st) {
  int rows = TX < 256 ? 256 / TX : 1;
  if (a.T < rows * sm_count()) rows = 1;
  const dim3 grid((a.T + rows - 1) / rows), block(TX, rows);
  if (a.res) single_kernel<T, TX, true><<<grid, block, 0, st>>>(a);
  else single_kernel<T, TX, false><<<grid, block, 0, st>>>(a);
}
template <class T>
void go_singles(const NormArgs &a, cudaStream_t st) {
  const int threads = (a.H + kSingles - 1) / kSingles;
  if (threads <= 32) go_single<T, 32>(a, st);
  else if (threads <= 64) go_single<T, 64>(a, st);
  else if (threads <= 128) go_single<T, 128>(a, st);
  else if (threads <= 256) go_single<T, 256>(a, st);
  else if (threads <= 384) go_single<T, 384>(a, st);
  else if (threads <= 512) go_single<T, 512>(a, st);
  else if (threads <= 768) go_single<T, 768>(a, st);
  else go_single<T, 1024>(a, st);
}

// Steps between powers of two, since columns beyond the row are computed too (16384 x 1025 by 256
// threads 49 us, by 160 34).  Others than these were not measured; rows just above 512 and 1280 elements
// compute the most columns that they do not have (97 and 60 %).
template <class T, int TX, bool RES>
bool go_walk(const NormArgs &a, cudaStream_t st) {
  constexpr int kSmem = 2 * (RES ? 2 : 1) * Rows<TX, kWalk, (int)sizeof(T)>::kPitch;
  if (!allow_smem<walk_kernel<T, TX, RES>>(kSmem)) return false;
  const int most = sm_count() * (TX > 640 ? 1 : 1536 / TX > 16 ? 16 : 1536 / TX);
  walk_kernel<T, TX, RES><<<a.T < most ? a.T : most, TX, kSmem, st>>>(a);
  return true;
}
template <class T, int TX>
bool go_walk(const NormArgs &a, cudaStream_t st) {
  return a.res ? go_walk<T, TX, true>(a, st) : go_walk<T, TX, false>(a, st);
}
template <class T>
bool go_walks(const NormArgs &a, cudaStream_t st) {
  const int threads = (a.H + kWalk - 1) / kWalk;
  return threads <= 32    ? go_walk<T, 32>(a, st)
         : threads <= 64  ? go_walk<T, 64>(a, st)
         : threads <= 128 ? go_walk<T, 128>(a, st)
         : threads <= 160 ? go_walk<T, 160>(a, st)
         : threads <= 256 ? go_walk<T, 256>(a, st)
         : threads <= 320 ? go_walk<T, 320>(a, st)
         : threads <= 384 ? go_walk<T, 384>(a, st)
         : threads <= 512 ? go_walk<T, 512>(a, st)
         : threads <= 576 ? go_walk<T, 576>(a, st)
         : threads <= 640 ? go_walk<T, 640>(a, st)
         : threads <= 768 ? go_walk<T, 768>(a, st)
                          : go_walk<T, 1024>(a, st);
}

template <class T>
int norm_typed(const NormArgs &a, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const int ob = a.out_fmt == MCEMU_INT8 || a.out_fmt == MCEMU_E4M3 || a.out_fmt == MCEMU_E5M2 ? 1 : (int)sizeof(T);
  const bool wide = a.H % V == 0 && rows16(a.x, a.ldx, sizeof(T)) && rows16(a.res, a.ldr, sizeof(T)) &&
                    rows16(a.h, a.ldh, sizeof(T)) && rows16(a.w, 0, 4) && rows_on(a.y, a.ldy, ob, V * ob);
  if (wide && a.H <= kMaxThreads * kMaxPer * V) go_vectors<T, V>(a, st);
  else if (a.H <= kMaxThreads * kWalk && a.T >= 2 * sm_count()) {
    if (!go_walks<T>(a, st)) return MCEMU_ERR_CUDA;
  }
  else if (a.H <= kMaxThreads * kSingles) go_singles<T>(a, st);
  else if (wide) rmsnorm_long_kernel<T, V><<<a.T, kMaxThreads, 0, st>>>(a);
  else rmsnorm_long_kernel<T, 1><<<a.T, kMaxThreads, 0, st>>>(a);
  return launch_status();
}

}  // namespace

int launch_rmsnorm(int fmt, const NormArgs &a, void *stream) {
  cudaStream_t st = (cudaStream_t)stream;
  return fmt == MCEMU_FP32 ? norm_typed<float>(a, st) : fmt == MCEMU_FP16 ? norm_typed<__half>(a, st)
                                                                          : norm_typed<__nv_bfloat16>(a, st);
}

}  // namespace mcemu
