// act8.cu -- activation checkpoints in 8 bits: int8 codes with a power-of-two scale for each
// 128 elements of a row (include/mcemu_ops.h).
//
// Bound by HBM: 3 bytes an element from bf16.  The scale is a power of two so that a code
// times its scale has seven significant bits and is exact in bfloat16: the weight
// gradient's matrix operand needs no second rounding.
#include "ops_common.cuh"

namespace mcemu {
namespace {

constexpr int kBlock = MCEMU_ACT8_BLOCK;

// Largest exponent of a type: 127 * 2^e is finite in it.
template <class T> constexpr int kTopExp = 121;
template <> constexpr int kTopExp<__half> = 9;

// The least e >= -120 with amax <= 127 * 2^e, at most `top`; MCEMU_ACT8_NAN for a NaN or an
// infinity; -7 for a block of zeros.  amax = m * 2^(x - 127) with m in [1, 2) gives
// e = x - 127 - 6, one more when m > 127/64.
__device__ __forceinline__ int exponent_of(float amax, int top) {
  const uint32_t u = __float_as_uint(amax) & 0x7FFFFFFFu;
  if (u >= 0x7F800000u) return MCEMU_ACT8_NAN;
  if (u == 0) return -7;
  const int e = (int)(u >> 23) - 133 + ((u & 0x7FFFFFu) > 0x7E0000u);
  return e < -120 ? -120 : e > top ? top : e;
}
// 2^-e for e in [-120, 121]; 0 for a block that is not finite, whose codes do not matter.
__device__ __forceinline__ float inverse_of(int e) {
  return e == MCEMU_ACT8_NAN ? 0.f : __uint_as_float((uint32_t)(127 - e) << 23);
}
// x * 2^-e, kept within the codes' range: only a block at the top exponent can leave it.
__device__ __forceinline__ float code_of(float x, float inv) { return fminf(fmaxf(x * inv, -127.f), 127.f); }

// Largest magnitude of a vector.  16-bit types in pairs.
template <class T, int V>
__device__ __forceinline__ float amax_of(const Vec<T, V> &x) {
  if constexpr (sizeof(T) == 2) {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    T2 m = __habs2(*(const T2 *)&x.v[0]);
#pragma unroll
    for (int i = 2; i < V; i += 2) m = __hmax2_nan(m, __habs2(*(const T2 *)&x.v[i]));
    return max_nan(to_f(m.x), to_f(m.y));
  } else {
    float m = fabsf(x.v[0]);
#pragma unroll
    for (int i = 1; i < V; i++) m = max_nan(m, fabsf(x.v[i]));
    return m;
  }
}

// Blocks along the columns: the grid's second axis, which ends at 65535, and its third.  (One axis
// and a division in place of three: 70 us for 16384 x 8192 bf16 in place of 64.)
__device__ __forceinline__ int across() { return blockIdx.y + blockIdx.z * gridDim.y; }
dim3 grid_of(int high, int wide) {
  const int y = wide < 65535 ? wide : 65535;
  return dim3(high, y, (wide + y - 1) / y);
}

// blockDim.x * VEC columns by blockDim.y * kRows rows to a block of 256 threads, kRows rows to a
// thread so that as many loads are in flight; 128 / VEC neighbouring lanes share a block of 128.
constexpr int kRows = 4;

template <class T, int VEC>
__global__ void __launch_bounds__(256) compress_kernel(int T_, int H, const T *__restrict__ x, int64_t ldx,
                                                       int8_t *__restrict__ q, int64_t ldq, int8_t *__restrict__ e,
                                                       int64_t lde) {
  const int i = (across() * (int)blockDim.x + threadIdx.x) * VEC;
  const int64_t row0 = (int64_t)blockIdx.x * (blockDim.y * kRows) + threadIdx.y;
  Vec<T, VEC> v[kRows];
  bool in[kRows];
#pragma unroll
  for (int r = 0; r < kRows; r++) {
    const int64_t row = row0 + r * blockDim.y;
    in[r] = i < H && row < T_;
    if (in[r]) v[r] = load_vec<T, VEC>(x + row * ldx + i);
  }
#pragma unroll
  for (int r = 0; r < kRows; r++) {
    const int64_t row = row0 + r * blockDim.y;
    float amax = in[r] ? amax_of<T, VEC>(v[r]) : 0.f;
#pragma unroll
    for (int o = kBlock / VEC / 2; o; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    if (!in[r]) continue;
    const int ex = exponent_of(amax, kTopExp<T>);
    const float inv = inverse_of(ex);
    Vec<int8_t, VEC> o;
    if (ex == kTopExp<T>) {
      float c[VEC];
#pragma unroll
      for (int j = 0; j < VEC; j++) c[j] = code_of(to_f(v[r].v[j]), inv);
      o = to_int8<VEC>(c);
    } else {
      // a power of two scales without rounding, so that the sum with round_bits' constant may
      // be one fused operation
      uint32_t c[VEC];
      float f[VEC];
      unpack<T, VEC>(v[r], f);
#pragma unroll
      for (int j = 0; j < VEC; j++) c[j] = __float_as_uint(fmaf(f[j], inv, 12582912.f));
#pragma unroll
      for (int j = 0; j < VEC; j += 4) *(uint32_t *)&o.v[j] = bytes4(c[j], c[j + 1], c[j + 2], c[j + 3]);
    }
    store_vec(q + row * ldq + i, o);
    if (i % kBlock == 0) e[row * lde + i / kBlock] = (int8_t)ex;
  }
}

// Rows that no vector fits: a warp to a block of 128, element by element; eight blocks of a
// row by kRows rows to 256 threads.
template <class T>
__global__ void __launch_bounds__(256) compress_any_kernel(int T_, int H, const T *__restrict__ x, int64_t ldx,
                                                           int8_t *__restrict__ q, int64_t ldq, int8_t *__restrict__ e,
                                                           int64_t lde) {
  const int lane = threadIdx.x & 31, b = across() * 8 + (threadIdx.x >> 5);
  const int64_t row0 = (int64_t)blockIdx.x * kRows;
  if (b * kBlock >= H) return;
  T v[kRows][4];
#pragma unroll
  for (int r = 0; r < kRows; r++)
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int i = b * kBlock + j * 32 + lane;
      v[r][j] = i < H && row0 + r < T_ ? x[(row0 + r) * ldx + i] : from_f<T>(0.f);
    }
#pragma unroll
  for (int r = 0; r < kRows; r++) {
    const int64_t row = row0 + r;
    if (row >= T_) break;
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 4; j++) amax = max_nan(amax, fabsf(to_f(v[r][j])));
    amax = warp_max(amax);
    const int ex = exponent_of(amax, kTopExp<T>);
    const float inv = inverse_of(ex);
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int i = b * kBlock + j * 32 + lane;
      if (i < H) q[row * ldq + i] = (int8_t)__float2int_rn(code_of(to_f(v[r][j]), inv));
    }
    if (lane == 0) e[row * lde + b] = (int8_t)ex;
  }
}

template <class T, int VEC>
__global__ void __launch_bounds__(256) expand_kernel(int64_t tasks, int per_row, const int8_t *__restrict__ q,
                                                     int64_t ldq, const int8_t *__restrict__ e, int64_t lde,
                                                     T *__restrict__ x, int64_t ldx) {
  const int64_t task = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (task >= tasks) return;
  const int64_t row = task / per_row;
  const int i = (int)(task - row * per_row) * VEC;
  const Vec<int8_t, VEC> v = load_vec<int8_t, VEC>(q + row * ldq + i);
  const float s = act8_scale(e[row * lde + i / kBlock]);
  Vec<T, VEC> o;
#pragma unroll
  for (int j = 0; j < VEC; j++) o.v[j] = from_f<T>((float)v.v[j] * s);
  store_vec(x + row * ldx + i, o);
}

unsigned blocks_for(int64_t threads) { return (unsigned)((threads + 255) / 256); }

template <class T>
int compress_typed(int T_, int H, const void *x, int64_t ldx, int8_t *q, int64_t ldq, int8_t *e, int64_t lde,
                   cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  if (H % V == 0 && rows16(x, ldx, sizeof(T)) && rows_on(q, ldq, 1, V)) {
    const int items = H / V;
    int tx = 32;
    while (tx < 256 && tx < items) tx *= 2;
    const dim3 block(tx, 256 / tx);
    const int rows = 256 / tx * kRows;
    const dim3 grid = grid_of((T_ + rows - 1) / rows, (items + tx - 1) / tx);
    compress_kernel<T, V><<<grid, block, 0, st>>>(T_, H, (const T *)x, ldx, q, ldq, e, lde);
  } else {
    const dim3 grid = grid_of((T_ + kRows - 1) / kRows, (H + 8 * kBlock - 1) / (8 * kBlock));
    compress_any_kernel<T><<<grid, 256, 0, st>>>(T_, H, (const T *)x, ldx, q, ldq, e, lde);
  }
  return launch_status();
}

template <class T>
int expand_typed(int T_, int H, const int8_t *q, int64_t ldq, const int8_t *e, int64_t lde, void *x, int64_t ldx,
                 cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const bool wide = H % V == 0 && rows16(x, ldx, sizeof(T)) && rows_on(q, ldq, 1, V);
  const int per_row = wide ? H / V : H;
  const int64_t tasks = (int64_t)T_ * per_row;
  if ((tasks + 255) / 256 > INT32_MAX) return MCEMU_ERR_UNSUPPORTED;
  if (wide) expand_kernel<T, V><<<blocks_for(tasks), 256, 0, st>>>(tasks, per_row, q, ldq, e, lde, (T *)x, ldx);
  else expand_kernel<T, 1><<<blocks_for(tasks), 256, 0, st>>>(tasks, per_row, q, ldq, e, lde, (T *)x, ldx);
  return launch_status();
}

}  // namespace

int launch_act8_compress(int fmt, int T, int H, const void *x, int64_t ldx, int8_t *q, int64_t ldq, int8_t *e,
                         int64_t lde, void *stream) {
  cudaStream_t st = (cudaStream_t)stream;
  return fmt == MCEMU_FP32   ? compress_typed<float>(T, H, x, ldx, q, ldq, e, lde, st)
         : fmt == MCEMU_FP16 ? compress_typed<__half>(T, H, x, ldx, q, ldq, e, lde, st)
                             : compress_typed<__nv_bfloat16>(T, H, x, ldx, q, ldq, e, lde, st);
}

int launch_act8_expand(int fmt, int T, int H, const int8_t *q, int64_t ldq, const int8_t *e, int64_t lde, void *x,
                       int64_t ldx, void *stream) {
  cudaStream_t st = (cudaStream_t)stream;
  return fmt == MCEMU_FP32   ? expand_typed<float>(T, H, q, ldq, e, lde, x, ldx, st)
         : fmt == MCEMU_FP16 ? expand_typed<__half>(T, H, q, ldq, e, lde, x, ldx, st)
                             : expand_typed<__nv_bfloat16>(T, H, q, ldq, e, lde, x, ldx, st);
}

}  // namespace mcemu
