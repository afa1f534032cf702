// ops_common.cuh -- what the 8-bit layer operators' kernels share: vectors of elements
// in registers, warp and row reductions, launch bookkeeping.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>

#include "ops.h"

namespace mcemu {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// V consecutive elements moved as one access of V * sizeof(T) bytes (at most 16).
template <class T, int V>
struct alignas(sizeof(T) * V) Vec {
  T v[V];
};
template <class T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const T *p) { return *reinterpret_cast<const Vec<T, V> *>(p); }
template <class T, int V>
__device__ __forceinline__ void store_vec(T *p, const Vec<T, V> &x) { *reinterpret_cast<Vec<T, V> *>(p) = x; }

// Maximum that keeps a NaN (fmaxf drops it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = max_nan(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
  return x;
}

// Value of a checkpoint's exponent: 2^e, NaN for MCEMU_ACT8_NAN (e >= -120 otherwise).
__device__ __forceinline__ float act8_scale(int e) {
  return __int_as_float(e == MCEMU_ACT8_NAN ? 0x7FC00000 : (e + 127) << 23);
}

// Sixteen bytes of a row of K from k on, zeros beyond its end; any alignment, no access
// outside the row.
__device__ __forceinline__ uint4 row16(const int8_t *row, int k, int K, bool wide) {
  if (wide && k + 16 <= K) return __ldg((const uint4 *)(row + k));
  uint32_t w[4] = {0, 0, 0, 0};
  const int off = (int)((uintptr_t)(row + k) & 3);
  if (k >= off && k - off + 20 <= K) {          // five whole words around the sixteen bytes
    const uint32_t *p = (const uint32_t *)(row + k - off);
    uint32_t v[5];
#pragma unroll
    for (int i = 0; i < 5; i++) v[i] = __ldg(p + i);
#pragma unroll
    for (int i = 0; i < 4; i++) w[i] = __funnelshift_r(v[i], v[i + 1], 8 * off);
  } else {
#pragma unroll
    for (int i = 0; i < 16; i++)
      if (k + i < K) w[i >> 2] |= (uint32_t)(uint8_t)row[k + i] << (8 * (i & 3));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Multiprocessors of the current device, looked up once per device.
inline int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (dev < 64 && known[dev].load(std::memory_order_relaxed)) return known[dev].load(std::memory_order_relaxed);
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 1;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

inline int launch_status() { return cudaGetLastError() == cudaSuccess ? MCEMU_OK : MCEMU_ERR_CUDA; }

// Whether a row-major operand's rows all start on 16-byte boundaries (an absent one does).
inline bool rows16(const void *p, int64_t ld, int elem_bytes) {
  return !p || (((uintptr_t)p & 15) == 0 && (ld * elem_bytes) % 16 == 0);
}
// The same for boundaries of n bytes.
inline bool rows_on(const void *p, int64_t ld, int elem_bytes, int n) {
  return !p || (((uintptr_t)p & (n - 1)) == 0 && (ld * elem_bytes) % n == 0);
}

}  // namespace mcemu
