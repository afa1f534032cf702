// ops_common.cuh -- what the 8-bit layer operators' kernels share: vectors of elements
// in registers, warp and row reductions, launch bookkeeping.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

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

// A vector to fp32; 16-bit types a register's two halves at a time.
template <class T, int V>
__device__ __forceinline__ void unpack(const Vec<T, V> &x, float (&f)[V]) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value && V > 1) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const uint32_t u = *(const uint32_t *)&x.v[i];
      f[i] = __uint_as_float(u << 16);
      f[i + 1] = __uint_as_float(u & 0xFFFF0000u);
    }
  } else if constexpr (std::is_same<T, __half>::value && V > 1) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 p = __half22float2(*(const __half2 *)&x.v[i]);
      f[i] = p.x;
      f[i + 1] = p.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) f[i] = to_f(x.v[i]);
  }
}
// fp32 rounded to the type, 16-bit types in pairs.
template <class T, int V>
__device__ __forceinline__ Vec<T, V> pack(const float (&f)[V]) {
  Vec<T, V> r;
  if constexpr (std::is_same<T, __nv_bfloat16>::value && V > 1) {
#pragma unroll
    for (int i = 0; i < V; i += 2) *(__nv_bfloat162 *)&r.v[i] = __floats2bfloat162_rn(f[i], f[i + 1]);
  } else if constexpr (std::is_same<T, __half>::value && V > 1) {
#pragma unroll
    for (int i = 0; i < V; i += 2) *(__half2 *)&r.v[i] = __floats2half2_rn(f[i], f[i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) r.v[i] = from_f<T>(f[i]);
  }
  return r;
}

// Sums rounded to the type.  16-bit types in pairs: the sum of two such numbers rounds the same
// straight to the type as through fp32 (where fp32 would round, the smaller operand lies below
// half a step of the type).
template <class T, int V>
__device__ __forceinline__ Vec<T, V> add_vec(const Vec<T, V> &a, const Vec<T, V> &b) {
  Vec<T, V> r;
  if constexpr (sizeof(T) == 2 && V > 1) {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
#pragma unroll
    for (int i = 0; i < V; i += 2) *(T2 *)&r.v[i] = __hadd2_rn(*(const T2 *)&a.v[i], *(const T2 *)&b.v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) r.v[i] = from_f<T>(to_f(a.v[i]) + to_f(b.v[i]));
  }
  return r;
}

// Numbers of at most 2^22 in magnitude rounded to integers (ties to even) in the low bits of
// the result: 1.5 * 2^23 puts the units digit last.  Two full-rate instructions where a
// conversion is a quarter-rate one.
__device__ __forceinline__ uint32_t round_bits(float x) { return __float_as_uint(__fadd_rn(x, 12582912.f)); }
// Four of them to bytes.
__device__ __forceinline__ uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
// V numbers of at most 127 in magnitude to signed bytes (a NaN gives some byte).
template <int V>
__device__ __forceinline__ Vec<int8_t, V> to_int8(const float (&x)[V]) {
  Vec<int8_t, V> r;
  if constexpr (V == 1) {
    r.v[0] = (int8_t)__float2int_rn(x[0]);
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *(uint32_t *)&r.v[i] = bytes4(round_bits(x[i]), round_bits(x[i + 1]), round_bits(x[i + 2]), round_bits(x[i + 3]));
  }
  return r;
}

// Two fp32 operations at once, each rounded as its own (sm_100 and later).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(*(unsigned long long *)&d)
      : "l"(*(unsigned long long *)&a), "l"(*(unsigned long long *)&b), "l"(*(unsigned long long *)&c));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(*(unsigned long long *)&d)
      : "l"(*(unsigned long long *)&a), "l"(*(unsigned long long *)&b));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(*(unsigned long long *)&d)
      : "l"(*(unsigned long long *)&a), "l"(*(unsigned long long *)&b));
  return d;
}

// V signed bytes to fp32, exactly: a byte plus 128 as the last digits of 2^23, less 2^23 + 128.
template <int V>
__device__ __forceinline__ void bytes_to_f(const Vec<int8_t, V> &q, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = (float)q.v[0];
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const uint32_t b = *(const uint32_t *)&q.v[i] ^ 0x80808080u;
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const float2 u = make_float2(__uint_as_float(__byte_perm(b, 0x4B000000u, 0x7650 + j)),
                                     __uint_as_float(__byte_perm(b, 0x4B000000u, 0x7651 + j)));
        const float2 v = add2(u, make_float2(-8388736.f, -8388736.f));
        f[i + j] = v.x;
        f[i + j + 1] = v.y;
      }
    }
  }
}

// V weights from the i-th on, kept in fp32 (w32) or in T.
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
    unpack<T, VEC>(load_vec<T, VEC>((const T *)w + i), f);
  }
}

// Thirty-two bytes to a 32-byte boundary at once: a whole sector, where two 16-byte stores each
// write half of one.
__device__ __forceinline__ void store32(void *to, uint4 a, uint4 b) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
               "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// Asynchronous copies of 4, 8 or 16 bytes to shared memory by the thread that reads them there.
template <int BYTES>
__device__ __forceinline__ void copy_async(void *to, const void *from) {
  const uint32_t s = (uint32_t)__cvta_generic_to_shared(to);
  if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(from) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(s), "l"(from), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory"); }

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

// Lets a kernel have its dynamic shared memory, always the same; asked for once per device.
template <auto KERNEL>
bool allow_smem(int bytes) {
  static std::atomic<bool> ready[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev < 64 && ready[dev].load(std::memory_order_relaxed)) return true;
  if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  if (dev < 64) ready[dev].store(true, std::memory_order_relaxed);
  return true;
}

// A kernel that begins while the one before it on the stream still runs (programmatic dependent
// launch): its set-up overlaps, and grid_wait() in it waits for that kernel's end and results.
// The one before says with grid_go() that it may begin.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <class... P, class... A>
int launch_early(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) == cudaSuccess ? MCEMU_OK : MCEMU_ERR_CUDA;
}

inline int launch_status() { return cudaGetLastError() == cudaSuccess ? MCEMU_OK : MCEMU_ERR_CUDA; }

// A caller's workspace is aligned to 16 bytes, panels that store32 writes to 32: where they begin in
// one that is kPanelPad bytes longer.
constexpr size_t kPanelPad = 16;
inline uint8_t *panels_in(void *ws) { return (uint8_t *)(((uintptr_t)ws + 31) & ~(uintptr_t)31); }

// Whether a row-major operand's rows all start on 16-byte boundaries (an absent one does).
inline bool rows16(const void *p, int64_t ld, int elem_bytes) {
  return !p || (((uintptr_t)p & 15) == 0 && (ld * elem_bytes) % 16 == 0);
}
// The same for boundaries of n bytes.
inline bool rows_on(const void *p, int64_t ld, int elem_bytes, int n) {
  return !p || (((uintptr_t)p & (n - 1)) == 0 && (ld * elem_bytes) % n == 0);
}

}  // namespace mcemu
