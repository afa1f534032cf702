// fp8_quant.cu -- FP8 operands with a power-of-two scale for each block of 128 (include/mcemu_fp8.h).
//
// Bound by HBM: 3 bytes an element from bf16, 4 where the transposed codes are wanted too; both
// come from one reading.
#include "fp8.h"
#include "ops_common.cuh"

namespace mcemu {
namespace {

constexpr int kBlock = MCEMU_FP8_BLOCK;

// The least e >= -120 with amax <= 1.75 * 2^(TOP + e); MCEMU_FP8_NAN for a NaN or an infinity.
// amax = m * 2^x with m in [1, 2) gives e = x - TOP, one more when m > 1.75.
template <int TOP>
__device__ __forceinline__ int exponent_of(float amax) {
  const uint32_t u = __float_as_uint(amax) & 0x7FFFFFFFu;
  if (u >= 0x7F800000u) return MCEMU_FP8_NAN;
  const int e = (int)(u >> 23) - 127 - TOP + ((u & 0x7FFFFFu) > 0x600000u);
  return e < -120 ? -120 : e;
}
// 2^-e for e in [-120, 120]; NaN, which gives the code 0x7F, for a block that is not finite.
__device__ __forceinline__ float inverse_of(int e) {
  return __uint_as_float(e == MCEMU_FP8_NAN ? 0x7FC00000u : (uint32_t)(127 - e) << 23);
}
struct E4M3 {
  static constexpr int kTop = 8;
  static constexpr __nv_fp8_interpretation_t kKind = __NV_E4M3;
};
struct E5M2 {
  static constexpr int kTop = 15;
  static constexpr __nv_fp8_interpretation_t kKind = __NV_E5M2;
};
// A power of two scales without rounding (what falls below fp32 is a zero code by far).
template <class F>
__device__ __forceinline__ uint32_t codes2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, F::kKind);
}
template <class F>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  return codes2<F>(a, b) | codes2<F>(c, d) << 16;
}

// Largest magnitude, a NaN kept.
template <class T, int V>
__device__ __forceinline__ float amax_of(const Vec<T, V> &x) {
  float f[V];
  unpack<T, V>(x, f);
  float m = fabsf(f[0]);
#pragma unroll
  for (int i = 1; i < V; i++) m = max_nan(m, fabsf(f[i]));
  return m;
}

// V elements of a row from column c on, zeros beyond H.
template <class T, int V>
__device__ __forceinline__ Vec<T, V> some(const T *row, int c, int H, bool wide) {
  Vec<T, V> r;
  constexpr int kEach = 16 / sizeof(T);
  if (wide && c + V <= H) {
#pragma unroll
    for (int i = 0; i < V; i += kEach) *(uint4 *)&r.v[i] = __ldg((const uint4 *)(row + c + i));
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) r.v[i] = c + i < H ? row[c + i] : from_f<T>(0.f);
  }
  return r;
}
// Eight bytes of a row from column c on, `left` of them in it.
__device__ __forceinline__ void put8(uint8_t *row, int c, int left, uint2 v, bool wide) {
  if (wide && left >= 8) {
    *(uint2 *)(row + c) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (i < left) row[c + i] = (uint8_t)((i < 4 ? v.x : v.y) >> (8 * (i & 3)));
  }
}

// ---- rows alone -------------------------------------------------------------------
// Sixteen lanes to a block of a row, eight elements each; kRows rows a thread.
constexpr int kRows = 2;
template <class T, class F>
__global__ void __launch_bounds__(256) rows_kernel(const QuantArgs a, int64_t tasks, int blocks, bool wide_in, bool wide_out) {
  grid_go();
  const int lane = threadIdx.x & 15;
  const int64_t task0 = ((int64_t)blockIdx.x * 16 + (threadIdx.x >> 4)) * kRows;
  Vec<T, 8> v[kRows];
#pragma unroll
  for (int i = 0; i < kRows; i++) {
    const int64_t task = task0 + i;
    if (task >= tasks) continue;
    const int64_t row = task / blocks;
    v[i] = some<T, 8>((const T *)a.x + row * a.ldx, (int)(task - row * blocks) * kBlock + 8 * lane, a.H, wide_in);
  }
#pragma unroll
  for (int i = 0; i < kRows; i++) {
    const int64_t task = task0 + i;
    const int64_t row = task / blocks;
    const int block = (int)(task - row * blocks), c = block * kBlock + 8 * lane;
    float amax = task < tasks ? amax_of<T, 8>(v[i]) : 0.f;
#pragma unroll
    for (int o = 8; o; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    if (task >= tasks) continue;
    const int e = exponent_of<F::kTop>(amax);
    const float s = inverse_of(e);
    float f[8];
    unpack<T, 8>(v[i], f);
    put8(a.q + row * a.ldq, c, a.H - c,
         make_uint2(codes4<F>(f[0] * s, f[1] * s, f[2] * s, f[3] * s), codes4<F>(f[4] * s, f[5] * s, f[6] * s, f[7] * s)), wide_out);
    if (lane == 0) a.e[row * a.lde + block] = (int8_t)e;
  }
}

// ---- tiles of 128 x 128 -------------------------------------------------------------
// A tile in the registers of 256 threads: thread (tx, ty) = (t & 15, t >> 4) holds columns 8 tx .. + 7 of
// rows 8 ty .. + 7, so that its codes of a column are eight bytes of the transposed matrix.  They go
// through shared memory, 128 bytes a column, units of eight exchanged so that neither side
// meets a bank twice.
template <class T>
__device__ __forceinline__ void load_tile(Vec<T, 8> (&v)[8], const T *x, int64_t ld, int rows, int c, int H, bool wide) {
  const int ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int r = 8 * ty + i;
    if (r < rows) {
      v[i] = some<T, 8>(x + r * ld, c, H, wide);
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++) v[i].v[j] = from_f<T>(0.f);
    }
  }
}
// The codes of a thread's eight columns, column j scaled by s[j], to shared memory.
template <class T, class F>
__device__ __forceinline__ void turn_tile(const Vec<T, 8> (&v)[8], const float (&s)[8], uint2 *turned) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float f[8][8];
#pragma unroll
  for (int i = 0; i < 8; i++) unpack<T, 8>(v[i], f[i]);
#pragma unroll
  for (int j = 0; j < 8; j++)
    turned[(8 * tx + j) * 16 + (ty ^ tx)] =
        make_uint2(codes4<F>(f[0][j] * s[j], f[1][j] * s[j], f[2][j] * s[j], f[3][j] * s[j]),
                   codes4<F>(f[4][j] * s[j], f[5][j] * s[j], f[6][j] * s[j], f[7][j] * s[j]));
}
// And from there to `columns` rows of the transposed matrix, `left` bytes each at most.
__device__ __forceinline__ void put_turned(const uint2 *turned, uint8_t *to, int64_t ld, int columns, int left, bool wide) {
  const int unit = threadIdx.x & 15;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int c = (threadIdx.x >> 4) + 16 * i;
    if (c < columns && 8 * unit < left)
      put8(to + c * ld, 8 * unit, left - 8 * unit, turned[c * 16 + (unit ^ (c >> 3))], wide);
  }
}

// Group of the block-th block of 128 places: its first row of x, how many rows, and the blocks that groups
// fill in all; by a whole warp.  `outside` rows before the first group and behind the last are left over.
struct Place {
  int row, rows, filled, first, last;
};
__device__ __forceinline__ Place place_of(const QuantArgs &a, int block) {
  Place r{0, 0, 0, 0, a.T};
  if (!a.offsets) {
    r.filled = (a.T + kBlock - 1) / kBlock;
    r.row = block * kBlock;
    r.rows = min(kBlock, a.T - r.row);
    return r;
  }
  const int lane = threadIdx.x & 31;
  int most = 0, blocks = 0;
  for (int g0 = 0; g0 <= a.E; g0 += 32) {
    const int g = g0 + lane;
    int o = g <= a.E ? min(max(__ldg(a.offsets + g), 0), a.T) : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int other = __shfl_up_sync(0xFFFFFFFFu, o, d);
      if (lane >= d) o = max(o, other);
    }
    o = max(o, most);
    if (g0 == 0) r.first = __shfl_sync(0xFFFFFFFFu, o, 0);
    int begin = __shfl_up_sync(0xFFFFFFFFu, o, 1);               // of the group that ends at this offset
    if (lane == 0) begin = g0 ? most : o;
    int b = (o - begin + kBlock - 1) / kBlock;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int other = __shfl_up_sync(0xFFFFFFFFu, b, d);
      if (lane >= d) b += other;
    }
    const int before = b - (o - begin + kBlock - 1) / kBlock;
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, block >= blocks + before && block < blocks + b);
    if (hit) {
      const int from = __ffs(hit) - 1, skip = (block - blocks - __shfl_sync(0xFFFFFFFFu, before, from)) * kBlock;
      r.row = __shfl_sync(0xFFFFFFFFu, begin, from) + skip;
      r.rows = min(kBlock, __shfl_sync(0xFFFFFFFFu, o, from) - r.row);
    }
    most = __shfl_sync(0xFFFFFFFFu, o, 31);
    blocks += __shfl_sync(0xFFFFFFFFu, b, 31);
  }
  r.filled = blocks;
  r.last = most;
  return r;
}

// Codes and exponents of the rows that a tile's threads hold.
template <class T, class F>
__device__ __forceinline__ void put_rows(const QuantArgs &a, const Vec<T, 8> (&v)[8], int row, int rows, int block, bool wide) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, c = block * kBlock + 8 * tx;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    float amax = amax_of<T, 8>(v[i]);
#pragma unroll
    for (int o = 8; o; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    if (8 * ty + i >= rows) continue;
    const int64_t r = row + 8 * ty + i;
    const int e = exponent_of<F::kTop>(amax);
    const float s = inverse_of(e);
    float f[8];
    unpack<T, 8>(v[i], f);
    put8(a.q + r * a.ldq, c, a.H - c,
         make_uint2(codes4<F>(f[0] * s, f[1] * s, f[2] * s, f[3] * s), codes4<F>(f[4] * s, f[5] * s, f[6] * s, f[7] * s)), wide);
    if (tx == 0) a.e[r * a.lde + block] = (int8_t)e;
  }
}

// Columns, and with a.q rows: a block of threads takes one block of 128 places and every gridDim.y-th block
// of columns; rows outside all groups (rarely any) are dealt out over the blocks for their row codes.
template <class T, class F>
__global__ void __launch_bounds__(256) columns_kernel(const QuantArgs a, int places, bool wide_in, bool wide_q, bool wide_t) {
  __shared__ uint2 turned[128 * 16];
  __shared__ float peak[8][128];
  grid_go();
  const int tx = threadIdx.x & 15, warp = threadIdx.x >> 5, blocks = (a.H + kBlock - 1) / kBlock;
  const Place at = place_of(a, blockIdx.x);
  Vec<T, 8> v[8];
  for (int block = blockIdx.y; block < blocks; block += gridDim.y) {
    const int c = block * kBlock + 8 * tx;
    load_tile<T>(v, (const T *)a.x + (int64_t)at.row * a.ldx, a.ldx, at.rows, c, a.H, wide_in);
    if (a.q) put_rows<T, F>(a, v, at.row, at.rows, block, wide_q);
    // each column's largest magnitude: a thread's eight rows, the warp's two threads, the eight warps
    float m[8];
#pragma unroll
    for (int j = 0; j < 8; j++) m[j] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      float f[8];
      unpack<T, 8>(v[i], f);
#pragma unroll
      for (int j = 0; j < 8; j++) m[j] = max_nan(m[j], fabsf(f[j]));
    }
#pragma unroll
    for (int j = 0; j < 8; j++) m[j] = max_nan(m[j], __shfl_xor_sync(0xFFFFFFFFu, m[j], 16));
    __syncthreads();                          // the tile before has left shared memory
    if ((threadIdx.x & 16) == 0) {
#pragma unroll
      for (int j = 0; j < 8; j++) peak[warp][8 * tx + j] = m[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; j++)
#pragma unroll
      for (int q = 0; q < 8; q++) m[j] = max_nan(m[j], peak[q][8 * tx + j]);
    float s[8];
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const int e = exponent_of<F::kTop>(m[j]);
      s[j] = inverse_of(e);
      if (threadIdx.x < 16 && c + j < a.H) a.et[(int64_t)(c + j) * a.ldet + blockIdx.x] = (int8_t)e;
    }
    turn_tile<T, F>(v, s, turned);
    __syncthreads();
    put_turned(turned, a.qt + (int64_t)block * kBlock * a.ldqt + (int64_t)blockIdx.x * kBlock, a.ldqt, a.H - block * kBlock, kBlock,
               wide_t);
  }
  const int lead = (at.first + kBlock - 1) / kBlock, tail = (a.T - at.last + kBlock - 1) / kBlock;
  if (a.q)
    for (int o = blockIdx.x; o < lead + tail; o += places) {
      const int row = o < lead ? o * kBlock : at.last + (o - lead) * kBlock, rows = min(kBlock, (o < lead ? at.first : a.T) - row);
      for (int block = blockIdx.y; block < blocks; block += gridDim.y) {
        load_tile<T>(v, (const T *)a.x + (int64_t)row * a.ldx, a.ldx, rows, block * kBlock + 8 * tx, a.H, wide_in);
        put_rows<T, F>(a, v, row, rows, block, wide_q);
      }
    }
}

// Weights: one exponent to a tile.
template <class T, class F>
__global__ void __launch_bounds__(256) weight_kernel(const QuantWeightArgs a, int high, int wide, bool wide_in, bool wide_q,
                                                     bool wide_t) {
  __shared__ uint2 turned[128 * 16];
  __shared__ float peak[8];
  grid_go();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t tile = blockIdx.x, matrix = tile / ((int64_t)high * wide), t = tile - matrix * high * wide;
  const int down = (int)(t / wide), across = (int)(t - (int64_t)down * wide), n0 = down * kBlock, k0 = across * kBlock;
  const int c = k0 + 8 * tx, rows = min(kBlock, a.N - n0);
  Vec<T, 8> v[8];
  load_tile<T>(v, (const T *)a.w + matrix * a.w_stride + (int64_t)n0 * a.ldw, a.ldw, rows, c, a.K, wide_in);
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; i++) m = max_nan(m, amax_of<T, 8>(v[i]));
  m = warp_max(m);
  if ((threadIdx.x & 31) == 0) peak[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; i++) m = max_nan(m, peak[i]);
  const int e = exponent_of<F::kTop>(m);
  const float s = inverse_of(e);
  if (threadIdx.x == 0) {
    a.e[tile] = (int8_t)e;
    if (a.qt) a.et[(matrix * wide + across) * high + down] = (int8_t)e;
  }
#pragma unroll
  for (int i = 0; i < 8; i++) {
    if (8 * ty + i >= rows) break;
    float f[8];
    unpack<T, 8>(v[i], f);
    put8(a.q + matrix * a.q_stride + (int64_t)(n0 + 8 * ty + i) * a.ldq, c, a.K - c,
         make_uint2(codes4<F>(f[0] * s, f[1] * s, f[2] * s, f[3] * s), codes4<F>(f[4] * s, f[5] * s, f[6] * s, f[7] * s)), wide_q);
  }
  if (!a.qt) return;
  const float all[8] = {s, s, s, s, s, s, s, s};
  turn_tile<T, F>(v, all, turned);
  __syncthreads();
  put_turned(turned, a.qt + matrix * a.qt_stride + (int64_t)k0 * a.ldqt + n0, a.ldqt, a.K - k0, rows, wide_t);
}

template <class T, class F>
int quantize_typed(const QuantArgs &a, cudaStream_t st) {
  const int blocks = (a.H + kBlock - 1) / kBlock;
  const bool wide_in = rows16(a.x, a.ldx, sizeof(T)), wide_q = rows_on(a.q, a.ldq, 1, 8);
  if (!a.qt) {
    const int64_t tasks = (int64_t)a.T * blocks, grid = (tasks + 16 * kRows - 1) / (16 * kRows);
    if (grid > INT32_MAX) return MCEMU_ERR_UNSUPPORTED;
    rows_kernel<T, F><<<(unsigned)grid, 256, 0, st>>>(a, tasks, blocks, wide_in, wide_q);
    return launch_status();
  }
  const int places = (int)(mcemu_fp8_columns(a.T, a.E) / kBlock);
  int across = 16 * sm_count() / places + 1;
  across = across < blocks ? across : blocks;
  columns_kernel<T, F><<<dim3(places, across < 65535 ? across : 65535), 256, 0, st>>>(a, places, wide_in, wide_q, rows_on(a.qt, a.ldqt, 1, 8));
  return launch_status();
}
template <class T, class F>
int weight_typed(const QuantWeightArgs &a, cudaStream_t st) {
  const int high = (a.N + kBlock - 1) / kBlock, wide = (a.K + kBlock - 1) / kBlock;
  const int64_t tiles = (int64_t)high * wide * a.E;
  if ((int64_t)high * wide > INT32_MAX || tiles > INT32_MAX) return MCEMU_ERR_UNSUPPORTED;
  const auto on = [&](const void *p, int64_t ld, int64_t stride, int size, int n) {
    return rows_on(p, ld, size, n) && (a.E == 1 || stride * size % n == 0);
  };
  weight_kernel<T, F><<<(unsigned)tiles, 256, 0, st>>>(a, high, wide, on(a.w, a.ldw, a.w_stride, sizeof(T), 16),
                                                       on(a.q, a.ldq, a.q_stride, 1, 8), on(a.qt, a.ldqt, a.qt_stride, 1, 8));
  return launch_status();
}

}  // namespace

int launch_fp8_quantize(int fmt, const QuantArgs &a, void *stream) {
  cudaStream_t st = (cudaStream_t)stream;
  const bool four = a.out_fmt == MCEMU_E4M3;
  if (fmt == MCEMU_FP32) return four ? quantize_typed<float, E4M3>(a, st) : quantize_typed<float, E5M2>(a, st);
  if (fmt == MCEMU_FP16) return four ? quantize_typed<__half, E4M3>(a, st) : quantize_typed<__half, E5M2>(a, st);
  return four ? quantize_typed<__nv_bfloat16, E4M3>(a, st) : quantize_typed<__nv_bfloat16, E5M2>(a, st);
}

int launch_fp8_quantize_weight(int fmt, const QuantWeightArgs &a, void *stream) {
  cudaStream_t st = (cudaStream_t)stream;
  const bool four = a.out_fmt == MCEMU_E4M3;
  if (fmt == MCEMU_FP32) return four ? weight_typed<float, E4M3>(a, st) : weight_typed<float, E5M2>(a, st);
  if (fmt == MCEMU_FP16) return four ? weight_typed<__half, E4M3>(a, st) : weight_typed<__half, E5M2>(a, st);
  return four ? weight_typed<__nv_bfloat16, E4M3>(a, st) : weight_typed<__nv_bfloat16, E5M2>(a, st);
}

}  // namespace mcemu
