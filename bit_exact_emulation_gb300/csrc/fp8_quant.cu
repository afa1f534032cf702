// fp8_quant.cu -- FP8 operands with a power-of-two scale for each block of 128 (include/mcemu_fp8.h).
//
// Bound by HBM: 3 bytes an element from bf16, 4 where the transposed codes are wanted too; both
// come from one reading.  8192 x 8192 bf16: rows 33 us (6.0 TB/s), rows and columns 46.4 us (5.8), of 8
// groups 49.6 us (5.4; instructions issue in 0.63 of the cycles), weights both ways 42.0 us (6.4, 0.94 of the measured rate).
// fp32, 8192 x 4096: rows 26.3 us, rows and columns 40.5 (5.0): a tile is 64 registers of a thread, so that 128 hold two blocks of
// threads an SM and a few words spill, and nothing is asked for ahead.
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

// ---- eight elements of a row --------------------------------------------------------
// Magnitudes are compared as whole numbers, which orders them as numbers, a NaN above all; 16-bit types two at a
// time.  A `Peak` is the largest magnitude so far: two halves of a register, or fp32's bits.
template <class T>
__device__ __forceinline__ uint32_t peak_of(uint32_t a, uint32_t b) {
  if constexpr (sizeof(T) == 2) return __vmaxu2(a, b);
  else return max(a, b);
}
template <class T, int I>
__device__ __forceinline__ uint32_t magnitudes(const Vec<T, 8> &x) {           // of word I
  return ((const uint32_t *)&x)[I] & (sizeof(T) == 2 ? 0x7FFF7FFFu : 0x7FFFFFFFu);
}
template <class T>
__device__ __forceinline__ uint32_t row_peak(const Vec<T, 8> &x) {
  uint32_t m = peak_of<T>(peak_of<T>(magnitudes<T, 0>(x), magnitudes<T, 1>(x)), peak_of<T>(magnitudes<T, 2>(x), magnitudes<T, 3>(x)));
  if constexpr (sizeof(T) == 4)
    m = max(m, max(max(magnitudes<T, 4>(x), magnitudes<T, 5>(x)), max(magnitudes<T, 6>(x), magnitudes<T, 7>(x))));
  return m;
}
// A magnitude in the low half (or all) of a word.
template <class T>
__device__ __forceinline__ float magnitude(uint32_t m) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(m);
  else if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half((unsigned short)m));
  else return __uint_as_float(m << 16);
}
template <class T>
__device__ __forceinline__ float whole_peak(uint32_t m) {
  if constexpr (sizeof(T) == 2) m = max(m & 0xFFFFu, m >> 16);
  return magnitude<T>(m);
}
// Element i.
template <class T, int I>
__device__ __forceinline__ float element(const Vec<T, 8> &x) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    const uint32_t w = ((const uint32_t *)&x)[I / 2];
    return __uint_as_float(I & 1 ? w & 0xFFFF0000u : w << 16);
  } else {
    return to_f(x.v[I]);
  }
}
// Codes of the eight elements, all scaled by s.
template <class T, class F>
__device__ __forceinline__ uint2 row_codes(const Vec<T, 8> &x, float s) {
  const float2 ss = make_float2(s, s);
  float f[8];
  unpack<T, 8>(x, f);
  const float2 a = mul2(make_float2(f[0], f[1]), ss), b = mul2(make_float2(f[2], f[3]), ss);
  const float2 c = mul2(make_float2(f[4], f[5]), ss), d = mul2(make_float2(f[6], f[7]), ss);
  return make_uint2(codes4<F>(a.x, a.y, b.x, b.y), codes4<F>(c.x, c.y, d.x, d.y));
}

// Eight elements of a row from column c on, zeros beyond H, at any alignment: 16-bit ones out of the four or five
// words that hold them (of which two bytes may lie beside the row).  Without a branch, so that the loads of
// many rows are under way at once.
template <class T>
__device__ __forceinline__ Vec<T, 8> load8_any(const T *row, int c, int H) {
  Vec<T, 8> r;
  if constexpr (sizeof(T) == 2) {
    const uintptr_t p = (uintptr_t)(row + c);
    const uint32_t *from = (const uint32_t *)(p & ~(uintptr_t)3);
    const int odd = (int)(p >> 1) & 1, left = H - c;
    uint32_t w[5];
#pragma unroll
    for (int i = 0; i < 5; i++) w[i] = 2 * i - odd < left && left > 0 && (i < 4 || odd) ? __ldg(from + i) : 0u;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const uint32_t v = __funnelshift_r(w[i], w[i + 1], 16 * odd);
      ((uint32_t *)&r)[i] = 2 * i + 1 < left ? v : 2 * i < left ? v & 0xFFFFu : 0u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) r.v[i] = c + i < H ? row[c + i] : from_f<T>(0.f);
  }
  return r;
}
// Eight bytes of a row from column c on, `left` of them in it.
__device__ __forceinline__ void put8_any(uint8_t *row, int c, int left, uint2 v) {
  if (left >= 8 && ((uintptr_t)(row + c) & 7) == 0) {
    *(uint2 *)(row + c) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (i < left) row[c + i] = (uint8_t)((i < 4 ? v.x : v.y) >> (8 * (i & 3)));
  }
}

// A kernel's WIDE form takes rows of whole vectors, on 16-byte boundaries in x, 8 in q and 16 in qt; the
// other one any.
template <class T, bool WIDE>
__device__ __forceinline__ Vec<T, 8> load8(const T *row, int c, int H) {
  if constexpr (!WIDE) return load8_any<T>(row, c, H);
  Vec<T, 8> r = {};
  if (c < H) {
#pragma unroll
    for (int i = 0; i < 8; i += 16 / (int)sizeof(T)) *(uint4 *)&r.v[i] = __ldg((const uint4 *)(row + c + i));
  }
  return r;
}
template <bool WIDE>
__device__ __forceinline__ void put8(uint8_t *row, int c, int left, uint2 v) {
  if constexpr (WIDE) {
    if (left > 0) *(uint2 *)(row + c) = v;
  } else {
    put8_any(row, c, left, v);
  }
}

// ---- rows alone -------------------------------------------------------------------
// Sixteen lanes to a block of a row, eight elements each, kRows rows a thread; a block of threads takes `wide`
// (1 to 16) blocks of 16 / wide * kRows rows.  8192 x 8192 bf16 with two rows a thread 34.7 us, four 32.5, eight 43.2.
constexpr int kRows = 4;
template <class T, class F, bool WIDE>
__global__ void __launch_bounds__(256) rows_kernel(const QuantArgs a, int blocks, int wide) {
  grid_go();
  const int lane = threadIdx.x & 15, at = threadIdx.x >> 4, high = 16 / wide;
  const int block = (int)((blockIdx.y + blockIdx.z * gridDim.y) * wide) + at % wide, c = block * kBlock + 8 * lane;
  const int64_t row0 = (int64_t)blockIdx.x * (high * kRows) + at / wide;
  const T *x = (const T *)a.x + row0 * a.ldx;
  Vec<T, 8> v[kRows];
  uint32_t m[kRows];
#pragma unroll
  for (int i = 0; i < kRows; i++) {
    if constexpr (!WIDE) {
      v[i] = load8_any<T>(x + i * high * a.ldx, c, row0 + i * high < a.T ? a.H : 0);
    } else if (row0 + i * high < a.T && block < blocks) {
      v[i] = load8<T, WIDE>(x + i * high * a.ldx, c, a.H);
    } else {
      v[i] = Vec<T, 8>{};
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; i++) m[i] = row_peak<T>(v[i]);
  if constexpr (sizeof(T) == 2) {             // two rows to a word
#pragma unroll
    for (int i = 0; i < kRows; i += 2) {
      uint32_t w = __vmaxu2(__byte_perm(m[i], m[i + 1], 0x5410), __byte_perm(m[i], m[i + 1], 0x7632));
#pragma unroll
      for (int o = 8; o; o >>= 1) w = __vmaxu2(w, __shfl_xor_sync(0xFFFFFFFFu, w, o));
      m[i] = w & 0xFFFFu, m[i + 1] = w >> 16;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kRows; i++)
#pragma unroll
      for (int o = 8; o; o >>= 1) m[i] = max(m[i], __shfl_xor_sync(0xFFFFFFFFu, m[i], o));
  }
  uint8_t *q = a.q + row0 * a.ldq;
  int8_t *e = a.e + row0 * a.lde + block;
#pragma unroll
  for (int i = 0; i < kRows; i++) {
    if (row0 + i * high >= a.T || block >= blocks) break;
    const int ex = exponent_of<F::kTop>(magnitude<T>(m[i]));
    put8<WIDE>(q + i * high * a.ldq, c, a.H - c, row_codes<T, F>(v[i], inverse_of(ex)));
    if (lane == 0) e[i * high * a.lde] = (int8_t)ex;
  }
}

// ---- tiles of 128 x 128 -------------------------------------------------------------
// A tile in the registers of 256 threads: thread (tx, ty) = (t & 15, t >> 4) holds columns 8 tx .. + 7 of
// rows 8 ty .. + 7, so that its codes of a column are eight bytes of the transposed matrix.  They go
// through shared memory, 128 bytes a column, eight-byte units exchanged by the column so that neither side meets a bank twice.
template <class T, bool WIDE>
__device__ __forceinline__ void load_tile(Vec<T, 8> (&v)[8], const T *x, int64_t ld, int rows, int c, int H) {
  const int r0 = 8 * (threadIdx.x >> 4);
  x += r0 * ld;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    if constexpr (!WIDE) {
      v[i] = load8_any<T>(x + i * ld, c, r0 + i < rows ? H : 0);
    } else if (r0 + i < rows) {
      v[i] = load8<T, WIDE>(x + i * ld, c, H);
    } else {
      v[i] = Vec<T, 8>{};
    }
  }
}
// The same of 16-bit elements by copies into places of the thread's own, which are under way while it works on
// the tile before (loaded when they are needed, 8192 x 8192 in 8 groups took 53.1 us in place of 49.8).
template <class T>
__device__ __forceinline__ void ask_tile(uint4 *places, const T *x, int64_t ld, int rows, int c, int H) {
  const int r0 = 8 * (threadIdx.x >> 4);
  x += r0 * ld + c;
#pragma unroll
  for (int i = 0; i < 8; i++)
    if (r0 + i < rows && c < H) copy_async<16>(places + 256 * i + threadIdx.x, x + i * ld);
  copy_commit();
}
template <class T>
__device__ __forceinline__ void take_tile(Vec<T, 8> (&v)[8], const uint4 *places, int rows, int c, int H) {
  const int r0 = 8 * (threadIdx.x >> 4);
  copy_wait<0>();
#pragma unroll
  for (int i = 0; i < 8; i++) {
    if (r0 + i < rows && c < H) {
      *(uint4 *)&v[i] = places[256 * i + threadIdx.x];
    } else {
      v[i] = Vec<T, 8>{};
    }
  }
}
// Column j's codes of the thread's eight rows, scaled by s.
template <class T, class F, int J>
__device__ __forceinline__ void turn_column(const Vec<T, 8> (&v)[8], float s, uint2 *turned) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const float2 ss = make_float2(s, s);
  const float2 a = mul2(make_float2(element<T, J>(v[0]), element<T, J>(v[1])), ss), b = mul2(make_float2(element<T, J>(v[2]), element<T, J>(v[3])), ss);
  const float2 c = mul2(make_float2(element<T, J>(v[4]), element<T, J>(v[5])), ss), d = mul2(make_float2(element<T, J>(v[6]), element<T, J>(v[7])), ss);
  turned[(8 * tx + J) * 16 + (ty ^ ((tx & 7) << 1) ^ (tx >> 3))] = make_uint2(codes4<F>(a.x, a.y, b.x, b.y), codes4<F>(c.x, c.y, d.x, d.y));
}
template <class T, class F>
__device__ __forceinline__ void turn_tile(const Vec<T, 8> (&v)[8], const float (&s)[8], uint2 *turned) {
  turn_column<T, F, 0>(v, s[0], turned), turn_column<T, F, 1>(v, s[1], turned);
  turn_column<T, F, 2>(v, s[2], turned), turn_column<T, F, 3>(v, s[3], turned);
  turn_column<T, F, 4>(v, s[4], turned), turn_column<T, F, 5>(v, s[5], turned);
  turn_column<T, F, 6>(v, s[6], turned), turn_column<T, F, 7>(v, s[7], turned);
}
// And from there to `columns` rows of the transposed matrix, `left` bytes each at most: sixteen a thread, four times.
template <bool WIDE>
__device__ __forceinline__ void put_turned(const uint2 *turned, uint8_t *to, int64_t ld, int columns, int left) {
  const int unit = threadIdx.x & 7, c0 = threadIdx.x >> 3;
  to += c0 * ld + 16 * unit;
  left -= 16 * unit;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int c = c0 + 32 * i, tx = c >> 3;
    if (c >= columns || left <= 0) break;
    const uint4 w = *(const uint4 *)(turned + c * 16 + 2 * (unit ^ (tx & 7)));
    const uint4 v = tx & 8 ? make_uint4(w.z, w.w, w.x, w.y) : w;
    uint8_t *p = to + 32 * i * ld;
    if (left >= 16 && (WIDE || ((uintptr_t)p & 15) == 0)) {
      *(uint4 *)p = v;
    } else {
      put8_any(p, 0, left, make_uint2(v.x, v.y));
      put8_any(p, 8, left - 8, make_uint2(v.z, v.w));
    }
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

// Codes and exponents of the rows that a tile's threads hold: sixteen lanes have eight rows, and lane i makes the
// i-th one's exponent for all.
template <class T, class F, bool WIDE>
__device__ __forceinline__ void put_rows(const QuantArgs &a, const Vec<T, 8> (&v)[8], int row, int rows, int block) {
  const int tx = threadIdx.x & 15, r0 = 8 * (threadIdx.x >> 4), c = block * kBlock + 8 * tx;
  uint32_t m[8], mine;
#pragma unroll
  for (int i = 0; i < 8; i++) m[i] = row_peak<T>(v[i]);
  if constexpr (sizeof(T) == 2) {             // two rows to a word
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      m[i] = __vmaxu2(__byte_perm(m[i], m[i + 1], 0x5410), __byte_perm(m[i], m[i + 1], 0x7632));
#pragma unroll
      for (int o = 8; o; o >>= 1) m[i] = __vmaxu2(m[i], __shfl_xor_sync(0xFFFFFFFFu, m[i], o));
    }
    mine = tx & 4 ? (tx & 2 ? m[6] : m[4]) : (tx & 2 ? m[2] : m[0]);
    mine = tx & 1 ? mine >> 16 : mine & 0xFFFFu;
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++)
#pragma unroll
      for (int o = 8; o; o >>= 1) m[i] = max(m[i], __shfl_xor_sync(0xFFFFFFFFu, m[i], o));
    mine = tx & 4 ? (tx & 2 ? (tx & 1 ? m[7] : m[6]) : (tx & 1 ? m[5] : m[4])) : (tx & 2 ? (tx & 1 ? m[3] : m[2]) : (tx & 1 ? m[1] : m[0]));
  }
  const int ex = exponent_of<F::kTop>(magnitude<T>(mine));
  const float inverse = inverse_of(ex);
  if (tx < 8 && r0 + tx < rows) a.e[(int64_t)(row + r0 + tx) * a.lde + block] = (int8_t)ex;
  uint8_t *q = a.q + (int64_t)(row + r0) * a.ldq;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float s = __shfl_sync(0xFFFFFFFFu, inverse, (threadIdx.x & 16) + i);
    if (r0 + i < rows) put8<WIDE>(q + i * a.ldq, c, a.H - c, row_codes<T, F>(v[i], s));
  }
}

// The largest magnitudes of word W's columns over a thread's rows, and with the other thread of its warp.
template <class T, int W>
__device__ __forceinline__ uint32_t column_peak(const Vec<T, 8> (&v)[8]) {
  uint32_t m = magnitudes<T, W>(v[0]);
#pragma unroll
  for (int i = 1; i < 8; i++) m = peak_of<T>(m, magnitudes<T, W>(v[i]));
  return peak_of<T>(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
}

// Columns, and with a.q rows.  Of 16-bit elements a block of threads takes one block of 128 places and every gridDim.y-th
// block of columns; of fp32 (ALONG) as many tiles as every other, one after the other along the rows: 8192 x 4096 in
// fp32 40.0 us, by the former way 52.8; bf16 8192 x 8192, without groups as before, 50.7, by the former 46.5.  Rows outside all groups (rarely any)
// are dealt out over the blocks for their row codes.
template <class T, class F, bool WIDE>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 3 : 2) columns_kernel(const QuantArgs a, int64_t tiles) {
  constexpr int kWords = 2 * sizeof(T);       // of a thread's eight columns
  __shared__ __align__(16) uint2 turned[128 * 16];
  __shared__ __align__(16) uint32_t peak[8][16 * kWords];
  __shared__ __align__(16) float scale[kBlock];
  extern __shared__ __align__(16) uint4 places_ahead[];        // AHEAD: 2048
  constexpr bool AHEAD = WIDE && sizeof(T) == 2, ALONG = sizeof(T) == 4;
  grid_go();
  const int tx = threadIdx.x & 15, warp = threadIdx.x >> 5, blocks = (a.H + kBlock - 1) / kBlock;
  int place = blockIdx.x, block = blockIdx.y, left = 0;          // left: ALONG, tiles that are
  if constexpr (ALONG) {
    const int64_t first = tiles * blockIdx.x / gridDim.x;
    place = (int)(first / blocks);
    block = (int)(first - (int64_t)place * blocks);
    left = (int)(tiles * (blockIdx.x + 1) / gridDim.x - first);
  }
  Place at = place_of(a, place);
  Vec<T, 8> v[8];
  const T *x = (const T *)a.x + (int64_t)at.row * a.ldx;
  if constexpr (AHEAD) ask_tile<T>(places_ahead, x, a.ldx, at.rows, blockIdx.y * kBlock + 8 * tx, a.H);
  for (; ALONG ? left-- > 0 : block < blocks; block += ALONG ? 1 : gridDim.y) {
    if (ALONG && block == blocks) {
      block = 0;
      at = place_of(a, ++place);
      x = (const T *)a.x + (int64_t)at.row * a.ldx;
    }
    const int c = block * kBlock + 8 * tx;
    if constexpr (AHEAD) {
      take_tile<T>(v, places_ahead, at.rows, c, a.H);
      if (block + (int)gridDim.y < blocks)    // a column beyond that may be more than 32 bits count
        ask_tile<T>(places_ahead, x, a.ldx, at.rows, c + (int)gridDim.y * kBlock, a.H);
    } else {
      load_tile<T, WIDE>(v, x, a.ldx, at.rows, c, a.H);
    }
    uint32_t m[kWords];
    m[0] = column_peak<T, 0>(v), m[1] = column_peak<T, 1>(v), m[2] = column_peak<T, 2>(v), m[3] = column_peak<T, 3>(v);
    if constexpr (sizeof(T) == 4)
      m[4] = column_peak<T, 4>(v), m[5] = column_peak<T, 5>(v), m[6] = column_peak<T, 6>(v), m[7] = column_peak<T, 7>(v);
    __syncthreads();                          // the tile before has left shared memory
    if ((threadIdx.x & 16) == 0) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) *(uint4 *)&peak[warp][tx * kWords + i] = make_uint4(m[i], m[i + 1], m[i + 2], m[i + 3]);
    }
    if (a.q) put_rows<T, F, WIDE>(a, v, at.row, at.rows, block);
    __syncthreads();
    if (threadIdx.x < 16 * kWords) {          // a word's column, or two
      uint32_t all = peak[0][threadIdx.x];
#pragma unroll
      for (int w = 1; w < 8; w++) all = peak_of<T>(all, peak[w][threadIdx.x]);
      constexpr int kEach = 4 / sizeof(T);
#pragma unroll
      for (int j = 0; j < kEach; j++) {
        const int at_column = kEach * threadIdx.x + j, e = exponent_of<F::kTop>(magnitude<T>(kEach == 1 ? all : j ? all >> 16 : all & 0xFFFFu));
        scale[at_column] = inverse_of(e);
        if (block * kBlock + at_column < a.H) a.et[(int64_t)(block * kBlock + at_column) * a.ldet + place] = (int8_t)e;
      }
    }
    __syncthreads();
    float s[8];
    *(float4 *)&s[0] = *(const float4 *)&scale[8 * tx];
    *(float4 *)&s[4] = *(const float4 *)&scale[8 * tx + 4];
    turn_tile<T, F>(v, s, turned);
    __syncthreads();
    put_turned<WIDE>(turned, a.qt + (int64_t)block * kBlock * a.ldqt + (int64_t)place * kBlock, a.ldqt, a.H - block * kBlock, kBlock);
  }
  const int lead = (at.first + kBlock - 1) / kBlock, tail = (a.T - at.last + kBlock - 1) / kBlock;
  if (a.q)
    for (int64_t o = blockIdx.x + (int64_t)blockIdx.y * gridDim.x; o < (int64_t)(lead + tail) * blocks; o += (int64_t)gridDim.x * gridDim.y) {
      const int down = (int)(o / blocks), across = (int)(o - (int64_t)down * blocks);
      const int row = down < lead ? down * kBlock : at.last + (down - lead) * kBlock, rows = min(kBlock, (down < lead ? at.first : a.T) - row);
      load_tile<T, WIDE>(v, (const T *)a.x + (int64_t)row * a.ldx, a.ldx, rows, across * kBlock + 8 * tx, a.H);
      put_rows<T, F, WIDE>(a, v, row, rows, across);
    }
}

// Weights: one exponent to a tile.
template <class T, class F, bool WIDE>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 4 : 2) weight_kernel(const QuantWeightArgs a, int high, int wide) {
  __shared__ __align__(16) uint2 turned[128 * 16];
  __shared__ uint32_t peak[8];
  grid_go();
  const int tx = threadIdx.x & 15, r0 = 8 * (threadIdx.x >> 4), tile = blockIdx.x, per = high * wide;
  const int matrix = tile / per, t = tile - matrix * per, down = t / wide, across = t - down * wide;
  const int n0 = down * kBlock, k0 = across * kBlock, c = k0 + 8 * tx, rows = min(kBlock, a.N - n0);
  Vec<T, 8> v[8];
  load_tile<T, WIDE>(v, (const T *)a.w + matrix * a.w_stride + (int64_t)n0 * a.ldw, a.ldw, rows, c, a.K);
  uint32_t m = row_peak<T>(v[0]);
#pragma unroll
  for (int i = 1; i < 8; i++) m = peak_of<T>(m, row_peak<T>(v[i]));
#pragma unroll
  for (int o = 16; o; o >>= 1) m = peak_of<T>(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if ((threadIdx.x & 31) == 0) peak[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; i++) m = peak_of<T>(m, peak[i]);
  const int e = exponent_of<F::kTop>(whole_peak<T>(m));
  const float s = inverse_of(e);
  if (threadIdx.x == 0) {
    a.e[tile] = (int8_t)e;
    if (a.qt) a.et[(int64_t)matrix * per + across * high + down] = (int8_t)e;
  }
  uint8_t *q = a.q + matrix * a.q_stride + (int64_t)(n0 + r0) * a.ldq;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    if (r0 + i >= rows) break;
    put8<WIDE>(q + i * a.ldq, c, a.K - c, row_codes<T, F>(v[i], s));
  }
  if (!a.qt) return;
  const float all[8] = {s, s, s, s, s, s, s, s};
  turn_tile<T, F>(v, all, turned);
  __syncthreads();
  put_turned<WIDE>(turned, a.qt + matrix * a.qt_stride + (int64_t)k0 * a.ldqt + n0, a.ldqt, a.K - k0, rows);
}

template <class T, class F>
int quantize_typed(const QuantArgs &a, cudaStream_t st) {
  const int blocks = (a.H + kBlock - 1) / kBlock;
  const bool whole = a.H % 8 == 0 && rows16(a.x, a.ldx, sizeof(T)) && rows_on(a.q, a.ldq, 1, 8);
  if (!a.qt) {
    int wide = 1;
    while (wide < 16 && wide < blocks) wide *= 2;
    const int high = 16 / wide * kRows, across = (blocks + wide - 1) / wide, y = across < 65535 ? across : 65535;
    const dim3 grid((a.T + high - 1) / high, y, (across + y - 1) / y);
    if (whole) rows_kernel<T, F, true><<<grid, 256, 0, st>>>(a, blocks, wide);
    else rows_kernel<T, F, false><<<grid, 256, 0, st>>>(a, blocks, wide);
    return launch_status();
  }
  const int places = (int)(mcemu_fp8_columns(a.T, a.E) / kBlock);
  const int64_t tiles = (int64_t)places * blocks;
  dim3 grid;
  if (sizeof(T) == 4) {                       // as many blocks of threads as run at a time
    const int64_t most = 2 * sm_count();
    grid = dim3((unsigned)(tiles < most ? tiles : most));
  } else {
    // two rounds of the blocks of threads that run at a time, with so many tiles each, one's copies under way while
    // the one before is worked on.  8192 x 8192 in 8 groups: tiles each and microseconds 2 49.7, 4 49.8, 5 49.3, 8 55.2, 10 60.1.
    int64_t turns = tiles / (6 * sm_count());
    turns = turns < 1 ? 1 : turns < blocks ? turns : blocks;
    const int64_t across = (blocks + turns - 1) / turns;
    grid = dim3(places, across < 65535 ? across : 65535);
  }
  if (whole && rows_on(a.qt, a.ldqt, 1, 16)) {
    constexpr int kAhead = sizeof(T) == 2 ? 32768 : 0;
    if (!allow_smem<columns_kernel<T, F, true>>(kAhead)) return MCEMU_ERR_CUDA;
    columns_kernel<T, F, true><<<grid, 256, kAhead, st>>>(a, tiles);
  } else {
    columns_kernel<T, F, false><<<grid, 256, 0, st>>>(a, tiles);
  }
  return launch_status();
}
template <class T, class F>
int weight_typed(const QuantWeightArgs &a, cudaStream_t st) {
  const int high = (a.N + kBlock - 1) / kBlock, wide = (a.K + kBlock - 1) / kBlock;
  const int64_t tiles = (int64_t)high * wide * a.E;
  if (tiles > INT32_MAX) return MCEMU_ERR_UNSUPPORTED;
  const auto on = [&](const void *p, int64_t ld, int64_t stride, int size, int n) {
    return rows_on(p, ld, size, n) && (a.E == 1 || stride * size % n == 0);
  };
  const dim3 grid((unsigned)tiles);
  if (a.K % 8 == 0 && on(a.w, a.ldw, a.w_stride, sizeof(T), 16) && on(a.q, a.ldq, a.q_stride, 1, 8) && on(a.qt, a.ldqt, a.qt_stride, 1, 16))
    weight_kernel<T, F, true><<<grid, 256, 0, st>>>(a, high, wide);
  else
    weight_kernel<T, F, false><<<grid, 256, 0, st>>>(a, high, wide);
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
