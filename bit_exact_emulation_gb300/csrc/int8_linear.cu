// int8_linear.cu -- product of 8-bit integers with a scale for each token and channel
// (include/mcemu_ops.h has the formula).
//
// sm_103a has no fast 8-bit integer matrix instruction, so the sums run on the 16-bit floating
// one, exactly: an 8-bit integer is a binary16 number, a product is below 2^14 + 1, and a sum
// of 1024 products is an integer of at most 2^24, which fp32 accumulators hold without
// rounding (every partial sum too, in any order).  Every 1024 products the accumulators are
// therefore taken out of tensor memory and added to int32 sums in registers.
#include "panel.cuh"

namespace mcemu {
namespace {

// The output's bits from the exact sum: each step rounded to fp32, then to the type.
template <int OUT>
struct OutType { using T = float; };
template <> struct OutType<MCEMU_FP16> { using T = __half; };
template <> struct OutType<MCEMU_BF16> { using T = __nv_bfloat16; };
template <> struct OutType<MCEMU_INT32> { using T = int32_t; };

template <int OUT>
__device__ __forceinline__ typename OutType<OUT>::T scaled(int acc, float sx, float sw, bool biased, float bias) {
  if constexpr (OUT == MCEMU_INT32) {
    return acc;
  } else {
    float v = __fmul_rn(__fmul_rn((float)acc, sx), sw);
    if (biased) v = __fadd_rn(v, bias);
    return from_f<typename OutType<OUT>::T>(v);
  }
}

// Scale and bias of a channel (0 for those an int32 output does without).
template <int OUT>
__device__ __forceinline__ float2 channel(const LinearArgs &a, int n) {
  if constexpr (OUT == MCEMU_INT32) return make_float2(0.f, 0.f);
  return make_float2(__ldg(a.sw + n), a.bias ? __ldg(a.bias + n) : 0.f);
}

// Sixteen tokens of one channel.
template <int OUT>
__device__ __forceinline__ void put16(const LinearArgs &a, int m0, int n, const int *acc, float2 c) {
  using T = typename OutType<OUT>::T;
  T *y = (T *)a.y + (int64_t)m0 * a.ldy + n;
  const bool biased = a.bias != nullptr;
#pragma unroll
  for (int x = 0; x < 16; x++) {
    if (m0 + x < a.M) {
      const float sx = OUT == MCEMU_INT32 ? 0.f : __ldg(a.sx + m0 + x);
      *y = scaled<OUT>(acc[x], sx, c.x, biased, c.y);
    }
    y += a.ldy;
  }
}

// Four signed bytes to four binary16 numbers, exactly: b + 128 in the low mantissa bits of
// 1024, less 1152.
__device__ __forceinline__ void half4(uint32_t b, uint32_t &lo, uint32_t &hi) {
  b ^= 0x80808080u;
  const __half2 off = __half2half2(__ushort_as_half(0x6480));   // 1152
  uint32_t l = __byte_perm(b, 0x64646464u, 0x4140), h = __byte_perm(b, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*(__half2 *)&l, off), y = __hsub2(*(__half2 *)&h, off);
  lo = *(const uint32_t *)&x;
  hi = *(const uint32_t *)&y;
}

// ---------------------------------------------------------------------------
// Large products: both operands are widened to binary16 panels once (3 bytes of traffic an
// element, against a conversion for every tile that reads it), and pairs of CTAs multiply
// the panels with nothing but copies and matrix instructions in the loop.
// ---------------------------------------------------------------------------
struct Widen {
  const int8_t *src;
  int64_t ld;
  int rows, blocks;          // rows, and 128-row blocks of the panel
  uint8_t *to;
};

// One tile (128 rows by 64 k) to a block.
__global__ void __launch_bounds__(256) widen_kernel(const Widen x, const Widen w, int K, int ktiles, bool wide) {
  int64_t tile = blockIdx.x;
  const int64_t mine = (int64_t)x.blocks * ktiles;
  const Widen &o = tile < mine ? x : w;
  if (tile >= mine) tile -= mine;
  const int block = (int)(tile / ktiles), kt = (int)(tile - (int64_t)block * ktiles);
  uint8_t *to = o.to + tile * panel::kTileBytes;
#pragma unroll
  for (int j = 0; j < 2; j++) {
    const int piece = threadIdx.x & 3, r = (threadIdx.x >> 2) + 64 * j, row = block * 128 + r;
    const int k = kt * 64 + 16 * piece;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row < o.rows && k < K) v = row16(o.src + (int64_t)row * o.ld, k, K, wide);
    uint4 lo, hi;
    half4(v.x, lo.x, lo.y);
    half4(v.y, lo.z, lo.w);
    half4(v.z, hi.x, hi.y);
    half4(v.w, hi.z, hi.w);
    const int at = r * 128 + (((2 * piece) ^ (r & 7)) << 4);
    *(uint4 *)(to + at) = lo;
    *(uint4 *)(to + (at ^ 16)) = hi;
  }
}

template <int OUT>
struct LinearEp {
  using Sum = int;
  LinearArgs a;
  static __device__ __forceinline__ void add(int &s, float v) { s += __float2int_rn(v); }
  __device__ __forceinline__ void store(int n, int m0, const int *sum, int) const {
    if (n >= a.N) return;
    put16<OUT>(a, m0, n, sum, channel<OUT>(a, n));
  }
};

int blocks128(int rows) { return (rows + 255) / 256 * 2; }
int ktiles_of(int K) { return (K + 63) / 64; }

template <int OUT>
int go_panels(const LinearArgs &a, bool wide, void *ws, cudaStream_t st) {
  const int kt = ktiles_of(a.K);
  Widen x{a.x, a.ldx, a.M, blocks128(a.M), (uint8_t *)ws};
  Widen w{a.w, a.ldw, a.N, blocks128(a.N), x.to + (int64_t)x.blocks * kt * panel::kTileBytes};
  const int64_t tiles = (int64_t)(x.blocks + w.blocks) * kt;
  if (!panel::panel_fits(x.blocks, kt) || !panel::panel_fits(w.blocks, kt)) return MCEMU_ERR_UNSUPPORTED;
  widen_kernel<<<(unsigned)tiles, 256, 0, st>>>(x, w, a.K, kt, wide);
  CUtensorMap mw, mx;
  int rc = panel::panel_map(&mw, w.to, w.blocks, kt);
  if (rc == MCEMU_OK) rc = panel::panel_map(&mx, x.to, x.blocks, kt);
  if (rc != MCEMU_OK) return rc;
  panel::Args g{kt, w.blocks / 2, x.blocks / 2, 1, kt, 1024 / panel::kTileK};
  return panel::launch<LinearEp<OUT>, 0, 0, 0>(g, mw, mx, LinearEp<OUT>{a}, st);
}

// ---------------------------------------------------------------------------
// Few tokens: the weights' bytes are what counts, and every warp widens what it reads in
// registers.  A block takes 16 * CH channels by 8 * NT tokens; its eight warps share K, 64 at a
// time in turn.  The warp-wide matrix instruction (m16n8k16, 1000 MAC a cycle and SM measured,
// against 250 for its 8-bit form and for dp4a alike) takes four k of a row from a lane, and
// which four is free as long as both operands agree: a lane reads 16 consecutive bytes of
// its rows and feeds them to four instructions.
// ---------------------------------------------------------------------------
constexpr int kWarps = 8;

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

template <int OUT, int NT, int CH>
__global__ void __launch_bounds__(32 * kWarps) few_kernel(const LinearArgs a, bool wide) {
  constexpr int kAhead = NT * CH >= 8 ? 2 : 4;               // pieces of 64 k in flight
  __shared__ int total[16 * CH][8 * NT + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * 16 * CH, m0 = blockIdx.y * 8 * NT;
  for (int i = threadIdx.x; i < 16 * CH * (8 * NT + 1); i += blockDim.x) (&total[0][0])[i] = 0;

  const int8_t *wrow[2 * CH], *xrow[NT];
  bool whave[2 * CH], xhave[NT];
#pragma unroll
  for (int r = 0; r < 2 * CH; r++) {
    whave[r] = n0 + 8 * r + g < a.N;
    wrow[r] = a.w + (whave[r] ? (int64_t)(n0 + 8 * r + g) * a.ldw : 0);
  }
#pragma unroll
  for (int j = 0; j < NT; j++) {
    xhave[j] = m0 + 8 * j + g < a.M;
    xrow[j] = a.x + (xhave[j] ? (int64_t)(m0 + 8 * j + g) * a.ldx : 0);
  }
  float acc[CH][NT][4];
  int sum[CH][NT][4];
#pragma unroll
  for (int i = 0; i < CH * NT * 4; i++) (&acc[0][0][0])[i] = 0.f, (&sum[0][0][0])[i] = 0;

  const int pieces = (a.K + 63) / 64;
  int since = 0;                                             // pieces since the sums were taken out
  for (int p = warp; p < pieces; p += kWarps * kAhead) {
    uint4 w[kAhead][2 * CH], x[kAhead][NT];
#pragma unroll
    for (int u = 0; u < kAhead; u++) {
      const int k = (p + u * kWarps) * 64 + 16 * t;
#pragma unroll
      for (int r = 0; r < 2 * CH; r++) {
        w[u][r] = make_uint4(0, 0, 0, 0);
        if (whave[r] && k < a.K) w[u][r] = row16(wrow[r], k, a.K, wide);
      }
#pragma unroll
      for (int j = 0; j < NT; j++) {
        x[u][j] = make_uint4(0, 0, 0, 0);
        if (xhave[j] && k < a.K) x[u][j] = row16(xrow[j], k, a.K, wide);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; u++) {
      const uint32_t *wu = &w[u][0].x, *xu = &x[u][0].x;
#pragma unroll
      for (int q = 0; q < 4; q++) {
        uint32_t af[CH][4];
#pragma unroll
        for (int c = 0; c < CH; c++) {
          half4(wu[(2 * c) * 4 + q], af[c][0], af[c][2]);
          half4(wu[(2 * c + 1) * 4 + q], af[c][1], af[c][3]);
        }
#pragma unroll
        for (int j = 0; j < NT; j++) {
          uint32_t bf[2];
          half4(xu[j * 4 + q], bf[0], bf[1]);
#pragma unroll
          for (int c = 0; c < CH; c++) mma16816(acc[c][j], af[c], bf);
        }
      }
    }
    since += kAhead;
    if (since + kAhead > 16 || p + kWarps * kAhead >= pieces) {   // 1024 products an accumulator at most
#pragma unroll
      for (int i = 0; i < CH * NT * 4; i++) {
        (&sum[0][0][0])[i] += __float2int_rn((&acc[0][0][0])[i]);
        (&acc[0][0][0])[i] = 0.f;
      }
      since = 0;
    }
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < CH; c++)
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
      for (int i = 0; i < 4; i++) atomicAdd(&total[16 * c + 8 * (i >> 1) + g][8 * j + 2 * t + (i & 1)], sum[c][j][i]);
  __syncthreads();
  using T = typename OutType<OUT>::T;
  for (int i = threadIdx.x; i < 16 * CH * 8 * NT; i += blockDim.x) {
    const int n = n0 + i % (16 * CH), m = m0 + i / (16 * CH);
    if (n < a.N && m < a.M) {
      const float2 c = channel<OUT>(a, n);
      ((T *)a.y)[(int64_t)m * a.ldy + n] = scaled<OUT>(total[i % (16 * CH)][i / (16 * CH)],
                                                       OUT == MCEMU_INT32 ? 0.f : a.sx[m], c.x, a.bias != nullptr, c.y);
    }
  }
}

template <int OUT, int NT, int CH>
int go_few(const LinearArgs &a, bool wide, cudaStream_t st) {
  const dim3 grid((a.N + 16 * CH - 1) / (16 * CH), (a.M + 8 * NT - 1) / (8 * NT));
  few_kernel<OUT, NT, CH><<<grid, 32 * kWarps, 0, st>>>(a, wide);
  return launch_status();
}

// Products that go through panels.
#ifndef MIN_PANEL
#define MIN_PANEL 64
#endif
bool by_panels(int M, int K) { return M > MIN_PANEL && K > 0; }

template <int OUT>
int go(const LinearArgs &a, bool rows, void *ws, cudaStream_t st) {
  if (by_panels(a.M, a.K)) return go_panels<OUT>(a, rows, ws, st);
  if (a.M <= 8) return go_few<OUT, 1, 1>(a, rows, st);
  if (a.M <= 16) return go_few<OUT, 2, 1>(a, rows, st);
  if (a.M <= 32) return go_few<OUT, 4, 2>(a, rows, st);
  return go_few<OUT, 8, 2>(a, rows, st);
}

}  // namespace

int int8_linear_timeouts(cudaStream_t st, unsigned int *got) { return tc::take_timeouts(st, got); }

size_t int8_linear_workspace(int M, int N, int K) {
  if (!by_panels(M, K)) return 0;
  return (size_t)(blocks128(M) + blocks128(N)) * ktiles_of(K) * panel::kTileBytes;
}

int launch_int8_linear(const LinearArgs &a, bool rows, void *ws, void *stream) {
  cudaStream_t st = (cudaStream_t)stream;
  switch (a.out_fmt) {
    case MCEMU_INT32: return go<MCEMU_INT32>(a, rows, ws, st);
    case MCEMU_FP32: return go<MCEMU_FP32>(a, rows, ws, st);
    case MCEMU_FP16: return go<MCEMU_FP16>(a, rows, ws, st);
    default: return go<MCEMU_BF16>(a, rows, ws, st);
  }
}

}  // namespace mcemu
