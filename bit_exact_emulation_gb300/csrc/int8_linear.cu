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

__device__ __forceinline__ void put_y(const LinearArgs &a, int m, int n, int acc, float sw, float bias) {
  const int64_t at = (int64_t)m * a.ldy + n;
  if (a.out_fmt == MCEMU_INT32) {
    ((int32_t *)a.y)[at] = acc;
    return;
  }
  float v = __fmul_rn(__fmul_rn((float)acc, a.sx[m]), sw);
  if (a.bias) v = __fadd_rn(v, bias);
  if (a.out_fmt == MCEMU_FP32) ((float *)a.y)[at] = v;
  else if (a.out_fmt == MCEMU_FP16) ((__half *)a.y)[at] = __float2half_rn(v);
  else ((__nv_bfloat16 *)a.y)[at] = __float2bfloat16_rn(v);
}

// Sixteen tokens of one channel.
__device__ __forceinline__ void put_y16(const LinearArgs &a, int m0, int n, const int *acc, float sw, float bias) {
#pragma unroll
  for (int x = 0; x < 16; x++)
    if (m0 + x < a.M) put_y(a, m0 + x, n, acc[x], sw, bias);
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
// Matrix kernel.  A tile is 128 channels (operand A) by BN tokens (operand B).  Eight worker warps read
// both operands 64 k at a time, widen them to binary16 and store them in the swizzle; one
// thread issues the matrix instructions; the workers take the accumulators out, one half of
// the columns to each four warps, and write the tile.  Two sets of accumulators let the
// matrix unit run on meanwhile.
// ---------------------------------------------------------------------------
constexpr int kStage = 64;                    // k of a stage: one 128-byte swizzle row
constexpr int kChunk = 1024 / kStage;         // stages between two transfers to int32
constexpr int kWorkers = 256;

template <int BN>
struct Shape {
  static constexpr int kRowsB = BN;                             // token rows
  static constexpr int kRows = 128 + kRowsB;
  static constexpr int kBytes = kRows * 128;                    // of one stage
  static constexpr int kStages = kBytes >= 32768 ? 5 : kBytes >= 24576 ? 6 : 8;
  static constexpr int kLoads = kRows * 4 / kWorkers;           // 16-byte pieces of a stage per worker
  static constexpr bool kMove = BN >= 128;                      // registers move to the workers
  static constexpr int kThreads = kMove ? 384 : kWorkers + 32;
  static constexpr int kSmem = kStages * kBytes + 1024 + 256;
};

struct MatArgs {
  LinearArgs a;
  int tiles_n, tiles_m;      // tiles over channels and tokens
};

template <int BN>
__global__ void __launch_bounds__(Shape<BN>::kThreads, 1) matrix_kernel(const MatArgs g) {
  using S = Shape<BN>;
  static_assert(S::kLoads * kWorkers == S::kRows * 4, "whole pieces per worker");
  extern __shared__ uint8_t raw[];
  const LinearArgs &a = g.a;
  const uint32_t base = (tc::smem_addr(raw) + 1023) & ~1023u;
  const uint32_t bars = base + S::kStages * S::kBytes;
  const uint32_t full = bars, empty = full + 8 * S::kStages, acc_full = empty + 8 * S::kStages,
                 acc_empty = acc_full + 16, drain = acc_empty + 16, slot = drain + 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.x, units = gridDim.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; s++) {
      tc::mbar_init(full + 8 * s, 8);
      tc::mbar_init(empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; s++) {
      tc::mbar_init(acc_full + 8 * s, 1);
      tc::mbar_init(acc_empty + 8 * s, 8);
    }
    tc::mbar_init(drain, 1);
    tc::mbar_init_fence();
  }
  if (warp == 8) tc::tmem_alloc<1>(slot, 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(slot));

  const int stages = (a.K + 2 * kStage - 1) / (2 * kStage) * 2, chunks = (stages + kChunk - 1) / kChunk;
  const int tiles = g.tiles_n * g.tiles_m;
  bool dead = false;

  if (warp >= 8) {
    if constexpr (S::kMove) tc::give_registers();
    if (warp == 8 && lane == 0) {
      constexpr uint32_t ins = tc::instruction(128, BN, 0, 0, 0);
      uint32_t it = 0, ch = 0;
      for (int tile = unit; tile < tiles && !dead; tile += units) {
        for (int c = 0; c < chunks && !dead; c++, ch++) {
          const uint32_t set = ch & 1;
          tc::mbar_wait(acc_empty + 8 * set, ((ch >> 1) & 1) ^ 1, dead);
          tc::fence_after();
          const int n = min(kChunk, stages - c * kChunk);
          for (int i = 0; i < n && !dead; i++, it++) {
            const uint32_t s = it % S::kStages;
            tc::mbar_wait(full + 8 * s, (it / S::kStages) & 1, dead);
            tc::fence_after();
            if (dead) break;
            const uint32_t at = base + s * S::kBytes;
            const uint64_t da = tc::operand(at, 16, 1024), db = tc::operand(at + 128 * 128, 16, 1024);
#pragma unroll
            for (int k = 0; k < kStage / 16; k++)
              tc::mma<1>(tmem + set * 256, da + 2 * k, db + 2 * k, ins, (i | k) != 0);
            tc::commit<1>(empty + 8 * s);
          }
          tc::commit<1>(acc_full + 8 * set);
        }
      }
      bool late = false;                       // everything issued has to end before the memory is given back
      tc::commit<1>(drain);
      tc::mbar_wait(drain, 0, late);
    }
    __syncwarp();
  } else {
    if constexpr (S::kMove) tc::take_registers();
    // pieces of a stage: piece p of a row is k 16p .. 16p + 15
    const int piece = threadIdx.x & 3, row0 = threadIdx.x >> 2;
    uint32_t store[S::kLoads];
#pragma unroll
    for (int j = 0; j < S::kLoads; j++) {
      const int r = row0 + 64 * j;
      store[j] = (r >> 3) * 1024 + (r & 7) * 128 + (((2 * piece) ^ (r & 7)) << 4);
    }
    const int8_t *src[S::kLoads];
    bool have[S::kLoads];
    int ltile = unit, lk = 0;                  // the load cursor runs two stages ahead of the store
    auto aim = [&]() {
      if (ltile >= tiles) {
#pragma unroll
        for (int j = 0; j < S::kLoads; j++) have[j] = false;
        return;
      }
      const int n0 = (ltile % g.tiles_n) * 128, m0 = (ltile / g.tiles_n) * BN;
#pragma unroll
      for (int j = 0; j < S::kLoads; j++) {
        const int r = row0 + 64 * j;
        if (r < 128) {
          have[j] = n0 + r < a.N;
          src[j] = a.w + (int64_t)(n0 + r) * a.ldw + 16 * piece;
        } else {
          have[j] = m0 + r - 128 < a.M;
          src[j] = a.x + (int64_t)(m0 + r - 128) * a.ldx + 16 * piece;
        }
      }
    };
    auto load = [&](uint4 (&v)[S::kLoads]) {
      const bool in = lk * kStage + 16 * piece < a.K;
#pragma unroll
      for (int j = 0; j < S::kLoads; j++) {
        v[j] = make_uint4(0, 0, 0, 0);
        if (have[j] && in) v[j] = __ldg((const uint4 *)(src[j] + (int64_t)lk * kStage));
      }
      if (++lk == stages) {
        lk = 0;
        ltile += units;
        aim();
      }
    };
    uint32_t it = 0, ch = 0;
    int tile = unit, c = 0, i = 0;             // the store cursor: tile, chunk of it, stage of the chunk
    int acc[BN / 2];
#pragma unroll
    for (int j = 0; j < BN / 2; j++) acc[j] = 0;
    const uint32_t mine = tmem + ((uint32_t)(warp & 3) << 21) + (warp >> 2) * (BN / 2);
    auto step = [&](uint4 (&v)[S::kLoads]) {
      const uint32_t s = it % S::kStages;
      tc::mbar_wait(empty + 8 * s, ((it / S::kStages) & 1) ^ 1, dead);
      const uint32_t at = base + s * S::kBytes;
#pragma unroll
      for (int j = 0; j < S::kLoads; j++) {
        uint32_t h[8];
        half4(v[j].x, h[0], h[1]);
        half4(v[j].y, h[2], h[3]);
        half4(v[j].z, h[4], h[5]);
        half4(v[j].w, h[6], h[7]);
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at + store[j]), "r"(h[0]), "r"(h[1]), "r"(h[2]),
                     "r"(h[3])
                     : "memory");
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at + (store[j] ^ 16)), "r"(h[4]), "r"(h[5]),
                     "r"(h[6]), "r"(h[7])
                     : "memory");
      }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(full + 8 * s);
      load(v);
      it++;
    };
    uint4 va[S::kLoads], vb[S::kLoads];
    aim();
    load(va);
    load(vb);
    int done_tile = 0;                         // of the chunk that waits to be taken out
    bool done_last = false;
    for (;;) {
      const bool more = tile < tiles;
      if (more) {
        step(va);
        step(vb);
      }
      // A chunk is taken out once the next one is two pairs of stages along (or all there), so
      // that the matrix unit has work meanwhile; the last one, at the end.
      const int n = min(kChunk, stages - c * kChunk);
      if (ch > 0 && (!more || i == min(4, n) - 2)) {
        const uint32_t set = (ch - 1) & 1;
        tc::mbar_wait(acc_full + 8 * set, ((ch - 1) >> 1) & 1, dead);
        __syncwarp();
        tc::fence_after();
        const bool write = done_last;
        const int n = (done_tile % g.tiles_n) * 128 + (warp & 3) * 32 + lane;
        const int m0 = (done_tile / g.tiles_n) * BN + (warp >> 2) * (BN / 2);
        const float sw = write && a.sw && n < a.N ? a.sw[n] : 0.f, bias = write && a.bias && n < a.N ? a.bias[n] : 0.f;
#pragma unroll
        for (int j = 0; j < BN / 2; j += 16) {
          float v[16];
          tc::tmem_load16(mine + set * 256 + j, v);
          tc::tmem_wait();
#pragma unroll
          for (int x = 0; x < 16; x++) acc[j + x] += __float2int_rn(v[x]);
          if (write) {
            if (n < a.N) put_y16(a, m0 + j, n, &acc[j], sw, bias);
#pragma unroll
            for (int x = 0; x < 16; x++) acc[j + x] = 0;
          }
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(acc_empty + 8 * set);
      }
      if (!more) break;
      i += 2;
      if (i == n) {
        done_tile = tile;
        done_last = c == chunks - 1;
        i = 0;
        ch++;
        if (++c == chunks) {
          c = 0;
          tile += units;
        }
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 8) {
    tc::fence_after();
    tc::tmem_free<1>(tmem, 512);
  }
}

template <int BN>
int go_matrix(const LinearArgs &a, cudaStream_t st) {
  using S = Shape<BN>;
  static std::atomic<bool> ready[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MCEMU_ERR_CUDA;
  if (dev >= 64 || !ready[dev].load()) {
    if (cudaFuncSetAttribute(matrix_kernel<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) != cudaSuccess)
      return MCEMU_ERR_CUDA;
    if (dev < 64) ready[dev].store(true);
  }
  MatArgs g{a, (a.N + 127) / 128, (a.M + BN - 1) / BN};
  const int64_t tiles = (int64_t)g.tiles_n * g.tiles_m;
  if (tiles > INT32_MAX / 2) return MCEMU_ERR_UNSUPPORTED;
  matrix_kernel<BN><<<(unsigned)(tiles < sm_count() ? tiles : sm_count()), S::kThreads, S::kSmem, st>>>(g);
  return launch_status();
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

struct LinearEp {
  using Sum = int;
  LinearArgs a;
  static __device__ __forceinline__ void add(int &s, float v) { s += __float2int_rn(v); }
  __device__ __forceinline__ void store(int n, int m0, const int *sum, int) const {
    if (n >= a.N) return;
    const float sw = a.sw ? __ldg(a.sw + n) : 0.f, bias = a.bias ? __ldg(a.bias + n) : 0.f;
    put_y16(a, m0, n, sum, sw, bias);
  }
};

int blocks128(int rows) { return (rows + 255) / 256 * 2; }
int ktiles_of(int K) { return (K + 63) / 64; }

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
  return panel::launch<LinearEp, 0, 0, 0>(g, mw, mx, LinearEp{a}, st);
}

// 32 x 32 outputs to a block of 256 threads, four to a thread.
__global__ void __launch_bounds__(256) linear_kernel(const LinearArgs a) {
  __shared__ int8_t xs[32][36], ws[32][36];
  const int m0 = blockIdx.y * 32, n0 = blockIdx.x * 32;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  int acc[4] = {0, 0, 0, 0};
  for (int k0 = 0; k0 < a.K; k0 += 32) {
#pragma unroll
    for (int r = 0; r < 4; r++) {
      const int i = ty + 8 * r, k = k0 + tx;
      xs[i][tx] = m0 + i < a.M && k < a.K ? a.x[(int64_t)(m0 + i) * a.ldx + k] : 0;
      ws[i][tx] = n0 + i < a.N && k < a.K ? a.w[(int64_t)(n0 + i) * a.ldw + k] : 0;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
      const int wv = *(const int *)&ws[tx][k];
#pragma unroll
      for (int r = 0; r < 4; r++) acc[r] = __dp4a(*(const int *)&xs[ty + 8 * r][k], wv, acc[r]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < 4; r++) {
    const int m = m0 + ty + 8 * r, n = n0 + tx;
    if (m < a.M && n < a.N) put_y(a, m, n, acc[r], a.sw ? a.sw[n] : 0.f, a.bias ? a.bias[n] : 0.f);
  }
}

}  // namespace

int int8_linear_timeouts(cudaStream_t st, unsigned int *got) { return tc::take_timeouts(st, got); }

// Products that go through panels: more than 16 tokens, and either enough of them to pay for
// the panels or rows that are not on 16-byte boundaries.
static bool by_panels(int M, int K, bool rows) { return M > 16 && K > 0 && (M > 256 || !rows || K % 16 != 0); }

size_t int8_linear_workspace(int M, int N, int K, int rows) {
  if (!by_panels(M, K, rows != 0)) return 0;
  return (size_t)(blocks128(M) + blocks128(N)) * ktiles_of(K) * panel::kTileBytes;
}

int launch_int8_linear(const LinearArgs &a, bool rows, void *ws, void *stream) {
  cudaStream_t st = (cudaStream_t)stream;
  if (by_panels(a.M, a.K, rows)) return go_panels(a, rows, ws, st);
  if (a.M > 16 && a.K > 0) {
    if (a.M <= 64) return go_matrix<64>(a, st);
    return go_matrix<128>(a, st);
  }
  linear_kernel<<<dim3((a.N + 31) / 32, (a.M + 31) / 32), 256, 0, st>>>(a);
  return launch_status();
}

}  // namespace mcemu
