// int8_linear.cu -- product of 8-bit integers with a scale for each token and channel
// (include/mcemu_ops.h has the formula).
//
// sm_103a has no fast 8-bit integer matrix instruction, so the sums run on the 16-bit floating
// one, exactly: an 8-bit integer is a binary16 number, a product is at most 2^14 in magnitude, and
// a sum of 1024 products is an integer of at most 2^24, which fp32 accumulators hold without
// rounding (every partial sum too, in any order, dropped bits or not).  Every 1024 products the
// accumulators are therefore taken out and added to int32 sums in registers.
//
// Three forms, chosen by form_of() below: few tokens (the weights' bytes are most of the work), a batch
// of them (bound by the widening of the weights), many (bound by the matrix unit).
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
// Many tokens: both operands are widened to binary16 panels once (3 bytes of traffic an element,
// against a conversion for every tile that reads it), and pairs of CTAs multiply the panels
// with nothing but copies and matrix instructions in the loop.  Bound by the matrix unit:
// 8192 x 8192 x 4096 to bf16 takes 319 us, 29 of them the widening (6.9 TB/s, some of it to L2):
// 1.72 PFLOP/s, 0.90 of the measured bf16 rate; the matrix unit is 84 % busy while it runs.
// ---------------------------------------------------------------------------
struct Widen {
  const int8_t *src;
  int64_t ld;
  int rows, blocks;          // rows, and 128-row blocks of the panel
  uint8_t *to;
};

// One tile (128 rows by 64 k) to a block, two pieces of sixteen k to a thread.  A piece becomes 32
// bytes, which the swizzle keeps in one sector, its halves exchanged in odd rows.
__global__ void __launch_bounds__(256) widen_kernel(const Widen x, const Widen w, int K, int ktiles, bool wide) {
  int64_t tile = blockIdx.x;
  grid_go();
  const int64_t mine = (int64_t)x.blocks * ktiles;
  const Widen &o = tile < mine ? x : w;
  if (tile >= mine) tile -= mine;
  const int block = (int)(tile / ktiles), kt = (int)(tile - (int64_t)block * ktiles);
  uint8_t *to = o.to + tile * panel::kTileBytes;
  const int piece = threadIdx.x & 3, r0 = threadIdx.x >> 2, k = kt * 64 + 16 * piece;
  uint4 v[2];
#pragma unroll
  for (int j = 0; j < 2; j++) {
    const int row = block * 128 + r0 + 64 * j;
    v[j] = make_uint4(0, 0, 0, 0);
    if (row < o.rows && k < K) v[j] = row16(o.src + (int64_t)row * o.ld, k, K, wide);
  }
#pragma unroll
  for (int j = 0; j < 2; j++) {
    const int r = r0 + 64 * j;
    uint4 lo, hi;
    half4(v[j].x, lo.x, lo.y);
    half4(v[j].y, lo.z, lo.w);
    half4(v[j].z, hi.x, hi.y);
    half4(v[j].w, hi.z, hi.w);
    store32(to + r * 128 + ((piece ^ ((r & 7) >> 1)) << 5), r & 1 ? hi : lo, r & 1 ? lo : hi);
  }
}

template <int OUT>
struct LinearEp {
  using Sum = int;
  LinearArgs a;
  static __device__ __forceinline__ void add(int &s, float v) { s += __float2int_rn(v); }
  __device__ __forceinline__ void store(const panel::Unit &, int n, int m0, const int *sum) const {
    if (n >= a.N) return;
    put16<OUT>(a, m0, n, sum, channel<OUT>(a, n));
  }
};

int blocks128(int rows) { return (rows + 255) / 256 * 2; }
int ktiles_of(int K) { return (K + 63) / 64; }

template <int OUT>
int go_panels(const LinearArgs &a, bool wide, void *ws, cudaStream_t st) {
  const int kt = ktiles_of(a.K);
  Widen x{a.x, a.ldx, a.M, blocks128(a.M), panels_in(ws)};
  Widen w{a.w, a.ldw, a.N, blocks128(a.N), x.to + (int64_t)x.blocks * kt * panel::kTileBytes};
  const int64_t tiles = (int64_t)(x.blocks + w.blocks) * kt;
  if (!panel::panel_fits(x.blocks, kt) || !panel::panel_fits(w.blocks, kt)) return MCEMU_ERR_UNSUPPORTED;
  widen_kernel<<<(unsigned)tiles, 256, 0, st>>>(x, w, a.K, kt, wide);
  const int rc = launch_status();
  if (rc != MCEMU_OK) return rc;              // the panels would be whatever the workspace held
  return panel::launch<LinearEp<OUT>, 0, 0>(panel::plan_of(a.N, a.M, kt, false), w.to, a.N, x.to, a.M, nullptr, 0, a.K,
                                            kt, 1024 / panel::kTileK, LinearEp<OUT>{a}, st);
}

// ---------------------------------------------------------------------------
// Few tokens: the weights' bytes are what counts, and every warp widens what it reads in
// registers.  A block takes 16 channels by 8 * NT tokens; its eight warps share K, 64 at a
// time in turn.  The warp-wide matrix instruction (m16n8k16, 1000 MAC a cycle and SM measured,
// against 250 for its 8-bit form and for dp4a alike) takes four k of a row from a lane, and
// which four is free as long as both operands agree: a lane reads 16 consecutive bytes of
// its rows and feeds them to four instructions.  One token by 4096 x 4096 weights: 4.7 us (3.5
// TB/s of weights, launch included), 16 tokens 5.5, 32 tokens 8.0 (there the matrix instructions
// and the widening of the tokens, done by every block, weigh as much as the loads).  Weights
// larger than L2 are no faster, half the memory's rate (16384 x 4096 19.2 us under the profiler): at K =
// 4096 a warp's share is one round of loads, and a block has none in flight while it works.
// ---------------------------------------------------------------------------
constexpr int kWarps = 8;

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// Sixteen bytes of a row from k on, asked for at one time and put together at another, so that many
// can be in flight.  WIDE: rows start on 16-byte boundaries and K is a multiple of 16.  Otherwise
// five aligned words around them where `inner` says that those lie within the row, for all lanes
// alike, and lane by lane near its ends.  A choice at each load made each wait for the one before
// it (1 x 20000 x 5001: 41 us, now 31; 16 x 9000 x 9001: 61, 37; 8 x 9000 x 9001: 29.8, 32.0).
template <bool WIDE>
struct Piece;
template <>
struct Piece<true> {
  uint4 v;
  __device__ __forceinline__ void ask(const int8_t *row, int k, int K, bool have, bool) {
    v = have && k < K ? __ldg((const uint4 *)(row + k)) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ uint32_t word(int q, const int8_t *, bool) const { return (&v.x)[q]; }
};
template <>
struct Piece<false> {
  uint32_t v[5];
  __device__ __forceinline__ void ask(const int8_t *row, int k, int K, bool have, bool inner) {
    if (inner) {
      const uint32_t *p = (const uint32_t *)(row + k - ((uintptr_t)row & 3));
#pragma unroll
      for (int i = 0; i < 5; i++) v[i] = have ? __ldg(p + i) : 0;
    } else {
      const uint4 x = have && k < K ? row16(row, k, K, false) : make_uint4(0, 0, 0, 0);
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = 0;
    }
  }
  __device__ __forceinline__ uint32_t word(int q, const int8_t *row, bool inner) const {
    return __funnelshift_r(v[q], v[q + 1], inner ? 8 * ((uint32_t)(uintptr_t)row & 3) : 0);
  }
};

__device__ __forceinline__ void put_any(const LinearArgs &a, int m, int n, int acc, float sx, float sw, float bias) {
  const int64_t at = (int64_t)m * a.ldy + n;
  const bool biased = a.bias != nullptr;
  if (a.out_fmt == MCEMU_BF16) ((__nv_bfloat16 *)a.y)[at] = scaled<MCEMU_BF16>(acc, sx, sw, biased, bias);
  else if (a.out_fmt == MCEMU_FP16) ((__half *)a.y)[at] = scaled<MCEMU_FP16>(acc, sx, sw, biased, bias);
  else if (a.out_fmt == MCEMU_FP32) ((float *)a.y)[at] = scaled<MCEMU_FP32>(acc, sx, sw, biased, bias);
  else ((int32_t *)a.y)[at] = acc;
}

template <int NT, bool WIDE>
__global__ void __launch_bounds__(32 * kWarps) few_kernel(const LinearArgs a, int blocks_n) {
  // pieces of 64 k in flight (unaligned rows: four of them measured 9.7 us for 1 x 4096 x 4099, two 8.7)
  constexpr int kAhead = WIDE ? (NT == 1 ? 8 : 4) : 2;
  constexpr int kOut = 16 * 8 * NT;                          // outputs of a block
  constexpr int kEach = (kOut + 32 * kWarps - 1) / (32 * kWarps);
  __shared__ int part[kWarps][kOut];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int mb = blockIdx.x / blocks_n, n0 = (blockIdx.x - mb * blocks_n) * 16, m0 = mb * 8 * NT;
  // this thread's outputs (a channel, every sixteenth token), their factors asked for early
  const int n = n0 + (threadIdx.x & 15);
  const bool scales = a.out_fmt != MCEMU_INT32;
  float sx[kEach];
#pragma unroll
  for (int i = 0; i < kEach; i++) {
    const int m = m0 + (threadIdx.x >> 4) + 16 * i;
    sx[i] = scales && m < a.M ? __ldg(a.sx + m) : 0.f;
  }
  const float sw = scales && n < a.N ? __ldg(a.sw + n) : 0.f, bias = scales && a.bias && n < a.N ? __ldg(a.bias + n) : 0.f;

  const int8_t *wrow[2], *xrow[NT];
  bool whave[2], xhave[NT];
#pragma unroll
  for (int r = 0; r < 2; r++) {
    whave[r] = n0 + 8 * r + g < a.N;
    wrow[r] = a.w + (whave[r] ? (int64_t)(n0 + 8 * r + g) * a.ldw : 0);
  }
#pragma unroll
  for (int j = 0; j < NT; j++) {
    xhave[j] = m0 + 8 * j + g < a.M;
    xrow[j] = a.x + (xhave[j] ? (int64_t)(m0 + 8 * j + g) * a.ldx : 0);
  }
  float acc[NT][4];
  int sum[NT][4];
#pragma unroll
  for (int i = 0; i < NT * 4; i++) (&acc[0][0])[i] = 0.f, (&sum[0][0])[i] = 0;

  const int pieces = (a.K + 63) / 64;
  int since = 0;                                             // pieces since the sums were taken out
  for (int p = warp; p < pieces; p += kWarps * kAhead) {
    Piece<WIDE> w[kAhead][2], x[kAhead][NT];
    bool inner[kAhead];              // whether the words around the piece lie within the rows
#pragma unroll
    for (int u = 0; u < kAhead; u++) {
      const int pu = p + u * kWarps, k = pu * 64 + 16 * t;
      inner[u] = !WIDE && pu > 0 && pu * 64 + 64 + 4 <= a.K;
#pragma unroll
      for (int r = 0; r < 2; r++) w[u][r].ask(wrow[r], k, a.K, whave[r], inner[u]);
#pragma unroll
      for (int j = 0; j < NT; j++) x[u][j].ask(xrow[j], k, a.K, xhave[j], inner[u]);
    }
#pragma unroll
    for (int u = 0; u < kAhead; u++) {
#pragma unroll
      for (int q = 0; q < 4; q++) {
        uint32_t af[4];
        half4(w[u][0].word(q, wrow[0], inner[u]), af[0], af[2]);
        half4(w[u][1].word(q, wrow[1], inner[u]), af[1], af[3]);
#pragma unroll
        for (int j = 0; j < NT; j++) {
          uint32_t bf[2];
          half4(x[u][j].word(q, xrow[j], inner[u]), bf[0], bf[1]);
          mma16816(acc[j], af, bf);
        }
      }
    }
    since += kAhead;
    if (since + kAhead > 16 || p + kWarps * kAhead >= pieces) {   // 1024 products an accumulator at most
#pragma unroll
      for (int i = 0; i < NT * 4; i++) {
        (&sum[0][0])[i] += __float2int_rn((&acc[0][0])[i]);
        (&acc[0][0])[i] = 0.f;
      }
      since = 0;
    }
  }
#pragma unroll
  for (int j = 0; j < NT; j++)
#pragma unroll
    for (int i = 0; i < 4; i++) part[warp][(8 * j + 2 * t + (i & 1)) * 16 + 8 * (i >> 1) + g] = sum[j][i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEach; i++) {
    const int at = threadIdx.x + 32 * kWarps * i, m = m0 + (at >> 4);
    if (at >= kOut || n >= a.N || m >= a.M) continue;
    int total = part[0][at];
#pragma unroll
    for (int p = 1; p < kWarps; p++) total += part[p][at];
    put_any(a, m, n, total, sx[i], sw, bias);
  }
}

template <int NT>
int go_few(const LinearArgs &a, bool wide, cudaStream_t st) {
  const int64_t blocks_n = ((int64_t)a.N + 15) / 16, blocks = blocks_n * (((int64_t)a.M + 8 * NT - 1) / (8 * NT));
  if (blocks > INT32_MAX) return MCEMU_ERR_UNSUPPORTED;
  if (wide) few_kernel<NT, true><<<(unsigned)blocks, 32 * kWarps, 0, st>>>(a, (int)blocks_n);
  else few_kernel<NT, false><<<(unsigned)blocks, 32 * kWarps, 0, st>>>(a, (int)blocks_n);
  return launch_status();
}

// ---------------------------------------------------------------------------
// A batch of tokens, too few to pay for panels: a block takes 128 channels by BN tokens and a part
// of K.  Worker warps read both operands 128 k at a time, kAhead stages ahead, widen them to
// binary16 and store them in the swizzle; one warp issues the matrix instructions.  The
// blocks of a cluster share K, and each adds up its share of the tile out of the others' shared
// memory, so that no second launch joins the parts.  128 x 8192 x 4096: 19.4 us (1.7 TB/s of
// weights).  Bound by the widening: some 60 instructions for 16 elements of a lane, sixteen warps
// on the four schedulers; the matrix unit is a fifth busy.  Rows that 16-byte loads do not fit cost
// another 15 to shift a piece into place (WIDE: none such; 128 x 8192 x 4097: 26.3 us).
// ---------------------------------------------------------------------------
constexpr int kStageK = 128;                  // k of a stage: two 128-byte swizzle rows, the first 64 k of all rows first
constexpr int kChunk = 1024 / kStageK;        // stages between two transfers to int32

template <int BN, bool WIDE>
struct Batch {
  static constexpr int kWorkers = 512;
  static constexpr int kEach = BN / (kWorkers / 128);           // accumulator columns a worker drains
  static constexpr int kRows = 128 + BN;
  static constexpr int kHalf = kRows * 128, kBytes = 2 * kHalf; // of one stage
  static constexpr int kStages = 2;
  static constexpr int kPass = kWorkers / 8;                    // rows that the workers load at a time
  static constexpr int kLoads = kRows / kPass;
  static constexpr int kRowBytes = WIDE ? kStageK : 192;        // of a row's copy
  static constexpr int kAhead = (BN <= 64 ? 4 : 3) - !WIDE;     // stages whose copies are in flight: what memory holds
  static constexpr int kColumns = BN;                           // tensor memory: a power of two, 32 at least
  static constexpr int kCopies = kAhead * kRows * kRowBytes;
  static constexpr int kSmem = kStages * kBytes + kCopies + 1024 + 256;     // also holds the tile's 128 * BN sums
};

template <int BN, bool WIDE>
__global__ void __launch_bounds__(Batch<BN, WIDE>::kWorkers + 32, 1) batch_kernel(const LinearArgs a, int tiles_n,
                                                                                  int per) {
  using S = Batch<BN, WIDE>;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (tc::smem_addr(raw) + 1023) & ~1023u;
  const uint32_t copies = base + S::kStages * S::kBytes, full = copies + S::kCopies, empty = full + 8 * S::kStages,
                 acc_full = empty + 8 * S::kStages, acc_empty = acc_full + 8, drain = acc_empty + 8, slot = drain + 8;
  constexpr int kMma = S::kWorkers / 32;        // the warp that issues
  const int warp = tc::warp_number(), lane = threadIdx.x & 31;
  const uint32_t parts = tc::cluster_size(), rank = tc::cta_rank();
  const int tile = blockIdx.x / parts, n0 = (tile % tiles_n) * 128, m0 = (tile / tiles_n) * BN;
  const int stages = (a.K + kStageK - 1) / kStageK, s0 = (int)rank * per;
  const int s1 = max(s0, min(stages, s0 + per));

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; s++) {
      tc::mbar_init(full + 8 * s, kMma);
      tc::mbar_init(empty + 8 * s, 1);
    }
    tc::mbar_init(acc_full, 1);
    tc::mbar_init(acc_empty, kMma);
    tc::mbar_init(drain, 1);
    tc::mbar_init_fence();
  }
  if (warp == kMma) tc::tmem_alloc<1>(slot, S::kColumns);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(slot));
  tmem = __shfl_sync(0xFFFFFFFFu, tmem, 0);
  bool dead = false;
  int sum[S::kEach];
#pragma unroll
  for (int j = 0; j < S::kEach; j++) sum[j] = 0;

  if (warp == kMma) {
    constexpr uint32_t ins = tc::instruction(128, BN, 0, 0, 0);
    uint32_t it = 0, ch = 0;
    for (int c = s0; c < s1 && !dead; c += kChunk, ch++) {
      tc::mbar_wait_warp(acc_empty, (ch & 1) ^ 1, dead);
      tc::fence_after();
      const int n = min(kChunk, s1 - c);
      for (int i = 0; i < n && !dead; i++, it++) {
        const uint32_t s = it % S::kStages, at = base + s * S::kBytes;
        tc::mbar_wait_warp(full + 8 * s, (it / S::kStages) & 1, dead);
        if (dead) break;
        tc::fence_after();
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const uint32_t half = at + h * S::kHalf;
          const uint64_t da = tc::operand(half, 16, 1024), db = tc::operand(half + 128 * 128, 16, 1024);
#pragma unroll
          for (int k = 0; k < 4; k++) tc::mma<1>(tmem, da + 2 * k, db + 2 * k, ins, (i | h | k) != 0);
        }
        tc::commit<1>(empty + 8 * s);
      }
      tc::commit<1>(acc_full);
    }
    bool late = false;                       // everything issued ends before the memory is given back
    tc::commit<1>(drain);
    tc::mbar_wait_warp(drain, 0, late);
  } else {
    // Pieces of a stage: piece p of a row is k 16p .. 16p + 15.  A warp reads whole 128-byte
    // lines of four rows; eight lanes that store together hold two rows' pieces of one half,
    // which lie in different banks.
    const int piece = (lane & 3) + 4 * (lane >> 4), row0 = warp * 4 + ((lane >> 2) & 3);
    const uint32_t store = (piece >> 2) * S::kHalf + (row0 >> 3) * 1024 + (row0 & 7) * 128 +
                           (((2 * (piece & 3)) ^ (row0 & 7)) << 4);      // of row0; kPass rows on, 128 bytes each
    const int8_t *pw = a.w + (int64_t)(n0 + row0) * a.ldw + 16 * piece, *px = a.x + (int64_t)(m0 + row0) * a.ldx + 16 * piece;
    const int rows_w = a.N - n0 - row0, rows_x = a.M - m0 - row0;
    // WIDE: a thread copies its pieces ahead into places of its own, so that no barrier and no
    // register waits for them (loaded to registers one stage ahead: 128 x 8192 x 4096 in 22 us in
    // place of 20.1).
    // Otherwise a warp copies the aligned units around its rows, nine to a row and stage, and a
    // lane takes its piece out of two of them (with copies of single words in place of units
    // 128 x 8192 x 4097 took 34 us).  Rows lie 192 bytes apart, so that eight lanes that load
    // together read different banks.  Bytes beyond K are not read but zeros; up to 15 before a
    // row, in the unit that holds its first, are read and shifted out.
    const uint32_t place = WIDE ? copies + threadIdx.x * 16 : copies + warp * (4 * S::kLoads * S::kRowBytes);
    const int rows_mine_w = a.N - n0 - warp * 4, rows_mine_x = a.M - m0 - warp * 4;
    const auto unit_of = [&](int r, int unit, int &off) {          // of row r after the warp's first
      const int8_t *p = r < 128 ? a.w + (int64_t)(n0 + warp * 4 + r) * a.ldw : a.x + (int64_t)(m0 + warp * 4 + r - 128) * a.ldx;
      off = (int)((uintptr_t)p & 15);
      return p - off + 16 * unit;
    };
    // a lane copies unit lane & 7 of row lane / 8 and those 64 rows on, and one row's ninth
    int off_uw, off_ux, off_ut;
    const int lane_row = lane >> 3, unit = lane & 7, tail_row = S::kPass * (lane >> 2) + (lane & 3);
    const int8_t *uw = unit_of(lane_row, unit, off_uw), *ux = unit_of(128 + lane_row, unit, off_ux),
                 *ut = unit_of(tail_row, 8, off_ut);
    const bool tail = lane < 4 * S::kLoads;
    const bool tail_in = tail && (tail_row < 128 ? tail_row < rows_mine_w : tail_row - 128 < rows_mine_x);
    const auto copy_unit = [&](uint32_t to, const int8_t *from, int left) {        // left: bytes of the row from there on
      const int bytes = max(0, min(16, left));
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to),
                   "l"(bytes ? from : (const int8_t *)((uintptr_t)a.w & ~(uintptr_t)15)), "r"(bytes)
                   : "memory");
    };
    const auto copy = [&](int s) {
      const uint32_t to = place + (uint32_t)((s - s0) % S::kAhead) * (S::kRows * S::kRowBytes);
      if constexpr (WIDE) {
        const int k = s < s1 ? s * kStageK : a.K;
        const bool in = k + 16 * piece < a.K;
#pragma unroll
        for (int j = 0; j < S::kLoads; j++) {
          const int r = S::kPass * j;                    // rows after row0
          const bool is_w = r < 128, have = in && (is_w ? r < rows_w : r - 128 < rows_x);
          const int8_t *from = !have ? a.w : is_w ? pw + r * a.ldw + k : px + (r - 128) * a.ldx + k;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + j * S::kWorkers * 16), "l"(from),
                       "r"(have ? 16 : 0)
                       : "memory");
        }
      } else if (s < s1) {
        const int k = s * kStageK;
#pragma unroll
        for (int j = 0; j < S::kLoads; j++) {
          const int r = S::kPass * j;
          const uint32_t at = to + (4 * j + lane_row) * S::kRowBytes + 16 * unit;
          if (r < 128) copy_unit(at, uw + r * a.ldw + k, lane_row + r < rows_mine_w ? a.K + off_uw - 16 * unit - k : 0);
          else
            copy_unit(at, ux + (r - 128) * a.ldx + k, lane_row + r - 128 < rows_mine_x ? a.K + off_ux - 16 * unit - k : 0);
        }
        if (tail) copy_unit(to + lane * S::kRowBytes + 128, ut + k, tail_in ? a.K + off_ut - 128 - k : 0);
      }
      copy_commit();
    };
    // where a row's first byte lies in its unit: the same for rows 64 apart
    const int off_w = (int)((uintptr_t)pw & 15), off_x = (int)((uintptr_t)px & 15);
    uint32_t it = 0;
    const auto step = [&](int stage) {
      const uint32_t s = it % S::kStages, at = base + s * S::kBytes;
      copy_wait<S::kAhead - 1>();
      uint4 v[S::kLoads];
      const uint32_t mine = place + (uint32_t)((stage - s0) % S::kAhead) * (S::kRows * S::kRowBytes);
      if constexpr (!WIDE) __syncwarp();
#pragma unroll
      for (int j = 0; j < S::kLoads; j++) {
        if constexpr (WIDE) {
          asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(v[j].x), "=r"(v[j].y), "=r"(v[j].z), "=r"(v[j].w)
                       : "r"(mine + j * S::kWorkers * 16)
                       : "memory");
        } else {
          uint32_t u[8];
          const int off = S::kPass * j < 128 ? off_w : off_x;
#pragma unroll
          for (int i = 0; i < 8; i += 4)
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(u[i]), "=r"(u[i + 1]), "=r"(u[i + 2]), "=r"(u[i + 3])
                         : "r"(mine + (4 * j + ((lane >> 2) & 3)) * S::kRowBytes + 16 * piece + 4 * i)
                         : "memory");
#pragma unroll
          for (int i = 0; i < 6; i++) u[i] = off & 8 ? u[i + 2] : u[i];
#pragma unroll
          for (int i = 0; i < 5; i++) u[i] = off & 4 ? u[i + 1] : u[i];
          const uint32_t shift = 8 * (off & 3);
          v[j] = make_uint4(__funnelshift_r(u[0], u[1], shift), __funnelshift_r(u[1], u[2], shift),
                            __funnelshift_r(u[2], u[3], shift), __funnelshift_r(u[3], u[4], shift));
        }
      }
      tc::mbar_wait(empty + 8 * s, ((it / S::kStages) & 1) ^ 1, dead);
#pragma unroll
      for (int j = 0; j < S::kLoads; j++) {
        uint32_t h[8];
        half4(v[j].x, h[0], h[1]);
        half4(v[j].y, h[2], h[3]);
        half4(v[j].z, h[4], h[5]);
        half4(v[j].w, h[6], h[7]);
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at + store + 128 * S::kPass * j), "r"(h[0]), "r"(h[1]), "r"(h[2]),
                     "r"(h[3])
                     : "memory");
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at + (store ^ 16) + 128 * S::kPass * j), "r"(h[4]), "r"(h[5]),
                     "r"(h[6]), "r"(h[7])
                     : "memory");
      }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(full + 8 * s);
      copy(stage + S::kAhead);
      it++;
    };
#pragma unroll
    for (int i = 0; i < S::kAhead; i++) copy(s0 + i);
    const uint32_t mine = tmem + ((uint32_t)(warp & 3) << 21) + (warp >> 2) * S::kEach;
    uint32_t ch = 0;
    for (int c = s0; c < s1; c += kChunk, ch++) {
      const int e = min(s1, c + kChunk);
      for (int s = c; s < e; s++) step(s);
      tc::mbar_wait(acc_full, ch & 1, dead);
      __syncwarp();
      tc::fence_after();
#pragma unroll
      for (int j = 0; j < S::kEach; j += 16) {
        float f[16];
        tc::tmem_load16(mine + j, f);
        tc::tmem_wait();
#pragma unroll
        for (int x = 0; x < 16; x++) sum[j + x] += __float2int_rn(f[x]);
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(acc_empty);
    }
  }
  copy_wait<0>();
  // sums to shared memory (token by channel), then this block's tokens out of every block's
  __syncthreads();
  if (warp < kMma) {
    const uint32_t at = base + ((warp >> 2) * S::kEach * 128 + (warp & 3) * 32 + lane) * 4;
#pragma unroll
    for (int j = 0; j < S::kEach; j++)
      asm volatile("st.shared.s32 [%0], %1;" ::"r"(at + j * 512), "r"(sum[j]) : "memory");
  }
  tc::cluster_sync();
  if (warp < kMma) {
    // four channels of every kMma-th token to a thread; all blocks' parts asked for at once
    const int r = lane * 4, n = n0 + r, share = (BN + parts - 1) / parts;
    const int end = min(a.M - m0, min(BN, (int)(rank + 1) * share));
    const bool scales = a.out_fmt != MCEMU_INT32;
    float sw[4], bias[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      sw[i] = scales && n + i < a.N ? __ldg(a.sw + n + i) : 0.f;
      bias[i] = scales && a.bias && n + i < a.N ? __ldg(a.bias + n + i) : 0.f;
    }
    for (int m = rank * share + warp; m < end; m += kMma) {
      const float sx = scales ? __ldg(a.sx + m0 + m) : 0.f;
      int4 v[8];
#pragma unroll
      for (uint32_t p = 0; p < 8; p++)
        if (p < parts) v[p] = tc::load_peer(base + (m * 128 + r) * 4, p);
      int sum4[4] = {0, 0, 0, 0};
#pragma unroll
      for (uint32_t p = 0; p < 8; p++)
        if (p < parts) sum4[0] += v[p].x, sum4[1] += v[p].y, sum4[2] += v[p].z, sum4[3] += v[p].w;
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (n + i < a.N) put_any(a, m0 + m, n + i, sum4[i], sx, sw[i], bias[i]);
    }
  }
  tc::fence_before();
  tc::cluster_sync();
  if (warp == kMma) {
    tc::fence_after();
    tc::tmem_free<1>(tmem, S::kColumns);
  }
}

// Parts of K, one to a block of a cluster (eight at most, the portable limit; two stages each at
// least), so that the stages that blocks go through one after another are fewest, with four more for
// each round of clusters after the first.  The clusters that run at a time are what a GB300
// of 152 multiprocessors reports for blocks that take one each: the larger, the fewer fit.  (A
// table, since the form, and with it the workspace's size, is known without a device.)  200 x 1024 x
// 4096 in six parts 11.5 us, in eight (two rounds) 18.3; 77 x 5003 x 2049 in three 12.8, in two 17.0;
// 128 x 12288 x 4096 in one 32.8, in four (three rounds) 36.2.
struct Split {
  int parts;
  int64_t steps;             // stages in a row and what rounds add
};
Split split_of(int64_t tiles, int stages) {
  constexpr int kClusters[9] = {0, 152, 76, 46, 36, 28, 23, 15, 15};
  Split best{1, 0};
  for (int parts = 1; parts <= 8 && (parts == 1 || stages >= 2 * parts); parts++) {
    const int64_t rounds = (tiles + kClusters[parts] - 1) / kClusters[parts];
    const int64_t steps = rounds * ((stages + parts - 1) / parts + 4) - 4;
    if (parts == 1 || steps < best.steps) best = Split{parts, steps};
  }
  return best;
}

template <int BN, bool WIDE>
int go_batch(const LinearArgs &a, cudaStream_t st) {
  using S = Batch<BN, WIDE>;
  static std::atomic<bool> ready[64];
  const auto kernel = batch_kernel<BN, WIDE>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MCEMU_ERR_CUDA;
  if (dev >= 64 || !ready[dev].load()) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) != cudaSuccess)
      return MCEMU_ERR_CUDA;
    if (dev < 64) ready[dev].store(true);
  }
  const int tiles_n = (a.N + 127) / 128, stages = (a.K + kStageK - 1) / kStageK;
  const int64_t tiles = (int64_t)tiles_n * ((a.M + BN - 1) / BN);
  const int parts = split_of(tiles, stages).parts;
  if (tiles * parts > INT32_MAX) return MCEMU_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * parts));
  cfg.blockDim = dim3(S::kWorkers + 32);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = parts;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t rc = cudaLaunchKernelEx(&cfg, kernel, a, tiles_n, (stages + parts - 1) / parts);
  return rc == cudaSuccess ? MCEMU_OK : MCEMU_ERR_CUDA;
}
// Which form: what ends soonest by these estimates in microseconds, whose constants are measured.
//
//                        batch  panels                           batch  panels
//   128 x  8192 x 4096    19.4    34.9      1024 x 2048 x 2048    21.1    16.0
//   256 x  8192 x 4096    32.8    35.9      2048 x 1024 x 1024    15.0    11.9
//   512 x  1024 x 1024     8.7    11.2      48 x 16384 x 4096     27.9    57.1
//   128 x  8192 x 4097    26.4    37.5      1024 x 2048 x 2049    28.2    18.2
//   256 x  8192 x 4097    45.0    38.3      77 x 5003 x 2049      12.7    18.8
//
// Few tokens, and K = 0, go the first way: 32 tokens by 4096 x 4096 (8192 x 4096) weights 8.0 us
// (14.4) against 10.7 (16.6) of the second.  Over rows that 16-byte loads do not fit it is the
// better up to 16 tokens (4096 x 4099: 12.0, 13.8), and beyond only for little work (32 tokens by
// 4096 x 4099: 18.0, 13.8; 1000 x 263: 5.5, 8.7).
enum class Form { few, batch, panels };

Form form_of(int M, int N, int K, bool wide) {
  if (M <= (wide ? 32 : 16) || K == 0) return Form::few;
  const int bn = M <= 64 ? 64 : 128, stages = (K + kStageK - 1) / kStageK;
  const int64_t tiles = ((int64_t)N + 127) / 128 * (((int64_t)M + bn - 1) / bn);
  const double stage = wide ? (bn == 64 ? 0.67 : 0.88) : (bn == 64 ? 0.90 : 1.20);
  const double batch = 6.0 + split_of(tiles, stages).steps * stage;
  if (M <= 32 && 4.5 + (double)N * K / 1.4e6 < batch) return Form::few;
  const panel::Plan p = panel::plan_of(N, M, ktiles_of(K), false);
  const double panels = 7.0 + 3.0 * ((double)M + N) * K / 6.9e6 + p.us;
  return panels < batch ? Form::panels : Form::batch;
}

}  // namespace

int int8_linear_timeouts(cudaStream_t st, unsigned int *got) { return tc::take_timeouts(st, got); }

size_t int8_linear_workspace(int M, int N, int K, bool rows) {
  if (form_of(M, N, K, rows && K % 16 == 0) != Form::panels) return 0;
  return (size_t)(blocks128(M) + blocks128(N)) * ktiles_of(K) * panel::kTileBytes + kPanelPad;
}

int launch_int8_linear(const LinearArgs &a, bool rows, void *ws, void *stream) {
  cudaStream_t st = (cudaStream_t)stream;
  const bool wide = rows && a.K % 16 == 0;
  switch (form_of(a.M, a.N, a.K, wide)) {
    case Form::few:
      if (a.M <= 8) return go_few<1>(a, wide, st);
      if (a.M <= 16) return go_few<2>(a, wide, st);
      return go_few<4>(a, wide, st);
    case Form::batch:
      if (a.M <= 64) return wide ? go_batch<64, true>(a, st) : go_batch<64, false>(a, st);
      return wide ? go_batch<128, true>(a, st) : go_batch<128, false>(a, st);
    default: break;
  }
  switch (a.out_fmt) {
    case MCEMU_INT32: return go_panels<MCEMU_INT32>(a, rows, ws, st);
    case MCEMU_FP32: return go_panels<MCEMU_FP32>(a, rows, ws, st);
    case MCEMU_FP16: return go_panels<MCEMU_FP16>(a, rows, ws, st);
    default: return go_panels<MCEMU_BF16>(a, rows, ws, st);
  }
}

}  // namespace mcemu
