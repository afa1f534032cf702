// fp8_pair.cuh -- FP8 products of many rows, on pairs of CTAs.
//
// A pair computes tiles of 256 rows of a by BN rows of b: each CTA holds 128 rows of a and half of
// b's, and 128 x BN accumulators, twice, so that one set is drained into registers while the other fills.
// The accumulators leave tensor memory every 1024 of k: the matrix unit truncates what it adds up.  Relative errors
// of 2048 x 4096 x 16384 against 64 bits, for normal values, with large channels and for positive ones: 9.7e-8, 1.2e-7
// and 1.9e-7; of a library's fp32 product of the same numbers 1.9e-7, 2.5e-7 and 8.4e-7.
// The exponents go to tensor memory eight blocks at a time: for a those of the CTA's own rows, for b those
// of all BN, in both CTAs.  (Four at a time the warps that bring them were the slowest: passing them on to
// the issuing CTA takes a release at cluster scope, 0.95 us.)  Tensor memory has 512 columns: two sets of accumulators and two
// of exponents (8 + 16 columns) leave BN at most 224.
//
// TURNED: the operands have changed places, so that a lane's row is a column of y.  A piece of results then leaves as
// rows of 32 neighbours, 128 bytes in fp32, from any row on: groups that begin amid a tile of tokens need no other
// way out, and only the pieces at their ends go by lanes.  Turned and not, us, a few launches and under the power limit:
// 16384 rows of 16 experts of 4096 x 2048 99 and 105, 114 and 120; weight gradients of 8 experts, 4096 x 2048 each in
// fp32, 113 and 123, 124 and 131; 8192 x 8192 x 4096 163 and 165, 187 and 190.
//
// Bound by power where there is much work: 8192 x 8192 x 4096 takes 163 us in a burst (3.4 PFLOP/s), 177 to 193
// under the 1.4 kW limit, at 1.5 GHz.  Of 177, copies without a use would take away 18, results without a
// place 20, both 28; two warps that issue in place of one took away 40, copies by two whole warps in place of a
// lane 15.  A library's product with a scale for each 32 of k, measured beside it: 172.
//
// Weight gradients of few rows an expert wait for their way out: for 8 experts of 4096 x 2048 in fp32, 16 rounds of tiles,
// 8192, 16384 and 32768 rows take 77, 113 and 190 us, so that a block of a tile takes 0.29 us and no blocks at all 40, as long
// as HBM takes for the 268 MB (28 with results in bf16).  A tile's two chunks are too little to hide them behind.
#pragma once
#include "fp8_tc.cuh"

namespace mcemu {
namespace fp8 {

// Eight warps drain; then come one for the copies of a, two that issue matrix instructions, one for the exponents
// of a, one for each 128 rows of b's, and as the last one for the copies of b.
constexpr int kPairThreads = 512;
constexpr int kPairChunk = 8;                 // blocks along k between two drains
// Registers of the warps that hold sums, and of the others: as many as 128 a thread at launch.
__device__ __forceinline__ void pair_take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 200;"); }
__device__ __forceinline__ void pair_give_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 56;"); }
template <int BN>
struct Pair {
  // A block along k has a slot, which is free again when its matrix instructions are done; the blocks are passed
  // on two at a time (a stage), since each wait costs the issuing warp 300 cycles.
  static constexpr int kBlockBytes = kTileBytes + BN / 2 * kBlock;
  static constexpr int kStages = BN > 128 ? 3 : 4, kBlocks = 2 * kStages;
  static constexpr int kRowTiles = 1 + (BN + 127) / 128;        // 128 rows of a and of b, whose exponents a CTA holds
  static constexpr int kScaleSlots = 3, kSlotBytes = 2 * kRowTiles * kScaleBytes;
  // A warp's place for results on their way out: 32 rows of 112 bytes (64), two pieces of its columns in 16 bits,
  // four in fp32.  Sixteen-byte stores of a row to a lane meet no bank twice at 112.
  static constexpr int kPieceBytes = BN == 224 ? 112 : 64, kOutBytes = 8 * 32 * kPieceBytes;
  static constexpr int kSmem =
      kBlocks * kBlockBytes + kScaleSlots * kSlotBytes + kOutBytes + 1024 + 512 + 2 * 4 * (MCEMU_FP8_MAX_GROUPS + 1);
  static_assert(kSmem <= 232448, "shared memory");
};

struct PairUnit {
  int g, a, b, end, k0, k1;  // group, first rows, where the rows of the one with groups end, blocks along k
};
struct PairGroups {
  const int *at, *before;
  int tiles_a, tiles_b, blocks;      // tiles of all rows of a, of b; blocks along k (not by_k)
};
template <bool TURNED>
__device__ __forceinline__ int units_of(const Fp8Product &p, const PairGroups &w) {
  return p.by_k ? p.E * w.tiles_a * w.tiles_b : w.before[p.E] * (TURNED ? w.tiles_a : w.tiles_b);
}
// The u-th unit; g is the group of an earlier one.  Groups are of a's rows, TURNED of b's.  Bands of eight tiles of a, so that the pairs at work
// share both operands in L2.
template <int BN, bool TURNED>
__device__ __forceinline__ PairUnit unit_at(const Fp8Product &p, const PairGroups &w, int u, int &g) {
  PairUnit r;
  int t, tiles_a = w.tiles_a, tiles_b = w.tiles_b;
  if (p.by_k) {
    const int each = tiles_a * tiles_b;
    g = u / each;
    t = u - g * each;
  } else {
    const int others = TURNED ? tiles_a : tiles_b;
    while (u >= w.before[g + 1] * others) g++;
    t = u - w.before[g] * others;
    (TURNED ? tiles_b : tiles_a) = w.before[g + 1] - w.before[g];
  }
  const int band = t / (8 * tiles_b), rest = t - band * 8 * tiles_b, width = min(8, tiles_a - band * 8);
  r.g = g;
  const int begin = p.by_k ? 0 : w.at[g];
  r.a = (TURNED ? 0 : begin) + (band * 8 + rest % width) * 256;
  r.b = (TURNED ? begin : 0) + rest / width * BN;
  r.end = p.by_k ? (TURNED ? p.b : p.a).rows : w.at[g + 1];
  r.k0 = p.by_k ? w.at[g] : 0;
  r.k1 = p.by_k ? w.at[g + 1] : w.blocks;
  return r;
}

// A warp's way through the units, bringing eight blocks' exponents of 128 rows to each slot: of the tile's rows
// of a, or of b, from `skip` on.
template <int BN, bool TURNED>
__device__ __forceinline__ void feed_scales(const Fp8Product &p, const PairGroups &w, int first, int step, int units, bool of_a,
                                            int skip, uint32_t scales, uint32_t sf_full, uint32_t sf_empty, bool &dead) {
  using S = Pair<BN>;
  Scales<4> v;
  uint32_t turn = 0;
  int g = 0;
  for (int u = first; u < units && !dead; u += step) {
    const PairUnit r = unit_at<BN, TURNED>(p, w, u, g);
    const int matrix = of_a != TURNED || p.by_k ? 0 : r.g;
    if (of_a) v.rows(p.a, matrix, r.a + skip);
    else v.rows(p.b, matrix, r.b + skip);
    for (int k = r.k0; k < r.k1; k += kPairChunk, turn++) {
      const uint32_t sf = turn % S::kScaleSlots, to = scales + sf * S::kSlotBytes;
      uint32_t x[2][4];
      v.load(0, k, r.k1, x);
      tc::mbar_wait_warp(sf_empty + 8 * sf, ((turn / S::kScaleSlots) & 1) ^ 1, dead);
      if (dead) return;
      store_scales(to, x[0]);
      store_scales(to + kScaleBytes, x[1]);
      tc::fence_async_smem();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive_at(sf_full + 8 * sf, 0);
    }
  }
}

// The units' chunks of `set`'s turn (every other one): waits for their operands and exponents and issues their
// matrix instructions into that set of accumulators.  By two warps, one to a set: waiting, passing on and issuing
// cost a warp some 2700 cycles for four blocks, and the matrix unit takes 1800 for them.
// A stage's barrier tells one use from the next by parity alone, so that a stage may be waited for only when its
// use before is known to be over: the warps pass a token (`pass`) when the last stage of a chunk has come.
template <int BN, bool TURNED>
__device__ __forceinline__ void issue(const Fp8Product &p, const PairGroups &w, int first, int step, int units, uint32_t set,
                                      uint32_t tmem, uint32_t base, uint32_t scales, uint32_t full, uint32_t empty,
                                      uint32_t sf_full, uint32_t sf_empty, uint32_t acc_full, uint32_t acc_empty,
                                      uint32_t drain, uint32_t pass, bool &dead) {
  using S = Pair<BN>;
  constexpr int kB = S::kRowTiles - 1;
  const uint32_t ins = instruction(256, BN, p.a.fmt, p.b.fmt), d = tmem + set * 256, sa = d + BN, sb = sa + 8;
  uint32_t s = 0, phase = 0, ch = 0, parity = 1;
  int g = 0;
  for (int u = first; u < units && !dead; u += step) {
    const PairUnit r = unit_at<BN, TURNED>(p, w, u, g);
    for (int k = r.k0; k < r.k1 && !dead; k += kPairChunk, ch++) {
      const int n = min(kPairChunk, r.k1 - k);
      if ((ch & 1) != set) {
        for (int i = 0; i < n; i += 2)
          if (++s == S::kStages) s = 0, phase ^= 1;
        continue;
      }
      const uint32_t sf = ch % S::kScaleSlots, from = scales + sf * S::kSlotBytes;
      tc::mbar_wait_warp(acc_empty, parity, dead);
      mbar_wait_warp_cluster(sf_full + 8 * sf, (ch / S::kScaleSlots) & 1, dead);
      if (dead) break;
      tc::fence_after();
      // into the columns of this set's chunk before, whose accumulators have been drained
#pragma unroll
      for (int t = 0; t < 2; t++) copy_scales<2>(sa + 4 * t, from + t * kScaleBytes);
#pragma unroll
      for (int t = 0; t < 2 * kB; t++)        // b's first four blocks of all its rows, then the other four
        copy_scales<2>(sb + 4 * ((t & 1) * kB + (t >> 1)), from + (2 + t) * kScaleBytes);
      tc::commit<2>(sf_empty + 8 * sf);
      tc::mbar_wait_warp(pass + 8 * set, parity ^ set, dead);     // set 0 begins
      parity ^= 1;
      for (int i = 0; i < n; i += 2) {
        tc::mbar_wait_warp(full + 8 * s, phase, dead);
        if (dead) break;
        if (i + 2 >= n && (threadIdx.x & 31) == 0) tc::mbar_arrive(pass + 8 * (set ^ 1));
        __syncwarp();
        tc::fence_after();
        const uint32_t half = i >> 2, fa = sa + 4 * half, fb = sb + 4 * kB * half, word = ins + (i & 3) * kNextByte;
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const uint32_t ta = base + (2 * s + h) * S::kBlockBytes;
          const uint64_t da = tc::operand(ta, 16, 1024), db = tc::operand(ta + kTileBytes, 16, 1024);
          if (i + h < n) {
#pragma unroll
            for (int x = 0; x < 4; x++) mma<2>(d, da + 2 * x, db + 2 * x, word + h * kNextByte, fa, fb, (i | h | x) != 0);
          }
          tc::commit<2>(empty + 8 * (2 * s + h));
        }
        if (++s == S::kStages) s = 0, phase ^= 1;
      }
      if (!dead) tc::commit<2>(acc_full);
    }
  }
  bool late = false;                          // everything issued ends before the memory is given back
  tc::commit_here<2>(drain);
  tc::mbar_wait_warp(drain, 0, late);
}

// Rows of N results from shared memory, by a warp, as vectors of type V.
template <class T, class V, int N>
__device__ __forceinline__ void copy_rows(T *y, int64_t ld, const T *from, int rows) {
  constexpr int kEach = sizeof(V) / sizeof(T), kRow = N / kEach;
#pragma unroll 4
  for (int t = threadIdx.x & 31; t < kRow * rows; t += 32) {
    const int i = t / kRow, c = t % kRow * kEach;
    *(V *)(y + i * ld + c) = *(const V *)(from + i * N + c);
  }
}

template <class T, int BN, bool TURNED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    pair_kernel(const Fp8Product p, const __grid_constant__ CUtensorMap ma,
                const __grid_constant__ CUtensorMap mb, const __grid_constant__ CUtensorMap my, bool boxes) {
  using S = Pair<BN>;
  constexpr int kStages = S::kStages, kBlocks = S::kBlocks, kSlots = S::kScaleSlots, kCols = BN / 2;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (tc::smem_addr(raw) + 1023) & ~1023u;
  const uint32_t scales = base + kBlocks * S::kBlockBytes, out = scales + kSlots * S::kSlotBytes, full = out + S::kOutBytes,
                 empty = full + 8 * kStages, sf_full = empty + 8 * kBlocks, sf_empty = sf_full + 8 * kSlots, acc_full = sf_empty + 8 * kSlots,
                 acc_empty = acc_full + 16, drain = acc_empty + 16, pass = drain + 16, slot = pass + 16;
  int *at = (int *)(raw + (slot + 16 - tc::smem_addr(raw))), *before = at + MCEMU_FP8_MAX_GROUPS + 1;
  const int warp = tc::warp_number(), lane = threadIdx.x & 31;
  const uint32_t rank = tc::cta_rank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; s++) tc::mbar_init(full + 8 * s, 1);
    for (int s = 0; s < kBlocks; s++) tc::mbar_init(empty + 8 * s, 1);
    for (int s = 0; s < kSlots; s++) {
      tc::mbar_init(sf_full + 8 * s, 2 * S::kRowTiles);         // a warp of each CTA for each 128 rows, on CTA 0's
      tc::mbar_init(sf_empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; s++) {
      tc::mbar_init(acc_full + 8 * s, 1);
      tc::mbar_init(acc_empty + 8 * s, 16);
      tc::mbar_init(drain + 8 * s, 1);
      tc::mbar_init(pass + 8 * s, 1);
    }
    tc::mbar_init_fence();
  }
  if (warp == 8) tc::tmem_alloc<2>(slot, 512);
  grid_go();
  grid_wait();                                // operands and offsets may be the work of the kernel before
  if (warp == 0) place_groups(p, TURNED ? BN : 256, at, before);
  tc::fence_before();
  tc::cluster_sync();
  tc::fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(slot));
  tmem = __shfl_sync(0xFFFFFFFFu, tmem, 0);
  bool dead = false;
  const PairGroups w{at, before, (p.a.rows + 255) / 256, (p.b.rows + BN - 1) / BN, (p.K + kBlock - 1) / kBlock};
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1, units = units_of<TURNED>(p, w);
  int g = 0;

  if (warp >= 8) pair_give_registers();
  if (warp == 8 || warp == 15) {              // copies this CTA's half of a, or of b
    const bool of_a = warp == 8;
    const CUtensorMap *map = of_a ? &ma : &mb;
    const uint32_t lead = at_rank(full, 0);
    uint32_t s = 0, stage = 0, phase = 1, it = 0;
    for (int u = first; u < units && !dead; u += step) {
      const PairUnit r = unit_at<BN, TURNED>(p, w, u, g);
      const int y = of_a ? r.a + (int)rank * 128 : r.b + (int)rank * (BN / 2), z = of_a != TURNED || p.by_k ? 0 : r.g;
      for (int k = r.k0; k < r.k1 && !dead; k += 2, it++) {
        const int n = min(2, r.k1 - k);
#pragma unroll
        for (int h = 0; h < 2; h++) {
          tc::mbar_wait_warp(empty + 8 * (s + h), phase, dead);  // of a block that there is not, too: see issue()
          if (dead) break;
          if (h == 0 && of_a && rank == 0 && lane == 0) tc::mbar_expect(full + 8 * stage, n * 2 * S::kBlockBytes);
          __syncwarp();
          if (h < n)
            box_load_pair(base + (s + h) * S::kBlockBytes + (of_a ? 0 : kTileBytes), map, (k + h) * kBlock, y, z, lead + 8 * stage);
        }
        s += 2;
        if (++stage == kStages) s = 0, stage = 0, phase ^= 1;
      }
    }
    if (of_a && rank == 0) {                  // all copies end before either CTA leaves
      bool late = false;
      for (uint32_t q = 0; q < kStages && q < it; q++) {
        const uint32_t last = it - 1 - (it - 1 - q) % kStages;        // the last use of stage q
        tc::mbar_wait_warp(full + 8 * q, (last / kStages) & 1, late);
      }
    }
  } else if (warp == 9 || warp == 10) {
    const uint32_t set = warp - 9;
    if (rank == 0)
      issue<BN, TURNED>(p, w, first, step, units, set, tmem, base, scales, full, empty, sf_full, sf_empty, acc_full + 8 * set,
                acc_empty + 8 * set, drain + 8 * set, pass, dead);
  } else if (warp == 11) {
    feed_scales<BN, TURNED>(p, w, first, step, units, true, (int)rank * 128, scales, sf_full, sf_empty, dead);
  } else if (warp > 11 && warp < 11 + S::kRowTiles) {
    feed_scales<BN, TURNED>(p, w, first, step, units, false, (warp - 12) * 128, scales + (warp - 11) * 2 * kScaleBytes, sf_full, sf_empty, dead);
  } else if (warp < 8) {
    pair_take_registers();
    const uint32_t mine = tmem + ((uint32_t)(warp & 3) << 21) + (warp >> 2) * kCols;
    uint32_t ch = 0;
    for (int u = first; u < units; u += step) {
      const PairUnit r = unit_at<BN, TURNED>(p, w, u, g);
      float sum[kCols];
#pragma unroll
      for (int j = 0; j < kCols; j++) sum[j] = 0.f;
      for (int k = r.k0; k < r.k1; k += kPairChunk, ch++) {
        const uint32_t set = ch & 1;
        tc::mbar_wait_warp(acc_full + 8 * set, (ch >> 1) & 1, dead);       // a whole warp's verdict: what follows is one's
        __syncwarp();
        tc::fence_after();
        float v[2][16];
        tc::tmem_load16(mine + set * 256, v[0]);
#pragma unroll
        for (int j = 0; j < kCols; j += 16) {
          tc::tmem_wait();
          if (j + 16 < kCols) tc::tmem_load16(mine + set * 256 + j + 16, v[(j >> 4) + 1 & 1]);
#pragma unroll
          for (int x = 0; x < 16; x++) sum[j + x] += v[(j >> 4) & 1][x];
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_lead(acc_empty + 8 * set);
      }
      // Out through shared memory, where the copy engine takes over while the matrix unit goes on with both sets (weight
      // gradients of 8 experts, 2048 x 4096 x 2048 each in fp32: not TURNED by the threads themselves 16 bytes of 32 rows at a
      // time for every other piece 1.24 of its time, by rows 1.04, with larger pieces and fewer slots 1.02; TURNED by the
      // threads themselves 1.04).  What the copy engine cannot write (rows that end a group amid the warp's, or TURNED
      // amid a piece; other alignments; the end of a row of y amid 16 bytes, which it fills with zeros to the end of
      // them, beside y) leaves by rows.
      constexpr int kPiece = S::kPieceBytes / sizeof(T), kVec = 16 / sizeof(T);
      const int row0 = r.a + (int)rank * 128 + (warp & 3) * 32, col0 = r.b + (warp >> 2) * kCols, z = p.by_k ? r.g : 0;
      const uint32_t place = out + warp * 32 * S::kPieceBytes;
      const bool whole = boxes && (row0 + 32 <= r.end || r.end == p.a.rows);
      const int row = TURNED ? p.a.rows : p.b.rows, inside = row * (int64_t)sizeof(T) % 16 ? row : INT32_MAX;     // of y
      if constexpr (TURNED) {                 // a lane's row of a is a column of y
        if (p.bias) {
          const float b = row0 + lane < p.a.rows ? __ldg(p.bias + row0 + lane) : 0.f;
#pragma unroll
          for (int j = 0; j < kCols; j++) sum[j] += b;
        }
      } else if (p.bias) {
        if (((uintptr_t)p.bias & 15) == 0 && col0 + kCols <= p.b.rows) {
#pragma unroll
          for (int j = 0; j < kCols; j += 4) {
            const float4 b = __ldg((const float4 *)(p.bias + col0 + j));
            sum[j] += b.x, sum[j + 1] += b.y, sum[j + 2] += b.z, sum[j + 3] += b.w;
          }
        } else {
#pragma unroll
          for (int j = 0; j < kCols; j++) sum[j] += col0 + j < p.b.rows ? __ldg(p.bias + col0 + j) : 0.f;
        }
      }
      if (row0 >= (TURNED ? p.a.rows : r.end) || dead) continue;
      if (p.accumulate && r.k0 == r.k1) continue;      // nothing to add: even a zero would change -0 and, by the copy engine, subnormals
      if constexpr (TURNED) {
        T *y = (T *)p.y + z * p.stride_y + (int64_t)col0 * p.ldy + row0 + lane;
#pragma unroll
        for (int j = 0; j < kCols; j += kPiece) {
          if (col0 + j >= r.end) break;
          if (boxes && row0 + 32 <= inside && (col0 + j + kPiece <= r.end || r.end == p.b.rows)) {
            if (lane == 0) boxes_left();
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kPiece; i++) put_shared<T>(place + (i * 32 + lane) * (int)sizeof(T), sum[j + i]);
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) box_store(&my, place, row0, col0 + j, z, p.accumulate);
          } else if (row0 + lane < p.a.rows) {
#pragma unroll
            for (int i = 0; i < kPiece; i++)
              if (col0 + j + i < r.end) put(y + (j + i) * p.ldy, sum[j + i], p.accumulate);
          }
        }
        continue;
      }
#pragma unroll
      for (int j = 0; j < kCols; j += kPiece) {
        if (col0 + j >= p.b.rows) break;
        if (lane == 0) boxes_left();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kPiece; i += kVec) {
          const uint4 v = pack16<T>(&sum[j + i]);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(place + lane * S::kPieceBytes + i * (int)sizeof(T)), "r"(v.x),
                       "r"(v.y), "r"(v.z), "r"(v.w)
                       : "memory");
        }
        if (whole && col0 + j + kPiece <= inside) {
          tc::fence_async_smem();
          __syncwarp();
          if (lane == 0) box_store(&my, place, col0 + j, row0, z, p.accumulate);
        } else {
          __syncwarp();
          const T *from = (const T *)(raw + (place - tc::smem_addr(raw)));
          T *y = (T *)p.y + z * p.stride_y + (int64_t)row0 * p.ldy + col0 + j;
          const int rows = min(32, r.end - row0), cols = min(kPiece, p.b.rows - col0 - j);
          const uint32_t where = (uint32_t)((uintptr_t)y | (uintptr_t)(p.ldy * (int64_t)sizeof(T)));
          if (cols < kPiece || p.accumulate || where % (sizeof(T) == 2 ? 4 : 8)) {
#pragma unroll 8
            for (int i = 0; i < rows; i++)
#pragma unroll
              for (int c = lane; c < kPiece; c += 32)
                if (c < cols) put_as(y + i * p.ldy + c, from[i * kPiece + c], p.accumulate);
          } else if (where % 16 == 0) {
            copy_rows<T, uint4, kPiece>(y, p.ldy, from, rows);
          } else if (where % 8 == 0) {
            copy_rows<T, uint2, kPiece>(y, p.ldy, from, rows);
          } else {
            copy_rows<T, typename std::conditional<sizeof(T) == 2, uint32_t, uint2>::type, kPiece>(y, p.ldy, from, rows);
          }
        }
      }
    }
    if (lane == 0) boxes_written();
  }
  __syncwarp();
  tc::fence_before();
  tc::cluster_sync();
  if (warp == 8) {
    tc::fence_after();
    tc::tmem_free<2>(tmem, 512);
  }
}

template <class T, int BN, bool TURNED>
int launch_pair(const Fp8Product &p, const CUtensorMap &ma, const CUtensorMap &mb, int64_t units, cudaStream_t st) {
  constexpr int kSize = sizeof(T);
  const bool boxes = rows16(p.y, p.ldy, kSize) && (!p.by_k || p.E == 1 || p.stride_y * kSize % 16 == 0);
  CUtensorMap my = ma;
  if (boxes) {
    constexpr int kPiece = Pair<BN>::kPieceBytes / kSize;
    const int rc = TURNED ? tensor_map(&my, p.out_fmt, p.y, p.a.rows, p.b.rows, p.ldy, p.by_k ? p.E : 1, p.stride_y, 32, kPiece)
                          : tensor_map(&my, p.out_fmt, p.y, p.b.rows, p.a.rows, p.ldy, p.by_k ? p.E : 1, p.stride_y, kPiece, 32);
    if (rc != MCEMU_OK) return rc;
  }
  if (!allow_smem<pair_kernel<T, BN, TURNED>>(Pair<BN>::kSmem)) return MCEMU_ERR_CUDA;
  const int pairs = units < sm_count() / 2 ? (int)units : sm_count() / 2;
  return launch_early(pair_kernel<T, BN, TURNED>, dim3(2 * pairs), dim3(kPairThreads), Pair<BN>::kSmem, st, p, ma, mb, my, boxes);
}

}  // namespace fp8
}  // namespace mcemu
