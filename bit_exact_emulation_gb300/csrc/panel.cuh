// panel.cuh -- product of two operands in 16-bit floating point on pairs of CTAs.
//
// An operand is either a panel, cut beforehand into tiles of 128 rows by 64 k, each the 16 KB
// image that the matrix instruction reads from shared memory (128-byte swizzle), tiles of
// one 128-row block following one another along k; or (MN-major only) a matrix in global
// memory, k by rows, from which the copy engine makes the same images.
//
// A pair computes 256 rows of A by BN (256 or 128) rows of B: each CTA holds 128 rows of A and half
// of B's (32 or 24 KB a stage) and 128 x BN accumulators, twice, so that one set is drained
// while the other fills.  The accumulators leave tensor memory every `chunk` stages and are added up in
// registers, in whatever type the caller's sums need; the matrix unit alone would drop the
// low bits of long sums (it truncates, it does not round).
//
// Both CTAs' copies count on the issuing CTA's barrier, by the hardware.  Passing a stage on by
// a thread's arrival on the other CTA's barrier, with the release that it takes, measured
// 0.95 us a k tile; now one takes 0.33 (256 x 256 x 64 on a pair, the clock under load).
#pragma once
#include "ops_common.cuh"
#include "tc.cuh"

namespace mcemu {
namespace panel {

constexpr int kTileBytes = 16384;             // 128 rows x 64 k x 2 bytes
constexpr int kTileK = 64;
template <int BN>
struct Size {
  static constexpr int kTilesBytes = kTileBytes + BN * 64;      // of one k tile: 128 rows of A, BN / 2 of B
  static constexpr int kStageBytes = 2 * kTilesBytes;           // a stage is two k tiles
  static constexpr int kStages = BN == 256 ? 3 : 4;
  static constexpr int kSmem = kStages * kStageBytes + 1024 + 256;
};
constexpr int kThreads = 384;                 // eight warps drain, one loads, one issues, two are idle

struct Args {
  int ka;                    // tiles along k
  int tiles_a, tiles_b;      // tiles of 256 rows of A and of BN rows of B
  int full, rest;            // tiles computed by one pair, and tiles whose sum several pairs share
  int parts, per_part;       // pairs to each of the latter, k tiles to a pair
  int chunk;                 // k tiles between two drains, an even number
};

// Where a unit of work lies: a tile, and of a shared one the slot of its part (-1 otherwise).
struct Unit {
  int ta, tb, slot, k0, k1;
};
__device__ __forceinline__ void tile_at(const Args &g, int t, int &ta, int &tb) {
  // bands of eight tiles of A, so that the pairs at work share both operands in L2
  const int band = t / (8 * g.tiles_b), rest = t - band * 8 * g.tiles_b, width = min(8, g.tiles_a - band * 8);
  ta = band * 8 + rest % width;
  tb = rest / width;
}
__device__ __forceinline__ int units_of(const Args &g) { return g.full + g.rest * g.parts; }
__device__ __forceinline__ Unit unit_at(const Args &g, int u) {
  Unit r;
  r.slot = u - g.full;
  const int part = r.slot < 0 ? 0 : r.slot / g.rest;
  tile_at(g, r.slot < 0 ? u : g.full + r.slot - part * g.rest, r.ta, r.tb);
  r.k0 = part * g.per_part;
  r.k1 = r.slot < 0 ? g.ka : min(g.ka, r.k0 + g.per_part);
  return r;
}

// Copies the two operands' part of k tile k for this CTA.  DIRECT: B is a matrix in memory.  The
// boxes of B's map are BN / 2 rows of a panel, or 64 by 64 elements of a matrix.
template <int BN, int DIRECT>
__device__ __forceinline__ void load_tiles(const Args &g, const CUtensorMap *ma, const CUtensorMap *mb, const Unit &w,
                                           int rank, int k, uint32_t at, uint32_t bar) {
  tc::box_load_pair(at, ma, 0, ((2 * w.ta + rank) * g.ka + k) * 128, bar);
  if constexpr (DIRECT) {
    const int x = w.tb * BN + rank * (BN / 2);
    tc::box_load_pair(at + kTileBytes, mb, x, k * kTileK, bar);
    if constexpr (BN == 256) tc::box_load_pair(at + kTileBytes + 8192, mb, x + 64, k * kTileK, bar);
  } else {
    const int block = BN == 256 ? 2 * w.tb + rank : w.tb;
    tc::box_load_pair(at + kTileBytes, mb, 0, (block * g.ka + k) * 128 + (BN == 256 ? 0 : 64 * rank), bar);
  }
}

// Ep: `Ep::Sum` is the type of the register sums; add(Sum &, float) takes one accumulator;
// store(unit, row of A, row of B, 16 sums along B) writes 16 outputs (a shared tile's part).  MN: operands are
// MN-major; BF16: bfloat16 (else binary16).
template <class Ep, int BN, int MN, int BF16, int DIRECT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    panel_kernel(const Args g, const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                 const Ep ep) {
  using S = Size<BN>;
  constexpr int kStages = S::kStages, kStageBytes = S::kStageBytes, kCols = BN / 2;      // columns a warp drains
  extern __shared__ uint8_t raw[];
  const uint32_t base = (tc::smem_addr(raw) + 1023) & ~1023u;
  const uint32_t full = base + kStages * kStageBytes, empty = full + 8 * kStages, acc_full = empty + 8 * kStages,
                 acc_empty = acc_full + 16, drain = acc_empty + 16, slot = drain + 8;
  const int warp = tc::warp_number(), lane = threadIdx.x & 31;
  const uint32_t rank = tc::cta_rank();
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1, units = units_of(g);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; s++) {
      tc::mbar_init(full + 8 * s, 1);
      tc::mbar_init(empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; s++) {
      tc::mbar_init(acc_full + 8 * s, 1);
      tc::mbar_init(acc_empty + 8 * s, 16);
    }
    tc::mbar_init(drain, 1);
    tc::mbar_init_fence();
  }
  if (warp == 8) tc::tmem_alloc<2>(slot, 512);
  tc::fence_before();
  tc::cluster_sync();
  tc::fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(slot));
  tmem = __shfl_sync(0xFFFFFFFFu, tmem, 0);
  bool dead = false;
  grid_go();
  grid_wait();                                // the panels are the work of the kernel before

  if (warp >= 8) tc::give_registers();
  if (warp == 8 && lane == 0) {               // loads this CTA's half of both operands
    uint32_t it = 0;
    for (int u = first; u < units; u += step) {
      const Unit w = unit_at(g, u);
      for (int k = w.k0; k < w.k1 && !dead; k += 2, it++) {
        const uint32_t s = it % kStages, at = base + s * kStageBytes;
        const bool two = k + 1 < w.k1;
        tc::mbar_wait(empty + 8 * s, ((it / kStages) & 1) ^ 1, dead);
        if (dead) break;
        if (rank == 0) tc::mbar_expect(full + 8 * s, (two ? 4 : 2) * S::kTilesBytes);
        load_tiles<BN, DIRECT>(g, &ma, &mb, w, rank, k, at, full + 8 * s);
        if (two) load_tiles<BN, DIRECT>(g, &ma, &mb, w, rank, k + 1, at + S::kTilesBytes, full + 8 * s);
      }
    }
    if (rank == 0) {                          // both CTAs' copies end before either leaves
      bool late = false;
      for (uint32_t s = 0; s < kStages && s < it; s++) {
        const uint32_t last = it - 1 - (it - 1 - s) % kStages;      // the last use of slot s
        tc::mbar_wait(full + 8 * s, (last / kStages) & 1, late);
      }
    }
  } else if (warp == 9 && rank == 0) {        // issues the pair's matrix instructions
    constexpr uint32_t ins = tc::instruction(256, BN, BF16, MN, MN);
    uint32_t s = 0, phase = 0, ch = 0;
    for (int u = first; u < units && !dead; u += step) {
      const Unit w = unit_at(g, u);
      for (int k = w.k0; k < w.k1 && !dead; k += g.chunk, ch++) {
        const uint32_t set = ch & 1, d = tmem + set * 256;
        tc::mbar_wait_warp(acc_empty + 8 * set, ((ch >> 1) & 1) ^ 1, dead);
        tc::fence_after();
        const int n = min(g.chunk, w.k1 - k);
        bool add = false;
        for (int i = 0; i < n; i += 2) {
          const uint32_t at = base + s * kStageBytes;
          tc::mbar_wait_warp(full + 8 * s, phase, dead);
          if (dead) break;
          tc::fence_after();
#pragma unroll
          for (int h = 0; h < 2; h++) {
            if (h && i + 1 >= n) break;
            // 64 k: MN-major eight atoms of eight, atoms of one k 8 KB apart along the rows
            const uint32_t ta = at + h * S::kTilesBytes, tb = ta + kTileBytes;
            const uint64_t da = MN ? tc::operand(ta, 8192, 1024) : tc::operand(ta, 16, 1024);
            const uint64_t db = MN ? tc::operand(tb, 8192, 1024) : tc::operand(tb, 16, 1024);
#pragma unroll
            for (int x = 0; x < 4; x++) {
              tc::mma<2>(d, da + (MN ? 128 : 2) * x, db + (MN ? 128 : 2) * x, ins, add);
              add = true;
            }
          }
          tc::commit<2>(empty + 8 * s);
          if (++s == kStages) s = 0, phase ^= 1;
        }
        tc::commit<2>(acc_full + 8 * set);
      }
    }
    bool late = false;                        // everything issued ends before the memory is given back
    tc::commit_here<2>(drain);
    tc::mbar_wait_warp(drain, 0, late);
  } else if (warp < 8) {
    tc::take_registers();
    const uint32_t mine = tmem + ((uint32_t)(warp & 3) << 21) + (warp >> 2) * kCols;
    uint32_t ch = 0;
    for (int u = first; u < units; u += step) {
      const Unit w = unit_at(g, u);
      typename Ep::Sum sum[kCols];
#pragma unroll
      for (int j = 0; j < kCols; j++) sum[j] = 0;
      const int ra = w.ta * 256 + rank * 128 + (warp & 3) * 32 + lane, rb = w.tb * BN + (warp >> 2) * kCols;
      for (int k = w.k0; k < w.k1; k += g.chunk, ch++) {
        const uint32_t set = ch & 1;
        tc::mbar_wait(acc_full + 8 * set, (ch >> 1) & 1, dead);
        __syncwarp();
        tc::fence_after();
        float v[2][16];
        tc::tmem_load16(mine + set * 256, v[0]);
#pragma unroll
        for (int j = 0; j < kCols; j += 16) {
          tc::tmem_wait();
          if (j + 16 < kCols) tc::tmem_load16(mine + set * 256 + j + 16, v[(j >> 4) + 1 & 1]);
#pragma unroll
          for (int x = 0; x < 16; x++) Ep::add(sum[j + x], v[(j >> 4) & 1][x]);
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_lead(acc_empty + 8 * set);
      }
      // the matrix unit has both sets to go on with meanwhile
#pragma unroll
      for (int j = 0; j < kCols; j += 16) ep.store(w, ra, rb + j, &sum[j]);
    }
  }
  __syncwarp();
  tc::fence_before();
  tc::cluster_sync();
  if (warp == 8) {
    tc::fence_after();
    tc::tmem_free<2>(tmem, 512);
  }
}

// Tensor map of a panel of `blocks` 128-row blocks, in boxes of `box` rows.
inline int panel_map(CUtensorMap *map, const void *panel, int blocks, int ktiles, int box) {
  return tc::tensor_map(map, panel, 64, (uint64_t)blocks * ktiles * 128, 64, box, false);
}
// What fits a panel: its rows are counted in 32 bits.
inline bool panel_fits(int64_t blocks, int64_t ktiles) { return blocks * ktiles * 128 <= INT32_MAX; }

// How a product is cut.  Every pair takes a tile at a time; what does not fill a last round may
// be shared (share = true): each of those tiles' sums by as many pairs as there are for it, in
// parts of at least eight k tiles that a second kernel joins.  Tiles have 128 rows of B in place of
// 256 where that ends sooner.  Of the possible cuts the one that an estimate in microseconds
// prefers: 0.33 a k tile of a round, 0.62 of that with 128 rows, 3 and the traffic of the parts for a
// join.  Weight gradients (accumulators taken out every 16 tiles), microseconds:
//
//                            256 rows   128 rows   shared
//   8192 x 4096 x 4096          182        196       169      (256 rows; 28 tiles of 256 shared)
//   1024 x 1024 x 1024          13.6       9.9      11.4      (128 rows)
//
// The pairs are those of a GB300's 152 multiprocessors: the workspace's size goes by the cut and is
// known without a device.  A launch has as many as there are.
constexpr int kPairs = 76;
struct Plan {
  int bn, full, rest, parts, per_part;
  double us;
};
inline Plan plan_of(int rows_a, int rows_b, int ktiles, bool share) {
  Plan best{};
  for (int bn = 256; bn >= 128; bn /= 2) {
    const int64_t tiles = ((int64_t)rows_a + 255) / 256 * (((int64_t)rows_b + bn - 1) / bn), rest = tiles % kPairs;
    const double round = ktiles * (bn == 256 ? 0.33 : 0.33 * 0.62), whole = (double)((tiles + kPairs - 1) / kPairs) * round;
    if (bn == 256 || whole < best.us) best = Plan{bn, (int)tiles, 0, 1, ktiles, whole};
    int parts = share && rest ? (int)(kPairs / rest) : 1;
    if (parts > ktiles / 8) parts = ktiles / 8;
    if (parts < 2) continue;
    const int per = (ktiles + parts - 1) / parts;
    parts = (ktiles + per - 1) / per;
    const double us = ((double)(tiles / kPairs) + (double)per / ktiles) * round + 3.0 + rest * parts * bn * 2048 / 6e6;
    if (us < best.us) best = Plan{bn, (int)(tiles - rest), (int)rest, parts, per, us};
  }
  return best;
}

template <class Ep, int BN, int MN, int BF16, int DIRECT>
int launch_tiles(const Args &g, const CUtensorMap &ma, const CUtensorMap &mb, const Ep &ep, cudaStream_t st) {
  static std::atomic<bool> ready[64];
  const auto kernel = panel_kernel<Ep, BN, MN, BF16, DIRECT>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MCEMU_ERR_CUDA;
  if (dev >= 64 || !ready[dev].load()) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Size<BN>::kSmem) != cudaSuccess)
      return MCEMU_ERR_CUDA;
    if (dev < 64) ready[dev].store(true);
  }
  const int units = g.full + g.rest * g.parts, pairs = units < sm_count() / 2 ? units : sm_count() / 2;
  return launch_early(kernel, dim3(2 * pairs), dim3(kThreads), Size<BN>::kSmem, st, g, ma, mb, ep);
}

// The product of panel a (rows_a rows) and b: a panel, or with `matrix` (MN-major) a matrix of
// k rows and ld elements between them.
template <class Ep, int MN, int BF16>
int launch(const Plan &p, const void *a, int rows_a, const void *b, int rows, const void *matrix, int64_t ld, int k,
           int ktiles, int chunk, const Ep &ep, cudaStream_t st) {
  if (((int64_t)rows_a + 255) / 256 * (((int64_t)rows + 127) / 128) > INT32_MAX / 4) return MCEMU_ERR_UNSUPPORTED;
  const int bn = p.bn, blocks_a = (rows_a + 255) / 256 * 2, blocks_b = (rows + 255) / 256 * 2;
  CUtensorMap ma, mb;
  int rc = panel_map(&ma, a, blocks_a, ktiles, 128);
  if (rc == MCEMU_OK)
    rc = matrix ? tc::tensor_map(&mb, matrix, rows, k, ld, 64, true) : panel_map(&mb, b, blocks_b, ktiles, bn / 2);
  if (rc != MCEMU_OK) return rc;
  const Args g{ktiles, blocks_a / 2, (rows + bn - 1) / bn, p.full, p.rest, p.parts, p.per_part, chunk};
  if constexpr (MN) {
    if (matrix)
      return bn == 256 ? launch_tiles<Ep, 256, MN, BF16, 1>(g, ma, mb, ep, st)
                       : launch_tiles<Ep, 128, MN, BF16, 1>(g, ma, mb, ep, st);
  }
  return bn == 256 ? launch_tiles<Ep, 256, MN, BF16, 0>(g, ma, mb, ep, st)
                   : launch_tiles<Ep, 128, MN, BF16, 0>(g, ma, mb, ep, st);
}

}  // namespace panel
}  // namespace mcemu
