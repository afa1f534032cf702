// panel.cuh -- product of two operands in 16-bit floating point on pairs of CTAs.
//
// An operand is either a panel, cut beforehand into tiles of 128 rows by 64 k, each the 16 KB
// image that the matrix instruction reads from shared memory (128-byte swizzle), tiles of
// one 128-row block following one another along k; or (MN-major only) a matrix in global
// memory, k by rows, from which the copy engine makes the same images.
//
// A pair computes 256 rows of A by 256 rows of B: each CTA holds 128 rows of both (32 KB a
// stage) and 128 x 256 accumulators, twice, so that one set is drained while the other
// fills.  The accumulators leave tensor memory every `chunk` stages and are added up in
// registers, in whatever type the caller's sums need; the matrix unit alone would drop the
// low bits of long sums (it truncates, it does not round).
//
// Both CTAs' copies count on the issuing CTA's barrier, by the hardware.  Passing a stage on by
// a thread's arrival on the other CTA's barrier, with the release that it takes, measured
// 0.95 us a stage in place of NEWSTAGE.
#pragma once
#include "ops_common.cuh"
#include "tc.cuh"

namespace mcemu {
namespace panel {

constexpr int kTileBytes = 16384;             // 128 rows x 64 k x 2 bytes
constexpr int kTileK = 64;
constexpr int kStages = 6;
constexpr int kStageBytes = 2 * kTileBytes;
constexpr int kSmem = kStages * kStageBytes + 1024 + 256;
constexpr int kThreads = 384;                 // eight warps drain, one loads, one issues, two are idle

struct Args {
  int ka;                    // tiles along k
  int tiles_a, tiles_b;      // 256-row tiles of either operand
  int splits, per_split;     // parts of the sum, k tiles to a part
  int chunk;                 // stages between two drains
};

// Where a unit of work lies.
struct Unit {
  int ta, tb, split, k0, k1;
};
__device__ __forceinline__ Unit unit_at(const Args &g, int u) {
  Unit r;
  const int tiles = g.tiles_a * g.tiles_b;
  r.split = u / tiles;
  const int t = u - r.split * tiles;
  // bands of eight tiles of A, so that the pairs at work share both operands in L2
  const int band = t / (8 * g.tiles_b), rest = t - band * 8 * g.tiles_b, width = min(8, g.tiles_a - band * 8);
  r.ta = band * 8 + rest % width;
  r.tb = rest / width;
  r.k0 = r.split * g.per_split;
  r.k1 = min(g.ka, r.k0 + g.per_split);
  return r;
}

// Copies the two operands' part of stage k for this CTA.  DIRECT: B is a matrix in memory.
template <int DIRECT>
__device__ __forceinline__ void load_stage(const Args &g, const CUtensorMap *ma, const CUtensorMap *mb, const Unit &w,
                                           int rank, int k, uint32_t at, uint32_t bar) {
  tc::box_load_pair(at, ma, 0, ((2 * w.ta + rank) * g.ka + k) * 128, bar);
  if constexpr (DIRECT) {
    const int x = w.tb * 256 + rank * 128;
    tc::box_load_pair(at + kTileBytes, mb, x, k * kTileK, bar);
    tc::box_load_pair(at + kTileBytes + 8192, mb, x + 64, k * kTileK, bar);
  } else {
    tc::box_load_pair(at + kTileBytes, mb, 0, ((2 * w.tb + rank) * g.ka + k) * 128, bar);
  }
}

// Ep: `Ep::Sum` is the type of the register sums; add(Sum &, float) takes one accumulator;
// store(row of A, row of B, 16 sums along B, split) writes 16 outputs.  MN: operands are
// MN-major; BF16: bfloat16 (else binary16).
template <class Ep, int MN, int BF16, int DIRECT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    panel_kernel(const Args g, const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                 const Ep ep) {
  extern __shared__ uint8_t raw[];
  const uint32_t base = (tc::smem_addr(raw) + 1023) & ~1023u;
  const uint32_t full = base + kStages * kStageBytes, empty = full + 8 * kStages, acc_full = empty + 8 * kStages,
                 acc_empty = acc_full + 16, drain = acc_empty + 16, slot = drain + 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc::cta_rank();
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1, units = g.tiles_a * g.tiles_b * g.splits;

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
  bool dead = false;
  grid_go();
  grid_wait();                                // the panels are the work of the kernel before

  if (warp >= 8) tc::give_registers();
  if (warp == 8 && lane == 0) {               // loads this CTA's half of both operands
    uint32_t it = 0;
    for (int u = first; u < units; u += step) {
      const Unit w = unit_at(g, u);
      for (int k = w.k0; k < w.k1 && !dead; k++, it++) {
        const uint32_t s = it % kStages;
        tc::mbar_wait(empty + 8 * s, ((it / kStages) & 1) ^ 1, dead);
        if (dead) break;
        if (rank == 0) tc::mbar_expect(full + 8 * s, 2 * kStageBytes);
        load_stage<DIRECT>(g, &ma, &mb, w, rank, k, base + s * kStageBytes, full + 8 * s);
      }
    }
    if (rank == 0) {                          // both CTAs' copies end before either leaves
      bool late = false;
      for (uint32_t s = 0; s < kStages && s < it; s++) {
        const uint32_t last = it - 1 - (it - 1 - s) % kStages;      // the last use of slot s
        tc::mbar_wait(full + 8 * s, (last / kStages) & 1, late);
      }
    }
  } else if (warp == 9 && lane == 0 && rank == 0) {   // issues the pair's matrix instructions
    constexpr uint32_t ins = tc::instruction(256, 256, BF16, MN, MN);
    uint32_t it = 0, ch = 0;
    for (int u = first; u < units && !dead; u += step) {
      const Unit w = unit_at(g, u);
      for (int k = w.k0; k < w.k1 && !dead; k += g.chunk, ch++) {
        const uint32_t set = ch & 1;
        tc::mbar_wait(acc_empty + 8 * set, ((ch >> 1) & 1) ^ 1, dead);
        tc::fence_after();
        const int n = min(g.chunk, w.k1 - k);
        for (int i = 0; i < n; i++, it++) {
          const uint32_t s = it % kStages, at = base + s * kStageBytes, fp = (it / kStages) & 1;
          tc::mbar_wait(full + 8 * s, fp, dead);
          if (dead) break;
          tc::fence_after();
          if constexpr (MN) {
            // 64 k = eight atoms of eight; atoms of one k lie 8 KB apart along the rows
            const uint64_t da = tc::operand(at, 8192, 1024), db = tc::operand(at + kTileBytes, 8192, 1024);
#pragma unroll
            for (int x = 0; x < 4; x++) tc::mma<2>(tmem + set * 256, da + 128 * x, db + 128 * x, ins, (i | x) != 0);
          } else {
            const uint64_t da = tc::operand(at, 16, 1024), db = tc::operand(at + kTileBytes, 16, 1024);
#pragma unroll
            for (int x = 0; x < 4; x++) tc::mma<2>(tmem + set * 256, da + 2 * x, db + 2 * x, ins, (i | x) != 0);
          }
          tc::commit<2>(empty + 8 * s);
        }
        tc::commit<2>(acc_full + 8 * set);
      }
    }
    bool late = false;                        // everything issued ends before the memory is given back
    tc::commit_here<2>(drain);
    tc::mbar_wait(drain, 0, late);
  } else if (warp < 8) {
    tc::take_registers();
    const uint32_t mine = tmem + ((uint32_t)(warp & 3) << 21) + (warp >> 2) * 128;
    uint32_t ch = 0;
    for (int u = first; u < units; u += step) {
      const Unit w = unit_at(g, u);
      typename Ep::Sum sum[128];
#pragma unroll
      for (int j = 0; j < 128; j++) sum[j] = 0;
      const int ra = w.ta * 256 + rank * 128 + (warp & 3) * 32 + lane, rb = w.tb * 256 + (warp >> 2) * 128;
      for (int k = w.k0; k < w.k1; k += g.chunk, ch++) {
        const uint32_t set = ch & 1;
        tc::mbar_wait(acc_full + 8 * set, (ch >> 1) & 1, dead);
        __syncwarp();
        tc::fence_after();
        float v[2][16];
        tc::tmem_load16(mine + set * 256, v[0]);
#pragma unroll
        for (int j = 0; j < 128; j += 16) {
          tc::tmem_wait();
          if (j + 16 < 128) tc::tmem_load16(mine + set * 256 + j + 16, v[(j >> 4) + 1 & 1]);
#pragma unroll
          for (int x = 0; x < 16; x++) Ep::add(sum[j + x], v[(j >> 4) & 1][x]);
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_lead(acc_empty + 8 * set);
      }
      // the matrix unit has both sets to go on with meanwhile
#pragma unroll
      for (int j = 0; j < 128; j += 16) ep.store(ra, rb + j, &sum[j], w.split);
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

// Tensor map of a panel of `blocks` 128-row blocks.
inline int panel_map(CUtensorMap *map, const void *panel, int blocks, int ktiles) {
  return tc::tensor_map(map, panel, 64, (uint64_t)blocks * ktiles * 128, 64, 128, false);
}
// What fits a panel: its rows are counted in 32 bits.
inline bool panel_fits(int64_t blocks, int64_t ktiles) { return blocks * ktiles * 128 <= INT32_MAX; }

template <class Ep, int MN, int BF16, int DIRECT>
int launch(const Args &g, const CUtensorMap &ma, const CUtensorMap &mb, const Ep &ep, cudaStream_t st) {
  static std::atomic<bool> ready[64];
  const auto kernel = panel_kernel<Ep, MN, BF16, DIRECT>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MCEMU_ERR_CUDA;
  if (dev >= 64 || !ready[dev].load()) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
      return MCEMU_ERR_CUDA;
    if (dev < 64) ready[dev].store(true);
  }
  const int64_t units = (int64_t)g.tiles_a * g.tiles_b * g.splits;
  if (units > INT32_MAX / 4) return MCEMU_ERR_UNSUPPORTED;
  const int pairs = (int)(units < sm_count() / 2 ? units : sm_count() / 2);
  return launch_early(kernel, dim3(2 * pairs), dim3(kThreads), kSmem, st, g, ma, mb, ep);
}

}  // namespace panel
}  // namespace mcemu
