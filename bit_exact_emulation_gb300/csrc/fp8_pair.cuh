// fp8_pair.cuh -- FP8 products of many rows, on pairs of CTAs.
//
// A pair computes tiles of 256 rows of a by BN rows of b: each CTA holds 128 rows of a and half of
// b's, and 128 x BN accumulators, twice, so that one set is drained into registers while the other fills.
// The exponents of a chunk (four blocks along k) go to tensor memory with the chunk: for a those of
// the CTA's own rows, for b those of all BN, in both CTAs.  Tensor memory has 512 columns: two sets of
// accumulators and two of exponents (4 + 8 columns) leave BN at most 224.
#pragma once
#include "fp8_tc.cuh"

namespace mcemu {
namespace fp8 {

constexpr int kPairThreads = 384;             // eight warps drain, then: copies, matrix instructions, exponents of a, of b
template <int BN>
struct Pair {
  static constexpr int kStageBytes = kTileBytes + BN / 2 * kBlock;
  static constexpr int kStages = BN > 192 ? 7 : BN > 128 ? 7 : 8;
  static constexpr int kScaleSlots = 4, kSlotBytes = 3 * kScaleBytes;
  static constexpr int kSmem = kStages * kStageBytes + kScaleSlots * kSlotBytes + 1024 + 512 + 2 * 4 * (MCEMU_FP8_MAX_GROUPS + 1);
};

struct PairUnit {
  int g, a, end, b, k0, k1;  // group, first row of a and where a's rows end, first row of b, blocks along k
};
struct PairGroups {
  const int *at, *before;
  int tiles_a, tiles_b, blocks;      // tiles of a (by_k), of b; blocks along k (not by_k)
};
__device__ __forceinline__ int units_of(const Fp8Product &p, const PairGroups &w) {
  return (p.by_k ? p.E * w.tiles_a : w.before[p.E]) * w.tiles_b;
}
// The u-th unit; g is the group of an earlier one.  Bands of eight tiles of a, so that the pairs at work
// share both operands in L2.
__device__ __forceinline__ PairUnit unit_at(const Fp8Product &p, const PairGroups &w, int bn, int u, int &g) {
  PairUnit r;
  int t, tiles_a = w.tiles_a;
  if (p.by_k) {
    const int each = tiles_a * w.tiles_b;
    g = u / each;
    t = u - g * each;
  } else {
    while (u >= w.before[g + 1] * w.tiles_b) g++;
    t = u - w.before[g] * w.tiles_b;
    tiles_a = w.before[g + 1] - w.before[g];
  }
  const int band = t / (8 * w.tiles_b), rest = t - band * 8 * w.tiles_b, width = min(8, tiles_a - band * 8);
  r.g = g;
  r.a = (p.by_k ? 0 : w.at[g]) + (band * 8 + rest % width) * 256;
  r.end = p.by_k ? p.a.rows : w.at[g + 1];
  r.b = rest / width * bn;
  r.k0 = p.by_k ? w.at[g] : 0;
  r.k1 = p.by_k ? w.at[g + 1] : w.blocks;
  return r;
}

template <class T, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    pair_kernel(const __grid_constant__ Fp8Product p, const __grid_constant__ CUtensorMap ma,
                const __grid_constant__ CUtensorMap mb) {
  using S = Pair<BN>;
  constexpr int kStages = S::kStages, kStageBytes = S::kStageBytes, kSlots = S::kScaleSlots, kCols = BN / 2;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (tc::smem_addr(raw) + 1023) & ~1023u;
  const uint32_t scales = base + kStages * kStageBytes, full = scales + kSlots * S::kSlotBytes, empty = full + 8 * kStages,
                 sf_full = empty + 8 * kStages, sf_empty = sf_full + 8 * kSlots, acc_full = sf_empty + 8 * kSlots,
                 acc_empty = acc_full + 16, drain = acc_empty + 16, slot = drain + 8;
  int *at = (int *)(raw + (slot + 16 - tc::smem_addr(raw))), *before = at + MCEMU_FP8_MAX_GROUPS + 1;
  const int warp = tc::warp_number(), lane = threadIdx.x & 31;
  const uint32_t rank = tc::cta_rank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; s++) {
      tc::mbar_init(full + 8 * s, 1);
      tc::mbar_init(empty + 8 * s, 1);
    }
    for (int s = 0; s < kSlots; s++) {
      tc::mbar_init(sf_full + 8 * s, 4);      // two warps of each CTA, on CTA 0's
      tc::mbar_init(sf_empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; s++) {
      tc::mbar_init(acc_full + 8 * s, 1);
      tc::mbar_init(acc_empty + 8 * s, 16);
    }
    tc::mbar_init(drain, 1);
    tc::mbar_init_fence();
  }
  if (warp == 8) tc::tmem_alloc<2>(slot, 512);
  grid_go();
  grid_wait();                                // operands and offsets may be the work of the kernel before
  if (warp == 0) place_groups(p, 256, at, before);
  tc::fence_before();
  tc::cluster_sync();
  tc::fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(slot));
  tmem = __shfl_sync(0xFFFFFFFFu, tmem, 0);
  bool dead = false;
  const PairGroups w{at, before, (p.a.rows + 255) / 256, (p.b.rows + BN - 1) / BN, (p.K + kBlock - 1) / kBlock};
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1, units = units_of(p, w);
  int g = 0;

  if (warp >= 8) tc::give_registers();
  if (warp == 8 && lane == 0) {               // copies this CTA's half of both operands
    uint32_t it = 0;
    for (int u = first; u < units && !dead; u += step) {
      const PairUnit r = unit_at(p, w, BN, u, g);
      const int y = r.a + (int)rank * 128, yb = r.b + (int)rank * (BN / 2), z = p.by_k ? 0 : r.g;
      for (int k = r.k0; k < r.k1; k++, it++) {
        const uint32_t s = it % kStages, to = base + s * kStageBytes;
        tc::mbar_wait(empty + 8 * s, ((it / kStages) & 1) ^ 1, dead);
        if (dead) break;
        if (rank == 0) tc::mbar_expect(full + 8 * s, 2 * kStageBytes);
        box_load_pair(to, &ma, k * kBlock, y, 0, full + 8 * s);
        box_load_pair(to + kTileBytes, &mb, k * kBlock, yb, z, full + 8 * s);
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
    const uint32_t ins = instruction(256, BN, p.a.fmt, p.b.fmt);
    uint32_t s = 0, phase = 0, ch = 0;
    for (int u = first; u < units && !dead; u += step) {
      const PairUnit r = unit_at(p, w, BN, u, g);
      for (int k = r.k0; k < r.k1 && !dead; k += kChunk, ch++) {
        const uint32_t set = ch & 1, d = tmem + set * 256, sa = d + BN, sb = sa + 4, sf = ch % kSlots;
        const uint32_t from = scales + sf * S::kSlotBytes;
        tc::mbar_wait_warp(acc_empty + 8 * set, ((ch >> 1) & 1) ^ 1, dead);
        mbar_wait_warp_cluster(sf_full + 8 * sf, (ch / kSlots) & 1, dead);
        if (dead) break;
        tc::fence_after();
        // Into the columns that the chunk before the last used: its accumulators have been drained.
        copy_scales<2>(sa, from);
        copy_scales<2>(sb, from + kScaleBytes);
        if (BN > 128) copy_scales<2>(sb + 4, from + 2 * kScaleBytes);
        tc::commit<2>(sf_empty + 8 * sf);
        const int n = min(kChunk, r.k1 - k);
        uint32_t word = ins;
        for (int i = 0; i < n; i++, word += kNextByte) {
          tc::mbar_wait_warp(full + 8 * s, phase, dead);
          if (dead) break;
          tc::fence_after();
          const uint32_t ta = base + s * kStageBytes;
          const uint64_t da = tc::operand(ta, 16, 1024), db = tc::operand(ta + kTileBytes, 16, 1024);
#pragma unroll
          for (int x = 0; x < 4; x++) mma<2>(d, da + 2 * x, db + 2 * x, word, sa, sb, (i | x) != 0);
          tc::commit<2>(empty + 8 * s);
          if (++s == kStages) s = 0, phase ^= 1;
        }
        tc::commit<2>(acc_full + 8 * set);
      }
    }
    bool late = false;                        // everything issued ends before the memory is given back
    tc::commit_here<2>(drain);
    tc::mbar_wait_warp(drain, 0, late);
  } else if (warp >= 10) {                    // exponents of this CTA's rows of a, or of b's
    uint32_t ch = 0;
    for (int u = first; u < units && !dead; u += step) {
      const PairUnit r = unit_at(p, w, BN, u, g);
      const int z = p.by_k ? 0 : r.g;
      for (int k = r.k0; k < r.k1 && !dead; k += kChunk, ch++) {
        const uint32_t sf = ch % kSlots, to = scales + sf * S::kSlotBytes;
        uint32_t v[2][4];
        if (warp == 10) {
          load_scales(p.a, 0, r.a + (int)rank * 128, k, r.k1, v[0]);
        } else {
          load_scales(p.b, z, r.b, k, r.k1, v[0]);
          if (BN > 128) load_scales(p.b, z, r.b + 128, k, r.k1, v[1]);
        }
        tc::mbar_wait_warp(sf_empty + 8 * sf, ((ch / kSlots) & 1) ^ 1, dead);
        if (dead) break;
        store_scales(to + (warp == 10 ? 0 : kScaleBytes), v[0]);
        if (BN > 128 && warp == 11) store_scales(to + 2 * kScaleBytes, v[1]);
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(sf_full + 8 * sf, 0);
      }
    }
  } else if (warp < 8) {
    tc::take_registers();
    const uint32_t mine = tmem + ((uint32_t)(warp & 3) << 21) + (warp >> 2) * kCols;
    uint32_t ch = 0;
    for (int u = first; u < units; u += step) {
      const PairUnit r = unit_at(p, w, BN, u, g);
      float sum[kCols];
#pragma unroll
      for (int j = 0; j < kCols; j++) sum[j] = 0.f;
      for (int k = r.k0; k < r.k1; k += kChunk, ch++) {
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
          for (int x = 0; x < 16; x++) sum[j + x] += v[(j >> 4) & 1][x];
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_lead(acc_empty + 8 * set);
      }
      // the matrix unit has both sets to go on with meanwhile
      const int row = r.a + (int)rank * 128 + (warp & 3) * 32 + lane, col = r.b + (warp >> 2) * kCols;
      T *y = (T *)p.y + (p.by_k ? r.g * p.stride_y : 0) + (int64_t)row * p.ldy + col;
      if (p.bias) {
#pragma unroll
        for (int j = 0; j < kCols; j++) sum[j] += col + j < p.b.rows ? __ldg(p.bias + col + j) : 0.f;
      }
      if (row < r.end && !dead) {
#pragma unroll
        for (int j = 0; j < kCols; j += 16) put16(y + j, &sum[j], p.b.rows - col - j, p.accumulate);
      }
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

template <class T, int BN>
int launch_pair(const Fp8Product &p, const CUtensorMap &ma, const CUtensorMap &mb, int64_t units, cudaStream_t st) {
  if (!allow_smem<pair_kernel<T, BN>>(Pair<BN>::kSmem)) return MCEMU_ERR_CUDA;
  const int pairs = units < sm_count() / 2 ? (int)units : sm_count() / 2;
  return launch_early(pair_kernel<T, BN>, dim3(2 * pairs), dim3(kPairThreads), Pair<BN>::kSmem, st, p, ma, mb);
}

}  // namespace fp8
}  // namespace mcemu
