// fp8_few.cuh -- FP8 products of few rows of a (tokens) by many of b (channels).
//
// The roles change: 128 channels are the matrix instruction's rows and BT tokens its columns, so that the
// weights stream through once at whatever rate memory gives.  The CTAs of a cluster share K; each has
// its own copies in flight (a ring of stages in shared memory), and pushes its sums of each token into the shared
// memory of the CTA that adds up that token's parts, in the order of the parts.  Clusters walk over the
// units of work, the next one's copies on their way while a unit is joined.
#pragma once
#include "fp8_tc.cuh"

namespace mcemu {
namespace fp8 {

constexpr int kFewThreads = 256;              // four warps drain, then: copies, matrix instructions, exponents of b, of a
template <int BT>
struct Few {
  static constexpr int kStageBytes = kTileBytes + BT * kBlock;
  static constexpr int kStages = BT <= 16 ? 10 : BT <= 32 ? 8 : BT <= 64 ? 6 : 4;
  static constexpr int kScaleSlots = 4, kSlotBytes = 2 * kScaleBytes;
  static constexpr int kJoinBytes = (BT + 8) * 512;
  static constexpr int kSmem = kStages * kStageBytes + kScaleSlots * kSlotBytes + kJoinBytes + 1024 + 512 +
                               2 * 4 * (MCEMU_FP8_MAX_GROUPS + 1);
};

struct FewUnit {
  int g, a, n, b;            // group, first token, how many, first channel
};
__device__ __forceinline__ FewUnit few_unit_at(const int *at, const int *before, int tiles_b, int bt, int u, int &g) {
  while (u >= before[g + 1] * tiles_b) g++;
  const int t = u - before[g] * tiles_b, tiles_a = before[g + 1] - before[g], a = at[g] + t % tiles_a * bt;
  return FewUnit{g, a, min(bt, at[g + 1] - a), t / tiles_a * 128};      // one tile of channels for all tokens, then the next
}

// Four bytes to `to`, counted on the barrier `bar` there (addresses in the cluster, of the same CTA).
__device__ __forceinline__ void push(uint32_t to, float v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(to),
               "r"(__float_as_uint(v)), "r"(bar)
               : "memory");
}

// A warp's way through the units, bringing a chunk's exponents of R * 32 rows of a or b to each slot.
template <int R, int BT>
__device__ __forceinline__ void few_scales(const Fp8Product &p, const int *at, const int *before, int tiles_b, int first, int step,
                                           int units, int k0, int k1, bool of_a, uint32_t scales, uint32_t sf_full,
                                           uint32_t sf_empty, bool &dead) {
  using S = Few<BT>;
  Scales<R> v;
  uint32_t ch = 0;
  int g = 0;
  for (int u = first; u < units && !dead; u += step) {
    const FewUnit r = few_unit_at(at, before, tiles_b, BT, u, g);
    if (of_a) v.rows(p.a, 0, r.a);
    else v.rows(p.b, r.g, r.b);
    for (int k = k0; k < k1; k += kChunk, ch++) {
      const uint32_t sf = ch % S::kScaleSlots;
      uint32_t x[1][4];
      v.load(0, k, k1, x);
      tc::mbar_wait_warp(sf_empty + 8 * sf, ((ch / S::kScaleSlots) & 1) ^ 1, dead);
      if (dead) return;
      store_scales(scales + sf * S::kSlotBytes, x[0]);
      tc::fence_async_smem();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) tc::mbar_arrive(sf_full + 8 * sf);
    }
  }
}

template <class T, int BT>
__global__ void __launch_bounds__(kFewThreads, 1)
    few_kernel(const __grid_constant__ Fp8Product p, const __grid_constant__ CUtensorMap ma,
               const __grid_constant__ CUtensorMap mb, int per) {
  using S = Few<BT>;
  constexpr int kStages = S::kStages, kStageBytes = S::kStageBytes, kSlots = S::kScaleSlots;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (tc::smem_addr(raw) + 1023) & ~1023u;
  const uint32_t scales = base + kStages * kStageBytes, join = scales + kSlots * S::kSlotBytes, full = join + S::kJoinBytes,
                 empty = full + 8 * kStages, sf_full = empty + 8 * kStages, sf_empty = sf_full + 8 * kSlots,
                 acc_full = sf_empty + 8 * kSlots, acc_empty = acc_full + 16, drain = acc_empty + 16, join_full = drain + 8,
                 join_empty = join_full + 8, slot = join_empty + 8;
  int *at = (int *)(raw + (slot + 16 - tc::smem_addr(raw))), *before = at + MCEMU_FP8_MAX_GROUPS + 1;
  const int warp = tc::warp_number(), lane = threadIdx.x & 31;
  const uint32_t parts = tc::cluster_size(), rank = tc::cta_rank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; s++) {
      tc::mbar_init(full + 8 * s, 1);
      tc::mbar_init(empty + 8 * s, 1);
    }
    for (int s = 0; s < kSlots; s++) {
      tc::mbar_init(sf_full + 8 * s, 2);
      tc::mbar_init(sf_empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; s++) {
      tc::mbar_init(acc_full + 8 * s, 1);
      tc::mbar_init(acc_empty + 8 * s, 4);
    }
    tc::mbar_init(drain, 1);
    tc::mbar_init(join_full, 1);
    tc::mbar_init(join_empty, 4 * parts);
    tc::mbar_init_fence();
  }
  if (warp == 5) tc::tmem_alloc<1>(slot, 512);
  grid_go();
  grid_wait();                                // operands and offsets may be the work of the kernel before
  if (warp == 0) place_groups(p, BT, at, before);
  tc::fence_before();
  tc::cluster_sync();
  tc::fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(slot));
  tmem = __shfl_sync(0xFFFFFFFFu, tmem, 0);
  bool dead = false;
  const int tiles_b = (p.b.rows + 127) / 128, blocks = (p.K + kBlock - 1) / kBlock;
  const int first = blockIdx.x / parts, step = gridDim.x / parts, units = before[p.E] * tiles_b;
  const int k0 = (int)rank * per, k1 = min(blocks, k0 + per);
  int g = 0;

  if (warp == 4) {
    if (lane == 0) {                          // copies both operands' parts
      uint32_t it = 0;
      for (int u = first; u < units && !dead; u += step) {
        const FewUnit r = few_unit_at(at, before, tiles_b, BT, u, g);
        for (int k = k0; k < k1; k++, it++) {
          const uint32_t s = it % kStages, to = base + s * kStageBytes;
          tc::mbar_wait(empty + 8 * s, ((it / kStages) & 1) ^ 1, dead);
          if (dead) break;
          tc::mbar_expect(full + 8 * s, kStageBytes);
          box_load(to, &mb, k * kBlock, r.b, r.g, full + 8 * s);
          box_load(to + kTileBytes, &ma, k * kBlock, r.a, 0, full + 8 * s);
        }
      }
      bool late = false;                      // the copies end before the CTA leaves
      for (uint32_t s = 0; s < kStages && s < it; s++) {
        const uint32_t last = it - 1 - (it - 1 - s) % kStages;
        tc::mbar_wait(full + 8 * s, (last / kStages) & 1, late);
      }
    }
  } else if (warp == 5) {                     // issues the matrix instructions
    const uint32_t ins = instruction(128, BT, p.b.fmt, p.a.fmt);
    uint32_t s = 0, phase = 0, ch = 0;
    for (int u = first; u < units && !dead; u += step) {
      for (int k = k0; k < k1 && !dead; k += kChunk, ch++) {
        const uint32_t set = ch & 1, d = tmem + set * 256, sb = d + 128, sa = sb + 4, sf = ch % kSlots;
        const uint32_t from = scales + sf * S::kSlotBytes;
        tc::mbar_wait_warp(acc_empty + 8 * set, ((ch >> 1) & 1) ^ 1, dead);
        tc::mbar_wait_warp(sf_full + 8 * sf, (ch / kSlots) & 1, dead);
        if (dead) break;
        tc::fence_after();
        // into the columns that the chunk before the last used: its accumulators have been drained
        copy_scales<1>(sb, from);
        copy_scales<1>(sa, from + kScaleBytes);
        tc::commit<1>(sf_empty + 8 * sf);
        const int n = min(kChunk, k1 - k);
        uint32_t word = ins;
        for (int i = 0; i < n; i++, word += kNextByte) {
          tc::mbar_wait_warp(full + 8 * s, phase, dead);
          if (dead) break;
          tc::fence_after();
          const uint32_t tb = base + s * kStageBytes;
          const uint64_t db = tc::operand(tb, 16, 1024), da = tc::operand(tb + kTileBytes, 16, 1024);
#pragma unroll
          for (int x = 0; x < 4; x++) mma<1>(d, db + 2 * x, da + 2 * x, word, sb, sa, (i | x) != 0);
          tc::commit<1>(empty + 8 * s);
          if (++s == kStages) s = 0, phase ^= 1;
        }
        tc::commit<1>(acc_full + 8 * set);
      }
    }
    bool late = false;                        // everything issued ends before the memory is given back
    tc::commit<1>(drain);
    tc::mbar_wait_warp(drain, 0, late);
  } else if (warp == 6) {                     // exponents of b's rows
    few_scales<4, BT>(p, at, before, tiles_b, first, step, units, k0, k1, false, scales, sf_full, sf_empty, dead);
  } else if (warp == 7) {                     // of a's
    few_scales<(BT + 31) / 32, BT>(p, at, before, tiles_b, first, step, units, k0, k1, true, scales + kScaleBytes, sf_full, sf_empty, dead);
  } else {
    const uint32_t mine = tmem + ((uint32_t)warp << 21);
    const int row = warp * 32 + lane;
    uint32_t ch = 0, turn = 0;
    for (int u = first; u < units; u += step, turn++) {
      const FewUnit r = few_unit_at(at, before, tiles_b, BT, u, g);
      float sum[BT];
#pragma unroll
      for (int j = 0; j < BT; j++) sum[j] = 0.f;
      for (int k = k0; k < k1; k += kChunk, ch++) {
        const uint32_t set = ch & 1;
        tc::mbar_wait(acc_full + 8 * set, (ch >> 1) & 1, dead);
        __syncwarp();
        tc::fence_after();
        float v[2][16];
        tc::tmem_load16(mine + set * 256, v[0]);
#pragma unroll
        for (int j = 0; j < BT; j += 16) {
          tc::tmem_wait();
          if (j + 16 < BT) tc::tmem_load16(mine + set * 256 + j + 16, v[(j >> 4) + 1 & 1]);
#pragma unroll
          for (int x = 0; x < 16; x++) sum[j + x] += v[(j >> 4) & 1][x];
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(acc_empty + 8 * set);
      }
      const int n = r.b + row;
      T *y = (T *)p.y + (int64_t)r.a * p.ldy + n;
      const bool in = n < p.b.rows;
      const float bias = p.bias && in ? __ldg(p.bias + n) : 0.f;
      if (parts == 1) {
        if (in && !dead) {
#pragma unroll
          for (int j = 0; j < BT; j++)
            if (j < r.n) put(y + j * p.ldy, sum[j] + bias, p.accumulate);
        }
        continue;
      }
      // tokens share * o to share * (o + 1) - 1 are joined by CTA o: part q's sums of its token c lie in
      // slot q * share + c
      const int share = (r.n + (int)parts - 1) / (int)parts, mine_n = max(0, min(share, r.n - (int)rank * share));
      if (threadIdx.x == 0) tc::mbar_expect(join_full, mine_n * parts * 512);
      tc::mbar_wait(join_empty, (turn & 1) ^ 1, dead);           // what was pushed last has been taken
      const uint32_t place = join + (rank * share * 128 + row) * 4;
      uint32_t to = at_rank(place, 0), bar = at_rank(join_full, 0);
      int o = 0, c = 0;
#pragma unroll
      for (int j = 0; j < BT; j++) {
        if (j < r.n && !dead) {
          push(to + c * 512, sum[j], bar);
          if (++c == share && j + 1 < r.n) {
            c = 0, o++;
            to = at_rank(place, o), bar = at_rank(join_full, o);
          }
        }
      }
      tc::mbar_wait(join_full, turn & 1, dead);
      if (!dead) (void)mbar_try_cluster(join_full, turn & 1);
      for (int i = 0; i < mine_n && !dead; i++) {
        float total = 0.f;
        for (uint32_t q = 0; q < parts; q++) {
          float v;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(join + ((q * share + i) * 128 + row) * 4) : "memory");
          total += v;
        }
        if (in) put(y + (int64_t)(rank * share + i) * p.ldy, total + bias, p.accumulate);
      }
      __syncwarp();
      if (lane < (int)parts) mbar_arrive_at(join_empty, lane);
    }
  }
  __syncwarp();
  tc::fence_before();
  tc::cluster_sync();                         // no CTA leaves while another pushes into it
  if (warp == 5) {
    tc::fence_after();
    tc::tmem_free<1>(tmem, 512);
  }
}

template <class T, int BT>
int launch_few(const Fp8Product &p, const CUtensorMap &ma, const CUtensorMap &mb, int64_t units, int parts, int per,
               int64_t clusters, cudaStream_t st) {
  if (!allow_smem<few_kernel<T, BT>>(Few<BT>::kSmem)) return MCEMU_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  const int64_t fit = sm_count() / parts, most = clusters < fit ? clusters : fit > 0 ? fit : 1;
  cfg.gridDim = dim3((unsigned)((units < most ? units : most) * parts));
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = Few<BT>::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = parts;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, few_kernel<T, BT>, p, ma, mb, per) == cudaSuccess ? MCEMU_OK : MCEMU_ERR_CUDA;
}

}  // namespace fp8
}  // namespace mcemu
