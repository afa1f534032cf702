// fp8_few.cuh -- FP8 products of few rows of a (tokens) by many of b (channels).
//
// The roles change: 128 channels are the matrix instruction's rows and BT tokens its columns, so that the
// weights stream through once at whatever rate memory gives.  The CTAs of a cluster share K; each has
// its own copies in flight (a ring of stages in shared memory), and sends its sums of each token into the shared
// memory of the CTA that adds up that token's parts, in the order of the parts.  (By the copy engine, a token's
// 128 sums in 512 bytes: threads that stored into the other CTAs took 330 cycles a store, 6600 for 77 tokens.)
// Clusters walk over the units of work, the next one's copies on their way while a unit is joined; with more
// than 32 tokens a cluster that shares K has one unit, whose sums leave through the stages' memory.
//
// Bound by HBM where there are weights enough: 128 rows through 32 experts of 2048 x 4096 take 43.7 us (6.1 TB/s, 0.89 of
// the measured rate).  One token by 4096 x 4096 takes 5.0 us, 2.5 of them for the bytes: setting up (barriers,
// tensor memory, a cluster's meeting), one memory latency, the join and the parting take 2000 cycles each or less.
#pragma once
#include "fp8_tc.cuh"

namespace mcemu {
namespace fp8 {

// Four warps drain; then come one for the copies of b, one that issues matrix instructions, one for the exponents
// of b, one for a's, one for the copies of a.
constexpr int kFewThreads = 288;
// CTAs that share K at most: eight, the portable limit of a cluster.
constexpr int kMostParts = 8;

template <int BT>
struct Few {
  static constexpr int kStageBytes = kTileBytes + BT * kBlock;
  static constexpr int kStages = BT <= 16 ? 9 : BT <= 32 ? 8 : BT <= 64 ? 6 : 4;
  static constexpr int kScaleSlots = 4, kSlotBytes = 2 * kScaleBytes;
  static constexpr int kSendBytes = BT <= 32 ? BT * 512 : 0;   // sums on their way out; with more tokens: the stages
  static constexpr int kJoinBytes = (BT + kMostParts - 1 + 3) * 512;    // three places to read over
  static constexpr int kSmem = kStages * kStageBytes + kScaleSlots * kSlotBytes + kSendBytes + kJoinBytes + 1024 + 512 +
                               2 * 4 * (MCEMU_FP8_MAX_GROUPS + 1);
  static_assert(kSmem <= 232448, "shared memory");
};

struct FewUnit {
  int g, a, n, b;            // group, first token, how many, first channel
};
__device__ __forceinline__ FewUnit few_unit_at(const int *at, const int *before, int tiles_b, int bt, int u, int &g) {
  while (u >= before[g + 1] * tiles_b) g++;
  const int t = u - before[g] * tiles_b, tiles_a = before[g + 1] - before[g], a = at[g] + t % tiles_a * bt;
  return FewUnit{g, a, min(bt, at[g + 1] - a), t / tiles_a * 128};      // one tile of channels for all tokens, then the next
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
    few_kernel(const Fp8Product p, const __grid_constant__ CUtensorMap ma,
               const __grid_constant__ CUtensorMap mb, int per) {
  using S = Few<BT>;
  constexpr int kStages = S::kStages, kStageBytes = S::kStageBytes, kSlots = S::kScaleSlots;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (tc::smem_addr(raw) + 1023) & ~1023u;
  const uint32_t scales = base + kStages * kStageBytes, send = S::kSendBytes ? scales + kSlots * S::kSlotBytes : base,
                 join = scales + kSlots * S::kSlotBytes + S::kSendBytes, full = join + S::kJoinBytes,
                 empty = full + 8 * kStages, sf_full = empty + 8 * kStages, sf_empty = sf_full + 8 * kSlots,
                 acc_full = sf_empty + 8 * kSlots, acc_empty = acc_full + 16, drain = acc_empty + 16, join_full = drain + 8,
                 join_empty = join_full + 8, slot = join_empty + 8;
  int *at = (int *)(raw + (slot + 16 - tc::smem_addr(raw))), *before = at + MCEMU_FP8_MAX_GROUPS + 1;
  const int warp = tc::warp_number(), lane = threadIdx.x & 31;
  const uint32_t parts = tc::cluster_size(), rank = tc::cta_rank();

  if (threadIdx.x == 128) prefetch_map(&mb);
  if (threadIdx.x == 256) prefetch_map(&ma);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; s++) {
      tc::mbar_init(full + 8 * s, 2);         // both copying warps
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

  if (warp == 4 || warp == 8) {               // copies b's part, or a's
    const bool of_b = warp == 4;
    const CUtensorMap *map = of_b ? &mb : &ma;
    uint32_t s = 0, phase = 1, it = 0;
    for (int u = first; u < units && !dead; u += step) {
      const FewUnit r = few_unit_at(at, before, tiles_b, BT, u, g);
      for (int k = k0; k < k1; k++, it++) {
        if (it >= kStages) tc::mbar_wait_warp(empty + 8 * s, phase, dead);
        if (dead) break;
        if (lane == 0) tc::mbar_expect(full + 8 * s, of_b ? kTileBytes : BT * kBlock);
        __syncwarp();
        box_load(base + s * kStageBytes + (of_b ? 0 : kTileBytes), map, k * kBlock, of_b ? r.b : r.a, of_b ? r.g : 0, full + 8 * s);
        if (++s == kStages) s = 0, phase ^= 1;
      }
    }
    bool late = false;                        // the copies end before the CTA leaves
    for (uint32_t q = 0; q < kStages && q < it; q++) {
      const uint32_t last = it - 1 - (it - 1 - q) % kStages;
      tc::mbar_wait_warp(full + 8 * q, (last / kStages) & 1, late);
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
        tc::mbar_wait_warp(acc_full + 8 * set, (ch >> 1) & 1, dead);       // a whole warp's verdict: what follows is one's
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
      // tokens share * o to share * (o + 1) - 1 are joined by CTA o, where part q's lie in places q * share and on;
      // a place has a token's 128 sums
      const int share = (r.n + (int)parts - 1) / (int)parts, mine_n = max(0, min(share, r.n - (int)rank * share));
      // Every CTA has taken what was sent last before anything is written over it (a push tells its arrival alone, to
      // the CTA that it goes to), and before the barrier is told of the next: one that joins nothing would
      // otherwise end two phases while a warp still waits for the first, and look as if it had ended none.
      if (warp == 0) {
        mbar_wait_warp_cluster(join_empty, (turn & 1) ^ 1, dead);
        if (lane == 0) tc::mbar_expect(join_full, mine_n * parts * 512);
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
      for (int j = 0; j < BT; j++)
        if (j < r.n) asm volatile("st.shared.f32 [%0], %1;" ::"r"(send + j * 512 + row * 4), "f"(sum[j]) : "memory");
      tc::fence_async_smem();
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (warp == 0) {
        const int o = lane, n_o = min(share, r.n - o * share);
        if (o < (int)parts && n_o > 0 && !dead)
          bulk_push(at_rank(join + rank * share * 512, o), send + o * share * 512, n_o * 512, at_rank(join_full, o));
        __syncwarp();
      }
      tc::mbar_wait_warp(join_full, turn & 1, dead);
      if (!dead) (void)mbar_try_cluster(join_full, turn & 1);
      y += (int64_t)rank * share * p.ldy;
      const float *from = (const float *)(raw + (join - tc::smem_addr(raw))) + row;
#pragma unroll 1
      for (int i = 0; i < mine_n; i += 4) {
        float total[4] = {0.f, 0.f, 0.f, 0.f};
        const float *at_q = from + i * 128;   // places behind the last are read and not used
#pragma unroll 1
        for (int q = 0; q < (int)parts; q++, at_q += share * 128) {
#pragma unroll
          for (int x = 0; x < 4; x++) total[x] += at_q[x * 128];
        }
        const int n = in && !dead ? min(4, mine_n - i) : 0;
#pragma unroll
        for (int x = 0; x < 4; x++, y += p.ldy)
          if (x < n) put(y, total[x] + bias, p.accumulate);
      }
      __syncwarp();
      if (lane < (int)parts) mbar_arrive_at(join_empty, lane);
    }
  }
  __syncwarp();
  tc::fence_before();
  tc::cluster_sync();                         // no CTA leaves before all have what was pushed
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
  if (BT > 32 && parts > 1 && units * parts > sm_count()) parts = 1, per = (p.K + kBlock - 1) / kBlock;      // one unit to a cluster
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
