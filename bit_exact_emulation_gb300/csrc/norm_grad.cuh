// norm_grad.cuh -- what the two files of the norm's gradients share: rmsnorm_grad.cu (rows in
// vectors, long rows, the join of dw) and rmsnorm_grad_single.cu (rows that no vector fits).
#pragma once
#include "ops_common.cuh"

namespace mcemu {

// Most blocks, each of which keeps a part of dw: one to a multiprocessor of a GB300's 152 (the
// workspace's size goes by them and is known without a device), more where a block is one group
// of threads for a short row.
inline int most_blocks(int T, int H) {
  const int per_sm = H <= 1024 ? 16 : H <= 16384 ? 16384 / H : 1, most = 152 * per_sm;
  return T < most ? T : most;
}

// Sum over the TX threads of a row (whole warps), which wait for one another alone.
template <int TX>
__device__ __forceinline__ float row_sum(float x, float *part) {
  x = warp_sum(x);
  if constexpr (TX > 32) {
    float *mine = part + threadIdx.y * (TX / 32);
    const int bar = threadIdx.y + 1;
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(TX) : "memory");
    if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = x;
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(TX) : "memory");
    x = 0.f;
#pragma unroll
    for (int i = 0; i < TX / 32; i++) x += mine[i];
  }
  return x;
}

// Rows of at most kMaxSingle elements at any strides, on `blocks` blocks that leave their parts of
// dw in `parts`.  Their number, -1 after an error.
constexpr int kMaxSingle = 8192;
template <class T, bool CKPT>
int launch_grad_single(const NormGradArgs &a, int blocks, float *parts, cudaStream_t st);

}  // namespace mcemu
