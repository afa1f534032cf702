// act8_wgrad.cu -- a linear layer's weight gradient from the 8-bit checkpoint of its input
// (include/mcemu_ops.h has the formula).
#include "ops_common.cuh"

namespace mcemu {
namespace {

// 32 x 32 outputs to a block of 256 threads, four to a thread.
__global__ void __launch_bounds__(256) wgrad_kernel(const WgradArgs a) {
  __shared__ float ds[32][33], xs[32][33];
  const int n0 = blockIdx.y * 32, k0 = blockIdx.x * 32;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int t0 = 0; t0 < a.T; t0 += 32) {
#pragma unroll
    for (int r = 0; r < 4; r++) {
      const int i = ty + 8 * r, t = t0 + i, n = n0 + tx, k = k0 + tx;
      ds[i][tx] = t < a.T && n < a.N ? __uint_as_float((uint32_t)a.dy[(int64_t)t * a.lddy + n] << 16) : 0.f;
      xs[i][tx] = t < a.T && k < a.K ? (float)a.q[(int64_t)t * a.ldq + k] *
                                           act8_scale(a.e[(int64_t)t * a.lde + k / MCEMU_ACT8_BLOCK])
                                     : 0.f;
    }
    __syncthreads();
#pragma unroll 8
    for (int i = 0; i < 32; i++)
#pragma unroll
      for (int r = 0; r < 4; r++) acc[r] = fmaf(ds[i][ty + 8 * r], xs[i][tx], acc[r]);
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < 4; r++) {
    const int n = n0 + ty + 8 * r, k = k0 + tx;
    if (n >= a.N || k >= a.K) continue;
    const int64_t at = (int64_t)n * a.lddw + k;
    if (a.out_fmt == MCEMU_FP32) ((float *)a.dW)[at] = a.accumulate ? ((float *)a.dW)[at] + acc[r] : acc[r];
    else ((__nv_bfloat16 *)a.dW)[at] = __float2bfloat16_rn(acc[r]);
  }
}

}  // namespace

size_t act8_wgrad_workspace(int T, int N, int K) { return 0; }

int launch_act8_wgrad(const WgradArgs &a, void *ws, void *stream) {
  wgrad_kernel<<<dim3((a.K + 31) / 32, (a.N + 31) / 32), 256, 0, (cudaStream_t)stream>>>(a);
  return launch_status();
}

}  // namespace mcemu
