// int8_linear.cu -- product of 8-bit integers with a scale for each token and channel
// (include/mcemu_ops.h has the formula).
#include "ops_common.cuh"

namespace mcemu {
namespace {

__device__ __forceinline__ void put_y(const LinearArgs &a, int m, int n, int acc) {
  const int64_t at = (int64_t)m * a.ldy + n;
  if (a.out_fmt == MCEMU_INT32) {
    ((int32_t *)a.y)[at] = acc;
    return;
  }
  float v = __fmul_rn(__fmul_rn((float)acc, a.sx[m]), a.sw[n]);
  if (a.bias) v = __fadd_rn(v, a.bias[n]);
  if (a.out_fmt == MCEMU_FP32) ((float *)a.y)[at] = v;
  else if (a.out_fmt == MCEMU_FP16) ((__half *)a.y)[at] = __float2half_rn(v);
  else ((__nv_bfloat16 *)a.y)[at] = __float2bfloat16_rn(v);
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
    if (m < a.M && n < a.N) put_y(a, m, n, acc[r]);
  }
}

}  // namespace

size_t int8_linear_workspace(int M, int N, int K) { return 0; }

int launch_int8_linear(const LinearArgs &a, void *ws, void *stream) {
  linear_kernel<<<dim3((a.N + 31) / 32, (a.M + 31) / 32), 256, 0, (cudaStream_t)stream>>>(a);
  return launch_status();
}

}  // namespace mcemu
