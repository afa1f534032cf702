// rmsnorm_grad_single.cu -- gradients of the root-mean-square norm for rows that no vector fits
// (include/mcemu_ops.h has the formulas).
#include "norm_grad.cuh"

namespace mcemu {
namespace {

constexpr int kPer = 8;                        // elements a thread

// Rows that no vector fits, at any strides: a group of TX threads to a block, one element of every
// TX to a thread, so that a thread keeps its columns, their weights and its part of dw.
template <class T, int TX, bool CKPT>
__global__ void __launch_bounds__(TX) single_kernel(const NormGradArgs a, float *__restrict__ parts) {
  __shared__ float sh[32];
  __shared__ float scales[2][kPer * TX / MCEMU_ACT8_BLOCK + 1];      // of this row's blocks of 128 and the next one's
  const int i0 = threadIdx.x, blocks = (a.H + MCEMU_ACT8_BLOCK - 1) / MCEMU_ACT8_BLOCK;
  float w[kPer], dw[kPer];
  grid_go();
#pragma unroll
  for (int p = 0; p < kPer; p++) {
    const int i = i0 + p * TX;
    dw[p] = w[p] = 0.f;
    if (i < a.H) w[p] = a.w32 ? ((const float *)a.w)[i] : to_f(((const T *)a.w)[i]);
  }
  int64_t row = blockIdx.x;
  if (CKPT && row < a.T)
    for (int i = threadIdx.x; i < blocks; i += TX) scales[0][i] = act8_scale(a.e[row * a.lde + i]);
  __syncthreads();
  for (int s = 0; row < a.T; row += gridDim.x, s ^= 1) {
    const T *pdy = (const T *)a.dy + row * a.lddy + i0, *pdr = (const T *)a.dres + row * a.lddr + i0;
    const T *ph = (const T *)a.h + row * a.ldh + i0;
    const int8_t *pq = a.q + row * a.ldq + i0;
    T dy[kPer], dr[kPer];
    typename std::conditional<CKPT, int8_t, T>::type in[kPer];
#pragma unroll
    for (int p = 0; p < kPer; p++) {
      if (i0 + p * TX >= a.H) continue;
      dy[p] = pdy[p * TX];
      if constexpr (CKPT) in[p] = pq[p * TX];
      else in[p] = ph[p * TX];
      if (a.dres) dr[p] = pdr[p * TX];
    }
    const float rstd = a.rstd[row];
    if (CKPT && row + gridDim.x < a.T)
      for (int i = threadIdx.x; i < blocks; i += TX)
        scales[s ^ 1][i] = act8_scale(a.e[(row + gridDim.x) * a.lde + i]);
    float z[kPer], dot = 0.f;
#pragma unroll
    for (int p = 0; p < kPer; p++) {
      z[p] = 0.f;
      if (i0 + p * TX >= a.H) continue;
      if constexpr (CKPT) z[p] = (float)in[p] * scales[s][(i0 + p * TX) / MCEMU_ACT8_BLOCK] * rstd;
      else z[p] = to_f(in[p]) * rstd;
      const float d = to_f(dy[p]);
      dot = fmaf(d * w[p], z[p], dot);
      dw[p] = fmaf(d, z[p], dw[p]);
    }
    if (TX == 32) __syncwarp();
    const float k = -(row_sum<TX>(dot, sh) / (float)a.H) * rstd;
    T *pdx = (T *)a.dx + row * a.lddx + i0;
#pragma unroll
    for (int p = 0; p < kPer; p++) {
      if (i0 + p * TX >= a.H) continue;
      const float g = to_f(dy[p]) * w[p];
      pdx[p * TX] = from_f<T>(fmaf(z[p], k, a.dres ? fmaf(g, rstd, to_f(dr[p])) : g * rstd));
    }
  }
#pragma unroll
  for (int p = 0; p < kPer; p++)
    if (i0 + p * TX < a.H) parts[(int64_t)blockIdx.x * a.H + i0 + p * TX] = dw[p];
}

template <class T, int TX, bool CKPT>
void go(const NormGradArgs &a, int blocks, float *parts, cudaStream_t st) {
  single_kernel<T, TX, CKPT><<<blocks, TX, 0, st>>>(a, parts);
}

}  // namespace

// Threads to a row: several steps between powers of two, since elements beyond the row are skipped
// one by one.
template <class T, bool CKPT>
void launch_grad_single(const NormGradArgs &a, int blocks, float *parts, cudaStream_t st) {
  const int threads = (a.H + kPer - 1) / kPer;
  if (threads <= 32) go<T, 32, CKPT>(a, blocks, parts, st);
  else if (threads <= 64) go<T, 64, CKPT>(a, blocks, parts, st);
  else if (threads <= 128) go<T, 128, CKPT>(a, blocks, parts, st);
  else if (threads <= 256) go<T, 256, CKPT>(a, blocks, parts, st);
  else if (threads <= 384) go<T, 384, CKPT>(a, blocks, parts, st);
  else if (threads <= 512) go<T, 512, CKPT>(a, blocks, parts, st);
  else if (threads <= 640) go<T, 640, CKPT>(a, blocks, parts, st);
  else if (threads <= 768) go<T, 768, CKPT>(a, blocks, parts, st);
  else go<T, 1024, CKPT>(a, blocks, parts, st);
}
template void launch_grad_single<float, true>(const NormGradArgs &, int, float *, cudaStream_t);
template void launch_grad_single<float, false>(const NormGradArgs &, int, float *, cudaStream_t);
template void launch_grad_single<__half, true>(const NormGradArgs &, int, float *, cudaStream_t);
template void launch_grad_single<__half, false>(const NormGradArgs &, int, float *, cudaStream_t);
template void launch_grad_single<__nv_bfloat16, true>(const NormGradArgs &, int, float *, cudaStream_t);
template void launch_grad_single<__nv_bfloat16, false>(const NormGradArgs &, int, float *, cudaStream_t);

}  // namespace mcemu
