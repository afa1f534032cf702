// rmsnorm_grad_single.cu -- gradients of the root-mean-square norm for rows that no vector fits
// (include/mcemu_ops.h has the formulas).
#include "norm_grad.cuh"
#include "norm_rows.cuh"

namespace mcemu {
namespace {

constexpr int kPer = 8;                        // elements a thread

// Rows that no vector fits, at any strides: a group of TX threads to a block, one element of every
// TX to a thread, so that a thread keeps its columns, their weights and its part of dw.  The
// next row is copied to shared memory meanwhile, whole units at a time; columns beyond a row are
// zeros there and need no questions until they are stored.  8191 x 4099 with a residual path: bf16 87
// us, fp32 88 (elements loaded one by one from memory 121, 134); between instruction issue (59 %) and
// latency.
template <class T, int TX, bool CKPT>
struct Single {
  using Dy = Rows<TX, kPer, sizeof(T)>;
  using In = Rows<TX, kPer, CKPT ? 1 : (int)sizeof(T)>;
  static constexpr int kStage = 2 * Dy::kPitch + In::kPitch;
};
template <class T, int TX, bool CKPT>
__global__ void __launch_bounds__(TX) single_kernel(const NormGradArgs a, float *__restrict__ parts) {
  using S = Single<T, TX, CKPT>;
  constexpr int kPitch = S::Dy::kPitch, kStage = S::kStage, kScales = kPer * TX / MCEMU_ACT8_BLOCK + 1;
  __shared__ float sums[2][32];
  __shared__ float scales[2][kScales];           // of this row's blocks of 128 and the next one's
  extern __shared__ __align__(16) uint8_t raw[];
  const int i0 = threadIdx.x, blocks = (a.H + MCEMU_ACT8_BLOCK - 1) / MCEMU_ACT8_BLOCK, left = a.H - i0;
  float2 w[kPer / 2], dw[kPer / 2];
  grid_go();
#pragma unroll
  for (int p = 0; p < kPer; p += 2) {
    float f[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 2; j++)
      if ((p + j) * TX < left) f[j] = a.w32 ? ((const float *)a.w)[i0 + (p + j) * TX] : to_f(((const T *)a.w)[i0 + (p + j) * TX]);
    w[p / 2] = make_float2(f[0], f[1]);
    dw[p / 2] = make_float2(0.f, 0.f);
  }
  for (int i = i0; i < 2 * kScales; i += TX) (&scales[0][0])[i] = 0.f;
  __syncthreads();
  typename S::Dy dys(a.dy, a.lddy, a.H), drs(a.dres, a.lddr, a.H);
  typename S::In ins(CKPT ? (const void *)a.q : a.h, CKPT ? a.ldq : a.ldh, a.H);
  const auto fetch = [&](uint8_t *to) {
    dys.fetch(to);
    if (a.dres) drs.fetch(to + kPitch);
    ins.fetch(to + 2 * kPitch);
  };
  int64_t row = blockIdx.x;
  float rstd_next = 0.f;
  if (row < a.T) {
    fetch(raw);
    rstd_next = a.rstd[row];
    if (CKPT && i0 < blocks) scales[0][i0] = act8_scale(a.e[row * a.lde + i0]);
  }
  copy_commit();
  for (int s = 0; row < a.T; row += gridDim.x, s ^= 1) {
    const int64_t next = row + gridDim.x;
    const uint8_t *cur = raw + s * kStage;
    const T *dy = (const T *)(cur + dys.off) + i0, *dr = (const T *)(cur + kPitch + drs.off) + i0;
    const uint8_t *in = cur + 2 * kPitch + ins.off + i0 * (CKPT ? 1 : (int)sizeof(T));
    const float rstd = rstd_next;
    int e_next = 0;
    copy_wait<0>();
    __syncthreads();                             // this row is there, and the one before is done with
    if (next < a.T) {
      fetch(raw + (s ^ 1) * kStage);
      rstd_next = a.rstd[next];
      if (CKPT && i0 < blocks) e_next = a.e[next * a.lde + i0];
    }
    copy_commit();
    const auto input = [&](int p) {
      if constexpr (!CKPT) return to_f(((const T *)in)[p * TX]);
      else if constexpr (TX % MCEMU_ACT8_BLOCK == 0)
        return (float)((const int8_t *)in)[p * TX] * scales[s][i0 / MCEMU_ACT8_BLOCK + p * (TX / MCEMU_ACT8_BLOCK)];
      else return (float)((const int8_t *)in)[p * TX] * scales[s][(i0 + p * TX) / MCEMU_ACT8_BLOCK];
    };
    const float2 r2 = make_float2(rstd, rstd);
    float2 z[kPer / 2], dot2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int p = 0; p < kPer; p += 2) {
      const float2 d = make_float2(to_f(dy[p * TX]), to_f(dy[(p + 1) * TX]));
      z[p / 2] = mul2(make_float2(input(p), input(p + 1)), r2);
      dot2 = fma2(mul2(d, w[p / 2]), z[p / 2], dot2);
      dw[p / 2] = fma2(d, z[p / 2], dw[p / 2]);
    }
    float dot = warp_sum(dot2.x + dot2.y);
    if constexpr (TX > 32) {
      const int lane = threadIdx.x & 31;
      if (lane == 0) sums[s][threadIdx.x >> 5] = dot;
      __syncthreads();
      dot = warp_sum(lane < TX / 32 ? sums[s][lane] : 0.f);
    }
    const float k = -(dot / (float)a.H) * rstd;
    const float2 k2 = make_float2(k, k);
    T *pdx = (T *)a.dx + row * a.lddx + i0;
#pragma unroll
    for (int p = 0; p < kPer; p += 2) {
      const float2 d = make_float2(to_f(dy[p * TX]), to_f(dy[(p + 1) * TX]));
      float2 g = mul2(d, w[p / 2]);
      if (a.dres) g = fma2(g, r2, make_float2(to_f(dr[p * TX]), to_f(dr[(p + 1) * TX])));
      else g = mul2(g, r2);
      g = fma2(z[p / 2], k2, g);
      if (p * TX < left) pdx[p * TX] = from_f<T>(g.x);
      if ((p + 1) * TX < left) pdx[(p + 1) * TX] = from_f<T>(g.y);
    }
    if (CKPT && i0 < blocks) scales[s ^ 1][i0] = act8_scale(e_next);
  }
  copy_wait<0>();
#pragma unroll
  for (int p = 0; p < kPer; p++)
    if (p * TX < left) parts[(int64_t)blockIdx.x * a.H + i0 + p * TX] = p & 1 ? dw[p / 2].y : dw[p / 2].x;
}

template <class T, int TX, bool CKPT>
bool go(const NormGradArgs &a, int blocks, float *parts, cudaStream_t st) {
  constexpr int kSmem = 2 * Single<T, TX, CKPT>::kStage;
  if (!allow_smem<single_kernel<T, TX, CKPT>>(kSmem)) return false;
  single_kernel<T, TX, CKPT><<<blocks, TX, kSmem, st>>>(a, parts);
  return true;
}

}  // namespace

// Threads to a row: several steps between powers of two, since columns beyond the row are computed
// too (16384 x 1025 bf16 by 256 threads 64 us, by 160 48).  Others than these were not measured; rows just
// above 512 and 1280 elements compute the most columns that they do not have (97 and 60 %).
template <class T, bool CKPT>
int launch_grad_single(const NormGradArgs &a, int blocks, float *parts, cudaStream_t st) {
  const int threads = (a.H + kPer - 1) / kPer;
  bool ok;
  if (threads <= 32) ok = go<T, 32, CKPT>(a, blocks, parts, st);
  else if (threads <= 64) ok = go<T, 64, CKPT>(a, blocks, parts, st);
  else if (threads <= 128) ok = go<T, 128, CKPT>(a, blocks, parts, st);
  else if (threads <= 160) ok = go<T, 160, CKPT>(a, blocks, parts, st);
  else if (threads <= 256) ok = go<T, 256, CKPT>(a, blocks, parts, st);
  else if (threads <= 320) ok = go<T, 320, CKPT>(a, blocks, parts, st);
  else if (threads <= 384) ok = go<T, 384, CKPT>(a, blocks, parts, st);
  else if (threads <= 512) ok = go<T, 512, CKPT>(a, blocks, parts, st);
  else if (threads <= 576) ok = go<T, 576, CKPT>(a, blocks, parts, st);
  else if (threads <= 640) ok = go<T, 640, CKPT>(a, blocks, parts, st);
  else if (threads <= 768) ok = go<T, 768, CKPT>(a, blocks, parts, st);
  else ok = go<T, 1024, CKPT>(a, blocks, parts, st);
  return ok ? blocks : -1;
}
template int launch_grad_single<float, true>(const NormGradArgs &, int, float *, cudaStream_t);
template int launch_grad_single<float, false>(const NormGradArgs &, int, float *, cudaStream_t);
template int launch_grad_single<__half, true>(const NormGradArgs &, int, float *, cudaStream_t);
template int launch_grad_single<__half, false>(const NormGradArgs &, int, float *, cudaStream_t);
template int launch_grad_single<__nv_bfloat16, true>(const NormGradArgs &, int, float *, cudaStream_t);
template int launch_grad_single<__nv_bfloat16, false>(const NormGradArgs &, int, float *, cudaStream_t);

}  // namespace mcemu
