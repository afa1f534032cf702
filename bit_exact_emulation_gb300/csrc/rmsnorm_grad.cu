// rmsnorm_grad.cu -- gradients of the root-mean-square norm, from its input or from an 8-bit
// checkpoint of it (include/mcemu_ops.h has the formulas).
//
// Bound by HBM: 7 bytes an element for bf16 gradients with a checkpoint and a residual path.
// Each group of threads walks over rows with its columns' weights and its part of dw in
// registers; the parts are added in a fixed order by a second, small kernel.
#include "norm_grad.cuh"

namespace mcemu {
namespace {

constexpr int kThreads = 512;                  // of a block

// One element of the norm's input, from h or from the checkpoint.
template <class T, bool CKPT>
__device__ __forceinline__ float input_at(const NormGradArgs &a, int64_t row, int i) {
  if constexpr (CKPT)
    return (float)a.q[row * a.ldq + i] * act8_scale(a.e[row * a.lde + i / MCEMU_ACT8_BLOCK]);
  else
    return to_f(((const T *)a.h)[row * a.ldh + i]);
}

// Where column k of dw lies in shared memory: a word is left out after every eight, so that lanes
// eight (or four) columns apart meet different banks.
__device__ __forceinline__ int padded(int k) { return k + (k >> 3); }

// blockDim.y rows at a time to a block, TX threads to a row, PER vectors of it to a thread.  The
// groups of threads that hold a row each run on their own.  A thread copies its pieces of the next
// row into shared memory while it works on the present one, so that loads are in flight
// throughout without a register for them.  TX is known to the compiler, so that the vectors
// of a row lie at fixed distances; 32 elements a thread, where the row is long enough, keep what a
// row costs on top of its elements small.  8192 x 4096 bf16 with a residual path: 45.8 us (the
// joining kernel included); rows loaded to registers when their turn comes 71; 8 elements a
// thread and TX a variable 86.
template <class T, int VEC, int PER, bool CKPT>
struct Stage {                                  // of kThreads threads
  Vec<T, VEC> dy[PER][kThreads], dr[PER][kThreads];
  typename std::conditional<CKPT, Vec<int8_t, VEC>, Vec<T, VEC>>::type in[PER][kThreads];
};

template <class T, int VEC, int PER, int TX, bool CKPT>
__global__ void __launch_bounds__(kThreads, 1) grad_kernel(const NormGradArgs a, float *__restrict__ parts) {
  using S = Stage<T, VEC, PER, CKPT>;
  __shared__ float sh[kThreads / 32];
  extern __shared__ __align__(16) uint8_t raw[];
  S *stages = (S *)raw;
  const int t = threadIdx.y * TX + threadIdx.x;
  grid_go();
  float2 dw[PER][VEC / 2];
#pragma unroll
  for (int p = 0; p < PER; p++)
#pragma unroll
    for (int j = 0; j < VEC / 2; j++) dw[p][j] = make_float2(0.f, 0.f);
  Vec<T, VEC> wv[PER];                          // weights in T stay in registers, fp32 ones are read again
  const bool keep = !a.w32 || sizeof(T) == 4;
#pragma unroll
  for (int p = 0; p < PER; p++) {
    const int i = (p * TX + threadIdx.x) * VEC;
    if (keep && i < a.H) wv[p] = load_vec<T, VEC>((const T *)a.w + i);
  }
  const auto weights = [&](int p, int i, float (&w)[VEC]) {
    if (keep) unpack<T, VEC>(wv[p], w);
    else load_w<T, VEC>(a.w, 1, i, w);
  };
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;

  float rstd = 0.f, rstd_next = 0.f;
  float scale[PER], scale_next[PER];
  const auto fetch = [&](int64_t r, S &to) {
#pragma unroll
    for (int p = 0; p < PER; p++) {
      const int i = (p * TX + threadIdx.x) * VEC;
      if (i >= a.H) continue;
      copy_async<16>(&to.dy[p][t], (const T *)a.dy + r * a.lddy + i);
      if (a.dres) copy_async<16>(&to.dr[p][t], (const T *)a.dres + r * a.lddr + i);
      if constexpr (CKPT) {
        copy_async<VEC>(&to.in[p][t], a.q + r * a.ldq + i);
        scale_next[p] = act8_scale(a.e[r * a.lde + i / MCEMU_ACT8_BLOCK]);
      } else {
        copy_async<16>(&to.in[p][t], (const T *)a.h + r * a.ldh + i);
      }
    }
    rstd_next = a.rstd[r];
  };
  if (row < a.T) fetch(row, stages[0]);
  copy_commit();
  for (int s = 0; row < a.T; row += step, s ^= 1) {
    rstd = rstd_next;
#pragma unroll
    for (int p = 0; p < PER; p++) scale[p] = CKPT ? scale_next[p] * rstd : rstd;      // z = f * scale
    if (row + step < a.T) fetch(row + step, stages[s ^ 1]);
    copy_commit();
    copy_wait<1>();
    const S &cur = stages[s];
    const auto get = [&](int p, float (&f)[VEC]) {
      if constexpr (CKPT) bytes_to_f<VEC>(cur.in[p][t], f);
      else unpack<T, VEC>(cur.in[p][t], f);
    };
    float dot = 0.f;
#pragma unroll
    for (int p = 0; p < PER; p++) {
      const int i = (p * TX + threadIdx.x) * VEC;
      if (i >= a.H) continue;
      float f[VEC], w[VEC], d[VEC];
      float2 some = make_float2(0.f, 0.f);
      const float2 s2 = make_float2(scale[p], scale[p]);
      get(p, f);
      unpack<T, VEC>(cur.dy[p][t], d);
      weights(p, i, w);
#pragma unroll
      for (int j = 0; j < VEC; j += 2) {
        const float2 z = mul2(make_float2(f[j], f[j + 1]), s2), d2 = make_float2(d[j], d[j + 1]);
        some = fma2(mul2(d2, make_float2(w[j], w[j + 1])), z, some);
        dw[p][j / 2] = fma2(d2, z, dw[p][j / 2]);
      }
      dot += some.x + some.y;
    }
    const float mean = row_sum<TX>(dot, sh) / (float)a.H;
#pragma unroll
    for (int p = 0; p < PER; p++) {
      const int i = (p * TX + threadIdx.x) * VEC;
      if (i >= a.H) continue;
      float f[VEC], w[VEC], d[VEC];
      get(p, f);
      unpack<T, VEC>(cur.dy[p][t], d);
      weights(p, i, w);
      // rstd * (g - z * mean) + dres, the factors of f in z * mean gathered (with rstd's among them they
      // would hold its square, which leaves fp32 for rows beyond 10^19 or below 10^-19)
      const float k = -(scale[p] * mean);
      const float2 k2 = make_float2(k, k), r2 = make_float2(rstd, rstd);
      float2 g[VEC / 2];
#pragma unroll
      for (int j = 0; j < VEC; j += 2) {
        g[j / 2] = mul2(make_float2(d[j], d[j + 1]), make_float2(w[j], w[j + 1]));
        g[j / 2] = fma2(make_float2(f[j], f[j + 1]), k2, g[j / 2]);
      }
      if (a.dres) {
        unpack<T, VEC>(cur.dr[p][t], d);
#pragma unroll
        for (int j = 0; j < VEC; j += 2) g[j / 2] = fma2(g[j / 2], r2, make_float2(d[j], d[j + 1]));
      } else {
#pragma unroll
        for (int j = 0; j < VEC; j += 2) g[j / 2] = mul2(g[j / 2], r2);
      }
#pragma unroll
      for (int j = 0; j < VEC; j += 2) f[j] = g[j / 2].x, f[j + 1] = g[j / 2].y;
      store_vec((T *)a.dx + row * a.lddx + i, pack<T, VEC>(f));
    }
  }
  copy_wait<0>();
  // the groups' parts of dw, side by side in the copies' memory, added in order
  float *mine = parts + (int64_t)blockIdx.x * a.H;
  const int pitch = padded(a.H) + 1;
  float *join = (float *)raw + threadIdx.y * pitch;
  if (blockDim.y > 1) __syncthreads();
#pragma unroll
  for (int p = 0; p < PER; p++) {
    const int i = (p * TX + threadIdx.x) * VEC;
    if (i >= a.H) continue;
#pragma unroll
    for (int j = 0; j < VEC; j++) {
      const float v = j & 1 ? dw[p][j / 2].y : dw[p][j / 2].x;
      if (blockDim.y > 1) join[padded(i + j)] = v;
      else mine[i + j] = v;
    }
  }
  if (blockDim.y == 1) return;
  __syncthreads();
  for (int i = t; i < a.H; i += TX * blockDim.y) {
    float s = ((float *)raw)[padded(i)];
    for (int g = 1; g < (int)blockDim.y; g++) s += ((float *)raw)[g * pitch + padded(i)];
    mine[i] = s;
  }
}

// dw[j] = sum over the blocks of parts[block][j]: 32 columns and 32 strands of blocks to a block
// of threads, a strand in four sums, the strands joined in a tree of five additions: 26 roundings in a
// row for 2432 blocks, where one sum a strand and one strand after another cost 106.
__global__ void __launch_bounds__(1024) join_kernel(const float *__restrict__ parts, int groups, int H, float *dw) {
  __shared__ float sh[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  grid_wait();
  if (col < H)
    for (int g = threadIdx.y; g < groups; g += 128)
#pragma unroll
      for (int j = 0; j < 4; j++)
        if (g + 32 * j < groups) s[j] += parts[(int64_t)(g + 32 * j) * H + col];
  sh[threadIdx.y][threadIdx.x] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  if (threadIdx.y == 0 && col < H) {
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; i++) v[i] = sh[i][threadIdx.x];
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
      for (int i = 0; i < o; i++) v[i] += v[i + o];
    dw[col] = v[0];
  }
}

// Rows longer than a block holds: mean(g z) of each row, then dx and parts of dw by columns.
template <class T, bool CKPT>
__global__ void __launch_bounds__(512) long_mean_kernel(const NormGradArgs a, float *__restrict__ mean) {
  __shared__ float sh[32];
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const float rstd = a.rstd[row];
    float dot = 0.f;
    for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
      float z[1], w[1];
      z[0] = input_at<T, CKPT>(a, row, i) * rstd;
      load_w<T, 1>(a.w, a.w32, i, w);
      dot = fmaf(to_f(((const T *)a.dy)[row * a.lddy + i]) * w[0], z[0], dot);
    }
    dot = row_sum<512>(dot, sh);
    if (threadIdx.x == 0) mean[row] = dot / (float)a.H;
  }
}
template <class T, bool CKPT>
__global__ void __launch_bounds__(256) long_grad_kernel(const NormGradArgs a, const float *__restrict__ mean,
                                                        float *__restrict__ parts) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= a.H) return;
  float w[1], dw = 0.f;
  load_w<T, 1>(a.w, a.w32, i, w);
  for (int64_t row = blockIdx.y; row < a.T; row += gridDim.y) {
    const float rstd = a.rstd[row], d = to_f(((const T *)a.dy)[row * a.lddy + i]);
    float z[1];
    z[0] = input_at<T, CKPT>(a, row, i) * rstd;
    dw = fmaf(d, z[0], dw);
    float x = rstd * (d * w[0] - z[0] * mean[row]);
    if (a.dres) x += to_f(((const T *)a.dres)[row * a.lddr + i]);
    ((T *)a.dx)[row * a.lddx + i] = from_f<T>(x);
  }
  parts[(int64_t)blockIdx.y * a.H + i] = dw;
}

// Blocks launched, -1 after an error.
template <class T, int VEC, int PER, int TX, bool CKPT>
int go(const NormGradArgs &a, float *parts, cudaStream_t st) {
  int rows = kThreads / TX;                    // as many as fit, but first a block on every multiprocessor
  if (rows > a.T / 152) rows = a.T / 152;
  if (rows < 1) rows = 1;
  if (TX > 32 && rows > 15) rows = 15;         // barriers
  const int need = (a.T + rows - 1) / rows, blocks = need < 152 ? need : 152;
  const size_t smem = 2 * sizeof(Stage<T, VEC, PER, CKPT>);
  static_assert(2 * sizeof(Stage<T, VEC, PER, CKPT>) >= kThreads / TX * (TX * PER * VEC * 9 / 8 + 2) * sizeof(float),
                "the parts of dw fit the copies' memory");
  if (!allow_smem<grad_kernel<T, VEC, PER, TX, CKPT>>((int)smem)) return -1;
  grad_kernel<T, VEC, PER, TX, CKPT><<<blocks, dim3(TX, rows), smem, st>>>(a, parts);
  return blocks;
}
template <class T, bool CKPT>
int grad_typed(const NormGradArgs &a, float *ws, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T), P = (V == 4 ? 16 : 32) / V;       // 32 columns a thread, 16 of fp32
  int groups = most_blocks(a.T, a.H);
  const bool wide = a.H % V == 0 && rows16(a.dy, a.lddy, sizeof(T)) && rows16(a.dres, a.lddr, sizeof(T)) &&
                    rows16(a.dx, a.lddx, sizeof(T)) && rows16(a.h, a.ldh, sizeof(T)) && rows16(a.w, 0, 4) &&
                    rows_on(a.q, a.ldq, 1, V);
  if (wide && a.H <= kThreads * V * P) {
    if (a.H <= 32 * V) groups = go<T, V, 1, 32, CKPT>(a, ws, st);
    else if (a.H <= 32 * V * P) groups = go<T, V, P, 32, CKPT>(a, ws, st);
    else if (a.H <= 64 * V * P) groups = go<T, V, P, 64, CKPT>(a, ws, st);
    else if (a.H <= 128 * V * P) groups = go<T, V, P, 128, CKPT>(a, ws, st);
    else if (a.H <= 256 * V * P) groups = go<T, V, P, 256, CKPT>(a, ws, st);
    else groups = go<T, V, P, 512, CKPT>(a, ws, st);
  } else if (a.H <= kMaxSingle) {
    groups = launch_grad_single<T, CKPT>(a, groups, ws, st);
  } else {
    float *mean = ws + (int64_t)groups * a.H;
    long_mean_kernel<T, CKPT><<<a.T < 152 * 4 ? a.T : 152 * 4, 512, 0, st>>>(a, mean);
    const int rc = launch_status();
    if (rc != MCEMU_OK) return rc;
    long_grad_kernel<T, CKPT><<<dim3((a.H + 255) / 256, groups), 256, 0, st>>>(a, mean, ws);
  }
  if (groups < 0) return MCEMU_ERR_CUDA;
  if (cudaGetLastError() != cudaSuccess) return MCEMU_ERR_CUDA;
  return launch_early(join_kernel, dim3((a.H + 31) / 32), dim3(32, 32), 0, st, ws, groups, a.H, a.dw);
}

template <class T>
int grad_any(const NormGradArgs &a, float *ws, cudaStream_t st) {
  return a.q ? grad_typed<T, true>(a, ws, st) : grad_typed<T, false>(a, ws, st);
}

}  // namespace

size_t rmsnorm_backward_workspace(int T, int H) {
  return ((size_t)most_blocks(T, H) * H + T) * sizeof(float);
}

int launch_rmsnorm_backward(int fmt, const NormGradArgs &a, void *ws, void *stream) {
  cudaStream_t st = (cudaStream_t)stream;
  float *f = (float *)ws;
  return fmt == MCEMU_FP32 ? grad_any<float>(a, f, st) : fmt == MCEMU_FP16 ? grad_any<__half>(a, f, st)
                                                                           : grad_any<__nv_bfloat16>(a, f, st);
}

}  // namespace mcemu
