// rmsnorm_grad.cu -- gradients of the root-mean-square norm, from its input or from an 8-bit
// checkpoint of it (include/mcemu_ops.h has the formulas).
//
// Bound by HBM: 7 bytes an element for bf16 gradients with a checkpoint and a residual path.
// Each group of threads walks over rows with its columns' weights and its part of dw in
// registers; the parts are added in a fixed order by a second, small kernel.
#include "ops_common.cuh"

namespace mcemu {
namespace {

constexpr int kMaxThreads = 512, kMaxPerThread = 32;
constexpr int kMaxRow = kMaxThreads * kMaxPerThread;   // longest row held in registers, half of it without vectors

// Blocks, each of which keeps a part of dw: as many as are resident, where there are rows for them.
int blocks_of(int T, int H) {
  const int most = H <= 2048 ? 4 * 152 : 2 * 152;
  return T < most ? T : most;
}

// Sum over the threads of a row (blockDim.x, whole warps); every row of the block calls it.
__device__ __forceinline__ float row_sum(float x, float *part) {
  x = warp_sum(x);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return x;
  float *mine = part + threadIdx.y * warps;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0.f;
  for (int i = 0; i < warps; i++) x += mine[i];
  return x;
}

// h of one vector, as stored or from the checkpoint.
template <class T, int VEC, bool CKPT>
struct Input {
  Vec<T, VEC> h;
  __device__ __forceinline__ void load(const NormGradArgs &a, int64_t row, int i) {
    h = load_vec<T, VEC>((const T *)a.h + row * a.ldh + i);
  }
  __device__ __forceinline__ void get(float (&f)[VEC], float rstd) const {
#pragma unroll
    for (int j = 0; j < VEC; j++) f[j] = to_f(h.v[j]) * rstd;
  }
};
template <class T, int VEC>
struct Input<T, VEC, true> {
  Vec<int8_t, VEC> q;
  int8_t e;
  __device__ __forceinline__ void load(const NormGradArgs &a, int64_t row, int i) {
    q = load_vec<int8_t, VEC>(a.q + row * a.ldq + i);
    e = a.e[row * a.lde + i / MCEMU_ACT8_BLOCK];
  }
  __device__ __forceinline__ void get(float (&f)[VEC], float rstd) const {
    const float s = act8_scale(e);
#pragma unroll
    for (int j = 0; j < VEC; j++) f[j] = (float)q.v[j] * s * rstd;
  }
};

template <class T, int VEC>
__device__ __forceinline__ void load_w(const NormGradArgs &a, int i, float (&f)[VEC]) {
#pragma unroll
  for (int j = 0; j < VEC; j++) f[j] = a.w32 ? ((const float *)a.w)[i + j] : to_f(((const T *)a.w)[i + j]);
}

// The vectors of a row that a thread holds, all loaded at once.
template <class T, int VEC, int PER, bool CKPT>
struct Row {
  Vec<T, VEC> dy[PER], dr[PER];
  Input<T, VEC, CKPT> in[PER];
  float rstd;
  __device__ __forceinline__ void load(const NormGradArgs &a, int64_t row) {
    if (row >= a.T) return;
    rstd = a.rstd[row];
#pragma unroll
    for (int p = 0; p < PER; p++) {
      const int i = (p * blockDim.x + threadIdx.x) * VEC;
      if (i < a.H) {
        dy[p] = load_vec<T, VEC>((const T *)a.dy + row * a.lddy + i);
        in[p].load(a, row, i);
        if (a.dres) dr[p] = load_vec<T, VEC>((const T *)a.dres + row * a.lddr + i);
      }
    }
  }
};

// blockDim.y rows at a time to a block, PER vectors of a row to a thread.  Where the registers
// allow it the next rows are loaded before the sum over the present ones is awaited.
template <class T, int VEC, int PER, bool CKPT>
__global__ void __launch_bounds__(kMaxThreads, VEC * PER <= 8 ? 2 : 1)
    grad_kernel(const NormGradArgs a, float *__restrict__ parts) {
  __shared__ float sh[32];
  extern __shared__ float join[];               // [blockDim.y][H] with several rows to a block
  float dw[PER][VEC];
#pragma unroll
  for (int p = 0; p < PER; p++)
#pragma unroll
    for (int j = 0; j < VEC; j++) dw[p][j] = 0.f;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t row0 = (int64_t)blockIdx.x * blockDim.y;
  constexpr bool kAhead = VEC * PER <= (VEC > 1 ? 16 : 8);
  Row<T, VEC, PER, CKPT> cur, nxt;
  if (kAhead) cur.load(a, row0 + threadIdx.y);
  for (; row0 < a.T; row0 += step) {
    const int64_t row = row0 + threadIdx.y;
    const bool live = row < a.T;
    if (kAhead) nxt.load(a, row + step);
    else cur.load(a, row);
    float dot = 0.f;
#pragma unroll
    for (int p = 0; p < PER; p++) {
      const int i = (p * blockDim.x + threadIdx.x) * VEC;
      if (i >= a.H || !live) continue;
      float z[VEC], w[VEC];
      cur.in[p].get(z, cur.rstd);
      load_w<T, VEC>(a, i, w);
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        const float d = to_f(cur.dy[p].v[j]);
        dot = fmaf(d * w[j], z[j], dot);
        dw[p][j] = fmaf(d, z[j], dw[p][j]);
      }
    }
    const float mean = row_sum(dot, sh) / (float)a.H;
#pragma unroll
    for (int p = 0; p < PER; p++) {
      const int i = (p * blockDim.x + threadIdx.x) * VEC;
      if (i >= a.H || !live) continue;
      float z[VEC], w[VEC];
      cur.in[p].get(z, cur.rstd);
      load_w<T, VEC>(a, i, w);
      Vec<T, VEC> o;
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        float x = cur.rstd * (to_f(cur.dy[p].v[j]) * w[j] - z[j] * mean);
        if (a.dres) x += to_f(cur.dr[p].v[j]);
        o.v[j] = from_f<T>(x);
      }
      store_vec((T *)a.dx + row * a.lddx + i, o);
    }
    if (kAhead) cur = nxt;
  }
  // dx may lie on dy or dres: a block only writes rows that it has read
  const bool several = blockDim.y > 1;
  float *mine = several ? join + (int64_t)threadIdx.y * a.H : parts + (int64_t)blockIdx.x * a.H;
#pragma unroll
  for (int p = 0; p < PER; p++) {
    const int i = (p * blockDim.x + threadIdx.x) * VEC;
    if (i < a.H) {
#pragma unroll
      for (int j = 0; j < VEC; j++) mine[i + j] = dw[p][j];
    }
  }
  if (!several) return;
  __syncthreads();
  for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < a.H; i += blockDim.x * blockDim.y) {
    float s = join[i];
    for (unsigned r = 1; r < blockDim.y; r++) s += join[r * a.H + i];
    parts[(int64_t)blockIdx.x * a.H + i] = s;
  }
}

// dw[j] = sum over the groups of parts[group][j]: 32 columns and eight strands of groups to
// a block, the strands joined in order.
__global__ void __launch_bounds__(256) join_kernel(const float *__restrict__ parts, int groups, int H, float *dw) {
  __shared__ float sh[8][33];
  const int col = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (col < H)
#pragma unroll 8
    for (int g = threadIdx.y; g < groups; g += 8) s += parts[(int64_t)g * H + col];
  sh[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && col < H) {
#pragma unroll
    for (int i = 1; i < 8; i++) s += sh[i][threadIdx.x];
    dw[col] = s;
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
      Input<T, 1, CKPT> in;
      float z[1], w[1];
      in.load(a, row, i);
      in.get(z, rstd);
      load_w<T, 1>(a, i, w);
      dot = fmaf(to_f(((const T *)a.dy)[row * a.lddy + i]) * w[0], z[0], dot);
    }
    dot = row_sum(dot, sh);
    if (threadIdx.x == 0) mean[row] = dot / (float)a.H;
  }
}
template <class T, bool CKPT>
__global__ void __launch_bounds__(256) long_grad_kernel(const NormGradArgs a, const float *__restrict__ mean,
                                                        float *__restrict__ parts) {
  const int i = blockIdx.y * blockDim.x + threadIdx.x;
  if (i >= a.H) return;
  float w[1], dw = 0.f;
  load_w<T, 1>(a, i, w);
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const float rstd = a.rstd[row], d = to_f(((const T *)a.dy)[row * a.lddy + i]);
    Input<T, 1, CKPT> in;
    float z[1];
    in.load(a, row, i);
    in.get(z, rstd);
    dw = fmaf(d, z[0], dw);
    float x = rstd * (d * w[0] - z[0] * mean[row]);
    if (a.dres) x += to_f(((const T *)a.dres)[row * a.lddr + i]);
    ((T *)a.dx)[row * a.lddx + i] = from_f<T>(x);
  }
  parts[(int64_t)blockIdx.x * a.H + i] = dw;
}

template <class T, int VEC, int PER, bool CKPT>
int go(const NormGradArgs &a, float *parts, cudaStream_t st) {
  const int items = (a.H + VEC - 1) / VEC, threads = ((items + PER - 1) / PER + 31) / 32 * 32;
  const int rows = threads < 256 && a.H <= 1024 ? 256 / threads : 1, most = blocks_of(a.T, a.H);
  const int blocks = (a.T + rows - 1) / rows < most ? (a.T + rows - 1) / rows : most;
  grad_kernel<T, VEC, PER, CKPT>
      <<<blocks, dim3(threads, rows), rows > 1 ? rows * a.H * sizeof(float) : 0, st>>>(a, parts);
  return blocks;
}

template <class T, bool CKPT>
int grad_typed(const NormGradArgs &a, float *ws, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  int groups = blocks_of(a.T, a.H);
  const bool wide = a.H % V == 0 && rows16(a.dy, a.lddy, sizeof(T)) && rows16(a.dres, a.lddr, sizeof(T)) &&
                    rows16(a.dx, a.lddx, sizeof(T)) && rows16(a.h, a.ldh, sizeof(T)) && rows_on(a.q, a.ldq, 1, V);
  if (a.H > (wide ? kMaxRow : kMaxRow / 2)) {
    float *mean = ws + (int64_t)groups * a.H;
    long_mean_kernel<T, CKPT><<<groups, 512, 0, st>>>(a, mean);
    long_grad_kernel<T, CKPT><<<dim3(groups, (a.H + 255) / 256), 256, 0, st>>>(a, mean, ws);
  } else if (wide) {
    if (a.H <= 4096) groups = go<T, V, 8 / V, CKPT>(a, ws, st);
    else if (a.H <= 8192) groups = go<T, V, 16 / V, CKPT>(a, ws, st);
    else groups = go<T, V, 32 / V, CKPT>(a, ws, st);
  } else {
    if (a.H <= 4096) groups = go<T, 1, 8, CKPT>(a, ws, st);
    else groups = go<T, 1, 16, CKPT>(a, ws, st);
  }
  join_kernel<<<(a.H + 31) / 32, dim3(32, 8), 0, st>>>(ws, groups, a.H, a.dw);
  return launch_status();
}

template <class T>
int grad_any(const NormGradArgs &a, float *ws, cudaStream_t st) {
  return a.q ? grad_typed<T, true>(a, ws, st) : grad_typed<T, false>(a, ws, st);
}

}  // namespace

size_t rmsnorm_backward_workspace(int T, int H) {
  return ((size_t)blocks_of(T, H) * H + (H > kMaxRow / 2 ? T : 0)) * sizeof(float);
}

int launch_rmsnorm_backward(int fmt, const NormGradArgs &a, void *ws, void *stream) {
  cudaStream_t st = (cudaStream_t)stream;
  float *f = (float *)ws;
  return fmt == MCEMU_FP32 ? grad_any<float>(a, f, st) : fmt == MCEMU_FP16 ? grad_any<__half>(a, f, st)
                                                                           : grad_any<__nv_bfloat16>(a, f, st);
}

}  // namespace mcemu
