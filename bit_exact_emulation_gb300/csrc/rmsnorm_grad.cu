// rmsnorm_grad.cu -- gradients of the root-mean-square norm, from its input or from an 8-bit
// checkpoint of it (include/mcemu_ops.h has the formulas).
//
// Bound by HBM: 7 bytes an element for bf16 gradients with a checkpoint and a residual path.
// Each group of threads walks over rows with its columns' weights and its part of dw in
// registers; the parts are added in a fixed order by a second, small kernel.
#include "ops_common.cuh"

namespace mcemu {
namespace {

constexpr int kThreads = 512;                  // of a block
constexpr int kMaxRow = 16384;                 // longest row held in registers, half of it without vectors

// Blocks, each of which keeps a part of dw: one to a multiprocessor, where there are rows for them.
int blocks_of(int T) { return T < 152 ? T : 152; }

// Sum over the threads of a row (blockDim.x, whole warps), which wait for one another alone.
__device__ __forceinline__ float row_sum(float x, float *part) {
  x = warp_sum(x);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return x;
  float *mine = part + threadIdx.y * warps;
  const int bar = threadIdx.y + 1;
  asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"((int)blockDim.x) : "memory");
  if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = x;
  asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"((int)blockDim.x) : "memory");
  x = 0.f;
  for (int i = 0; i < warps; i++) x += mine[i];
  return x;
}

// h of one vector, as stored or from the checkpoint: get() gives f with h = f * scale(j).
template <class T, int VEC, bool CKPT, bool SHIFT>
struct Input {
  Vec<T, VEC> h;
  __device__ __forceinline__ void load(const NormGradArgs &a, int64_t row, int i) {
    h = load_part<T, VEC, SHIFT>((const T *)a.h + row * a.ldh, i, a.H);
  }
  __device__ __forceinline__ void get(float (&f)[VEC]) const {
#pragma unroll
    for (int j = 0; j < VEC; j++) f[j] = to_f(h.v[j]);
  }
  __device__ __forceinline__ float scale(int, int) const { return 1.f; }
};
template <class T, int VEC, bool SHIFT>
struct Input<T, VEC, true, SHIFT> {
  Vec<int8_t, VEC> q;
  int8_t e, e2;              // of the block of 128 where the vector begins, and of the one where it ends
  __device__ __forceinline__ void load(const NormGradArgs &a, int64_t row, int i) {
    q = load_part<int8_t, VEC, SHIFT>(a.q + row * a.ldq, i, a.H);
    const int8_t *pe = a.e + row * a.lde;
    e = pe[max(i, 0) / MCEMU_ACT8_BLOCK];
    e2 = SHIFT ? pe[min(i + VEC - 1, a.H - 1) / MCEMU_ACT8_BLOCK] : e;
  }
  __device__ __forceinline__ void get(float (&f)[VEC]) const { bytes_to_f<VEC>(q, f); }
  __device__ __forceinline__ float scale(int i, int j) const {
    return act8_scale(SHIFT && ((i + j) & (MCEMU_ACT8_BLOCK - 1)) < j ? e2 : e);
  }
};

// The vectors of a row that a thread holds, all loaded at once.
template <class T, int VEC, int PER, bool CKPT, bool SHIFT>
struct Row {
  Vec<T, VEC> dy[PER], dr[PER];
  Input<T, VEC, CKPT, SHIFT> in[PER];
  __device__ __forceinline__ void load(const NormGradArgs &a, int64_t row, int back) {
#pragma unroll
    for (int p = 0; p < PER; p++) {
      const int i = (p * blockDim.x + threadIdx.x) * VEC - back;
      if (i < a.H) {
        dy[p] = load_part<T, VEC, SHIFT>((const T *)a.dy + row * a.lddy, i, a.H);
        in[p].load(a, row, i);
        if (a.dres) dr[p] = load_part<T, VEC, SHIFT>((const T *)a.dres + row * a.lddr, i, a.H);
      }
    }
  }
};

// blockDim.y rows at a time to a block, PER vectors of a row to a thread.  The groups of
// threads that hold a row each run on their own, so that while one waits for its sum the others
// load or store.  Many elements a thread (32 where the row is long enough) keep what a row costs
// on top of its elements small: 8 took 57 instructions an element, and 86 us for 8192 x 4096
// bf16 with a residual path in place of GRADNOW.
template <class T, int VEC, int PER, bool CKPT>
__global__ void __launch_bounds__(kThreads, 1) grad_kernel(const NormGradArgs a, float *__restrict__ parts) {
  __shared__ float sh[32];
  extern __shared__ float join[];               // [H]
  float dw[PER][VEC];
#pragma unroll
  for (int p = 0; p < PER; p++)
#pragma unroll
    for (int j = 0; j < VEC; j++) dw[p][j] = 0.f;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  for (int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; row < a.T; row += step) {
    Row<T, VEC, PER, CKPT, false> cur;
    cur.load(a, row, 0);
    const float rstd = a.rstd[row];
    float dot = 0.f;
#pragma unroll
    for (int p = 0; p < PER; p++) {
      const int i = (p * blockDim.x + threadIdx.x) * VEC;
      if (i >= a.H) continue;
      float f[VEC], w[VEC], some = 0.f;
      cur.in[p].get(f);
      load_w<T, VEC>(a.w, a.w32, i, w);
      const float s = cur.in[p].scale(i, 0) * rstd;      // z = f * s
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        const float d = to_f(cur.dy[p].v[j]), z = f[j] * s;
        some = fmaf(d * w[j], z, some);
        dw[p][j] = fmaf(d, z, dw[p][j]);
      }
      dot += some;
    }
    const float mean = row_sum(dot, sh) / (float)a.H;
#pragma unroll
    for (int p = 0; p < PER; p++) {
      const int i = (p * blockDim.x + threadIdx.x) * VEC;
      if (i >= a.H) continue;
      float f[VEC], w[VEC];
      cur.in[p].get(f);
      load_w<T, VEC>(a.w, a.w32, i, w);
      const float s = cur.in[p].scale(i, 0) * rstd;
      Vec<T, VEC> o;
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        const float x = rstd * fmaf(-(f[j] * s), mean, to_f(cur.dy[p].v[j]) * w[j]);
        o.v[j] = from_f<T>(a.dres ? x + to_f(cur.dr[p].v[j]) : x);
      }
      store_vec((T *)a.dx + row * a.lddx + i, o);
    }
  }
  // the groups' parts of dw, added in order
  for (int g = 0; g < (int)blockDim.y; g++) {
    float *to = blockDim.y > 1 ? join : parts + (int64_t)blockIdx.x * a.H;
    if ((int)threadIdx.y == g) {
#pragma unroll
      for (int p = 0; p < PER; p++) {
        const int i = (p * blockDim.x + threadIdx.x) * VEC;
        if (i < a.H) {
#pragma unroll
          for (int j = 0; j < VEC; j++) to[i + j] = g ? to[i + j] + dw[p][j] : dw[p][j];
        }
      }
    }
    __syncthreads();
  }
  if (blockDim.y > 1)
    for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < a.H; i += blockDim.x * blockDim.y)
      parts[(int64_t)blockIdx.x * a.H + i] = join[i];
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
      Input<T, 1, CKPT, false> in;
      float z[1], w[1];
      in.load(a, row, i);
      in.get(z);
      z[0] *= in.scale(i, 0) * rstd;
      load_w<T, 1>(a.w, a.w32, i, w);
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
  load_w<T, 1>(a.w, a.w32, i, w);
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const float rstd = a.rstd[row], d = to_f(((const T *)a.dy)[row * a.lddy + i]);
    Input<T, 1, CKPT, false> in;
    float z[1];
    in.load(a, row, i);
    in.get(z);
    z[0] *= in.scale(i, 0) * rstd;
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
  int rows = kThreads / threads;               // as many as fit, but first a block on every multiprocessor
  if (rows > a.T / 152) rows = a.T / 152;
  if (rows < 1) rows = 1;
  if (rows > 15) rows = 15;                    // barriers
  const int need = (a.T + rows - 1) / rows, blocks = need < blocks_of(a.T) ? need : blocks_of(a.T);
  grad_kernel<T, VEC, PER, CKPT><<<blocks, dim3(threads, rows), rows > 1 ? a.H * sizeof(float) : 0, st>>>(a, parts);
  return blocks;
}

template <class T, bool CKPT>
int grad_typed(const NormGradArgs &a, float *ws, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  int groups = blocks_of(a.T);
  const bool wide = a.H % V == 0 && rows16(a.dy, a.lddy, sizeof(T)) && rows16(a.dres, a.lddr, sizeof(T)) &&
                    rows16(a.dx, a.lddx, sizeof(T)) && rows16(a.h, a.ldh, sizeof(T)) && rows16(a.w, 0, 4) &&
                    rows_on(a.q, a.ldq, 1, V);
  if (a.H > (wide ? kMaxRow : kMaxRow / 2)) {
    float *mean = ws + (int64_t)groups * a.H;
    long_mean_kernel<T, CKPT><<<a.T < 152 * 4 ? a.T : 152 * 4, 512, 0, st>>>(a, mean);
    long_grad_kernel<T, CKPT><<<dim3(groups, (a.H + 255) / 256), 256, 0, st>>>(a, mean, ws);
  } else if (wide) {
    if (a.H <= 256) groups = go<T, V, 8 / V, CKPT>(a, ws, st);
    else if (a.H <= 512 || (V == 4 && a.H <= 8192)) groups = go<T, V, 16 / V, CKPT>(a, ws, st);
    else groups = go<T, V, 32 / V, CKPT>(a, ws, st);
  } else {
    if (a.H <= 1024) groups = go<T, 1, 4, CKPT>(a, ws, st);
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
  return ((size_t)blocks_of(T) * H + (H > kMaxRow / 2 ? T : 0)) * sizeof(float);
}

int launch_rmsnorm_backward(int fmt, const NormGradArgs &a, void *ws, void *stream) {
  cudaStream_t st = (cudaStream_t)stream;
  float *f = (float *)ws;
  return fmt == MCEMU_FP32 ? grad_any<float>(a, f, st) : fmt == MCEMU_FP16 ? grad_any<__half>(a, f, st)
                                                                           : grad_any<__nv_bfloat16>(a, f, st);
}

}  // namespace mcemu
