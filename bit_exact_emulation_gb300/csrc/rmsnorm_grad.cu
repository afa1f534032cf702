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

// Most blocks, each of which keeps a part of dw: one to a multiprocessor, more where a block is
// one group of threads for a short row.
int most_blocks(int T, int H) {
  const int per_sm = H <= 2048 ? 8 : H <= 16384 ? 16384 / H : 1, most = 152 * per_sm;
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

// h of one vector, as stored or from the checkpoint: f of get() times scale1() for the elements
// j with first(i, j), times scale2() for the others (a shifted vector may lie in two blocks of 128).
template <class T, int VEC, bool CKPT, bool SHIFT>
struct Input {
  Vec<T, VEC> h;
  __device__ __forceinline__ void load(const NormGradArgs &a, int64_t row, int i) {
    h = load_part<T, VEC, SHIFT>((const T *)a.h + row * a.ldh, i, a.H);
  }
  __device__ __forceinline__ void get(float (&f)[VEC]) const { unpack<T, VEC>(h, f); }
  __device__ __forceinline__ bool first(int, int) const { return true; }
  __device__ __forceinline__ float scale1() const { return 1.f; }
  __device__ __forceinline__ float scale2() const { return 1.f; }
};
template <class T, int VEC, bool SHIFT>
struct Input<T, VEC, true, SHIFT> {
  Vec<int8_t, VEC> q;
  int8_t e1, e2;
  __device__ __forceinline__ void load(const NormGradArgs &a, int64_t row, int i) {
    q = load_part<int8_t, VEC, SHIFT>(a.q + row * a.ldq, i, a.H);
    const int8_t *pe = a.e + row * a.lde;
    e1 = pe[max(i, 0) / MCEMU_ACT8_BLOCK];
    e2 = SHIFT ? pe[min(i + VEC - 1, a.H - 1) / MCEMU_ACT8_BLOCK] : e1;
  }
  __device__ __forceinline__ void get(float (&f)[VEC]) const { bytes_to_f<VEC>(q, f); }
  __device__ __forceinline__ bool first(int i, int j) const {
    return !SHIFT || j < MCEMU_ACT8_BLOCK - (i & (MCEMU_ACT8_BLOCK - 1));
  }
  __device__ __forceinline__ float scale1() const { return act8_scale(e1); }
  __device__ __forceinline__ float scale2() const { return act8_scale(e2); }
};

// Where column k of dw lies in shared memory: a word is left out after every eight, so that lanes
// eight (or four) columns apart meet different banks.
__device__ __forceinline__ int padded(int k) { return k + (k >> 3); }

// blockDim.y rows at a time to a block, TX threads to a row, PER vectors of it to a thread.  The
// groups of threads that hold a row each run on their own.  A thread copies its pieces of the next
// row into shared memory while it works on the present one, so that loads are in flight
// throughout without a register for them.  TX is known to the compiler, so that the vectors
// of a row lie at fixed distances; 32 elements a thread, where the row is long enough, keep what a
// row costs on top of its elements small.  8192 x 4096 bf16 with a residual path: GRADNOW us;
// rows loaded to registers when their turn comes 71; 8 elements a thread and TX a variable 86.
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
  float *join = (float *)(raw + 2 * sizeof(S));  // [H], padded, with several rows to a block
  const int t = threadIdx.y * TX + threadIdx.x;
  float dw[PER][VEC];
#pragma unroll
  for (int p = 0; p < PER; p++)
#pragma unroll
    for (int j = 0; j < VEC; j++) dw[p][j] = 0.f;
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
      float f[VEC], w[VEC], d[VEC], some = 0.f;
      get(p, f);
      unpack<T, VEC>(cur.dy[p][t], d);
      weights(p, i, w);
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        const float z = f[j] * scale[p];
        some = fmaf(d[j] * w[j], z, some);
        dw[p][j] = fmaf(d[j], z, dw[p][j]);
      }
      dot += some;
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
      // rstd * (g - z * mean) + dres, the factors of f gathered
      const float k = -(scale[p] * mean * rstd);
#pragma unroll
      for (int j = 0; j < VEC; j++) w[j] *= d[j];
      if (a.dres) unpack<T, VEC>(cur.dr[p][t], d);
#pragma unroll
      for (int j = 0; j < VEC; j++) f[j] = fmaf(f[j], k, a.dres ? fmaf(w[j], rstd, d[j]) : w[j] * rstd);
      store_vec((T *)a.dx + row * a.lddx + i, pack<T, VEC>(f));
    }
  }
  copy_wait<0>();
  // the groups' parts of dw, added in order
  float *mine = parts + (int64_t)blockIdx.x * a.H;
  for (int g = 0; g < (int)blockDim.y; g++) {
    if ((int)threadIdx.y == g) {
#pragma unroll
      for (int p = 0; p < PER; p++) {
        const int i = (p * TX + threadIdx.x) * VEC;
        if (i < a.H) {
#pragma unroll
          for (int j = 0; j < VEC; j++) {
            if (blockDim.y > 1) join[padded(i + j)] = g ? join[padded(i + j)] + dw[p][j] : dw[p][j];
            else mine[i + j] = dw[p][j];
          }
        }
      }
    }
    __syncthreads();
  }
  if (blockDim.y > 1)
    for (int i = t; i < a.H; i += TX * blockDim.y) mine[i] = join[padded(i)];
}

// Rows that do not start on 16-byte boundaries, but all alike: the vectors start on boundaries of
// memory, the columns of a thread change from row to row, and dw is kept in shared memory by the
// one group of threads that a block then has.
template <class T, int VEC, int PER, int TX, bool CKPT>
__global__ void __launch_bounds__(TX) shifted_kernel(const NormGradArgs a, float *__restrict__ parts) {
  __shared__ float sh[32];
  extern __shared__ float join[];               // [H], padded
  for (int i = threadIdx.x; i < padded(a.H) + 1; i += TX) join[i] = 0.f;
  __syncthreads();
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const T *pdy = (const T *)a.dy + row * a.lddy, *pdr = (const T *)a.dres + row * a.lddr;
    const int first = threadIdx.x * VEC - (int)(((uintptr_t)pdy / sizeof(T)) % VEC);
    Vec<T, VEC> dy[PER], dr[PER];
    Input<T, VEC, CKPT, true> in[PER];
#pragma unroll
    for (int p = 0; p < PER; p++) {
      const int i = first + p * TX * VEC;
      if (i < a.H) {
        dy[p] = load_part<T, VEC, true>(pdy, i, a.H);
        in[p].load(a, row, i);
        if (a.dres) dr[p] = load_part<T, VEC, true>(pdr, i, a.H);
      }
    }
    const float rstd = a.rstd[row];
    float dot = 0.f;
#pragma unroll
    for (int p = 0; p < PER; p++) {
      const int i = first + p * TX * VEC;
      if (i >= a.H) continue;
      float f[VEC], w[VEC], d[VEC], some = 0.f;
      in[p].get(f);
      unpack<T, VEC>(dy[p], d);
      load_w_part<T, VEC, true>(a.w, a.w32, i, a.H, w);
      const float s1 = in[p].scale1() * rstd, s2 = in[p].scale2() * rstd;
      float old[VEC];
#pragma unroll
      for (int j = 0; j < VEC; j++) old[j] = (unsigned)(i + j) < (unsigned)a.H ? join[padded(i + j)] : 0.f;
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        const float z = f[j] * (in[p].first(i, j) ? s1 : s2);
        some = fmaf(d[j] * w[j], z, some);
        old[j] = fmaf(d[j], z, old[j]);
      }
#pragma unroll
      for (int j = 0; j < VEC; j++)
        if ((unsigned)(i + j) < (unsigned)a.H) join[padded(i + j)] = old[j];
      dot += some;
    }
    const float mean = row_sum<TX>(dot, sh) / (float)a.H;
#pragma unroll
    for (int p = 0; p < PER; p++) {
      const int i = first + p * TX * VEC;
      if (i >= a.H) continue;
      float f[VEC], w[VEC], d[VEC];
      in[p].get(f);
      unpack<T, VEC>(dy[p], d);
      load_w_part<T, VEC, true>(a.w, a.w32, i, a.H, w);
      const float k1 = -(in[p].scale1() * rstd * mean * rstd), k2 = -(in[p].scale2() * rstd * mean * rstd);
#pragma unroll
      for (int j = 0; j < VEC; j++) w[j] *= d[j];
      if (a.dres) unpack<T, VEC>(dr[p], d);
#pragma unroll
      for (int j = 0; j < VEC; j++)
        f[j] = fmaf(f[j], in[p].first(i, j) ? k1 : k2, a.dres ? fmaf(w[j], rstd, d[j]) : w[j] * rstd);
      store_part<T, VEC, true>((T *)a.dx + row * a.lddx, i, a.H, pack<T, VEC>(f));
    }
    __syncthreads();                            // the next row's columns belong to other threads
  }
  float *mine = parts + (int64_t)blockIdx.x * a.H;
  for (int i = threadIdx.x; i < a.H; i += TX) mine[i] = join[padded(i)];
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

// Rows longer than a block holds, or whose operands lie differently in memory: mean(g z) of each row, then dx and parts of dw by columns.
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
      z[0] *= in.scale1() * rstd;
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
    z[0] *= in.scale1() * rstd;
    dw = fmaf(d, z[0], dw);
    float x = rstd * (d * w[0] - z[0] * mean[row]);
    if (a.dres) x += to_f(((const T *)a.dres)[row * a.lddr + i]);
    ((T *)a.dx)[row * a.lddx + i] = from_f<T>(x);
  }
  parts[(int64_t)blockIdx.x * a.H + i] = dw;
}

template <class K>
bool allow_smem(K kernel, size_t bytes) {
  return bytes <= 48 * 1024 ||
         cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess;
}

// Blocks launched, -1 after an error.
template <class T, int VEC, int PER, int TX, bool CKPT, bool SHIFT>
int go(const NormGradArgs &a, float *parts, cudaStream_t st) {
  if constexpr (SHIFT) {
    const int blocks = most_blocks(a.T, a.H);
    const size_t smem = (a.H + a.H / 8 + 2) * sizeof(float);
    if (!allow_smem(shifted_kernel<T, VEC, PER, TX, CKPT>, smem)) return -1;
    shifted_kernel<T, VEC, PER, TX, CKPT><<<blocks, TX, smem, st>>>(a, parts);
    return blocks;
  } else {
    int rows = kThreads / TX;                  // as many as fit, but first a block on every multiprocessor
    if (rows > a.T / 152) rows = a.T / 152;
    if (rows < 1) rows = 1;
    if (rows > 15) rows = 15;                  // barriers
    const int need = (a.T + rows - 1) / rows, blocks = need < 152 ? need : 152;
    const size_t smem = 2 * sizeof(Stage<T, VEC, PER, CKPT>) + (rows > 1 ? (a.H + a.H / 8 + 2) * sizeof(float) : 0);
    if (!allow_smem(grad_kernel<T, VEC, PER, TX, CKPT>, smem)) return -1;
    grad_kernel<T, VEC, PER, TX, CKPT><<<blocks, dim3(TX, rows), smem, st>>>(a, parts);
    return blocks;
  }
}

// The group of threads for rows of `span` columns.  32 columns a thread (16 of fp32) from the
// shared copies; 16 (8) with SHIFT, which has them in registers.
template <class T, int VEC, bool CKPT, bool SHIFT>
int pick(const NormGradArgs &a, int span, float *parts, cudaStream_t st) {
  constexpr int P = (VEC == 4 ? 16 : 32) / VEC / (SHIFT ? 2 : 1);
  if (span <= 32 * VEC) return go<T, VEC, 1, 32, CKPT, SHIFT>(a, parts, st);
  if (span <= 32 * VEC * P) return go<T, VEC, P, 32, CKPT, SHIFT>(a, parts, st);
  if (span <= 64 * VEC * P) return go<T, VEC, P, 64, CKPT, SHIFT>(a, parts, st);
  if (span <= 128 * VEC * P) return go<T, VEC, P, 128, CKPT, SHIFT>(a, parts, st);
  if (span <= 256 * VEC * P) return go<T, VEC, P, 256, CKPT, SHIFT>(a, parts, st);
  if constexpr (SHIFT)
    if (span > 512 * VEC * P) return go<T, VEC, P, 1024, CKPT, SHIFT>(a, parts, st);
  return go<T, VEC, P, 512, CKPT, SHIFT>(a, parts, st);
}

template <class T, bool CKPT>
int grad_typed(const NormGradArgs &a, float *ws, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T), kMost = kThreads * (V == 4 ? 16 : 32);      // columns held in registers
  int groups = most_blocks(a.T, a.H);
  Walk walk{V};
  walk.add(a.dy, a.lddy, sizeof(T));
  walk.add(a.dres, a.lddr, sizeof(T));
  walk.add(a.dx, a.lddx, sizeof(T));
  walk.add(a.h, a.ldh, sizeof(T));
  walk.add(a.q, a.ldq, 1);
  const bool wide = walk.ok && !walk.shifted() && a.H % V == 0 && rows16(a.w, 0, 4) && a.H <= kMost;
  // Rows that lie alike against 16-byte boundaries, as contiguous ones do whatever H is.
  const bool shift = walk.ok && !wide && a.H >= 64 && a.H + V - 1 <= kMost;
  if (wide) {
    groups = pick<T, V, CKPT, false>(a, a.H, ws, st);
  } else if (shift) {
    groups = pick<T, V, CKPT, true>(a, a.H + V - 1, ws, st);
  } else {
    float *mean = ws + (int64_t)groups * a.H;
    long_mean_kernel<T, CKPT><<<a.T < 152 * 4 ? a.T : 152 * 4, 512, 0, st>>>(a, mean);
    long_grad_kernel<T, CKPT><<<dim3(groups, (a.H + 255) / 256), 256, 0, st>>>(a, mean, ws);
  }
  if (groups < 0) return MCEMU_ERR_CUDA;
  join_kernel<<<(a.H + 31) / 32, dim3(32, 8), 0, st>>>(ws, groups, a.H, a.dw);
  return launch_status();
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
