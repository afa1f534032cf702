// fp8_product.cu -- FP8 products: which form a call takes, operands whose rows the copy engine
// cannot read, and sums of nothing.
#include "fp8_plan.h"
#include "ops_common.cuh"

namespace mcemu {
namespace {

constexpr int kBlock = MCEMU_FP8_BLOCK;

// Rows at any address to rows on 16-byte boundaries, sixteen bytes a thread.
__global__ void __launch_bounds__(256) align_kernel(const uint8_t *__restrict__ from, int64_t ld, int64_t stride, int rows,
                                                    int64_t tasks, int K, int ldto, uint8_t *__restrict__ to) {
  grid_go();
  const int64_t task = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (task >= tasks) return;
  const int units = ldto / 16;
  const int64_t row = task / units;
  const int k = (int)(task - row * units) * 16;
  const int64_t matrix = row / rows;
  *(uint4 *)(to + task * 16) = row16((const int8_t *)from + matrix * stride + (row - matrix * rows) * ld, k, K, false);
}

int align(const Fp8Operand &o, int matrices, int K, uint8_t *to, cudaStream_t st) {
  const int ldto = (K + 15) & ~15;
  const int64_t tasks = (int64_t)o.rows * matrices * (ldto / 16), blocks = (tasks + 255) / 256;
  if (blocks > INT32_MAX) return MCEMU_ERR_UNSUPPORTED;
  align_kernel<<<(unsigned)blocks, 256, 0, st>>>(o.q, o.ld, o.stride, o.rows, tasks, K, ldto, to);
  return launch_status();
}
int64_t aligned_bytes(int64_t rows, int matrices, int K) { return rows * matrices * ((K + 15) & ~15); }

// A product without blocks along k: bias, or zeros, in every row that belongs to a group.
template <class T>
__global__ void __launch_bounds__(256) empty_kernel(const Fp8Product p, int64_t tasks) {
  grid_go();
  grid_wait();
  const int64_t task = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (task >= tasks) return;
  const int64_t row = task / p.b.rows;
  const int n = (int)(task - row * p.b.rows);
  int64_t at = row * p.ldy;
  if (p.by_k) {
    const int64_t g = row / p.a.rows;
    at = g * p.stride_y + (row - g * p.a.rows) * p.ldy;
  } else if (p.offsets) {
    int most = 0, first = 0;
    for (int g = 0; g <= p.E; g++) {
      most = max(most, min(max(__ldg(p.offsets + g), 0), p.T));
      if (g == 0) first = most;
    }
    if (row < first || row >= most) return;
  }
  ((T *)p.y)[at + n] = from_f<T>(p.bias ? p.bias[n] : 0.f);
}
int launch_empty(const Fp8Product &p, cudaStream_t st) {
  if (p.accumulate) return MCEMU_OK;
  const int64_t tasks = (int64_t)p.a.rows * (p.by_k ? p.E : 1) * p.b.rows, blocks = (tasks + 255) / 256;
  if (blocks > INT32_MAX) return MCEMU_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)blocks), block(256);
  return p.out_fmt == MCEMU_FP32   ? launch_early(empty_kernel<float>, grid, block, 0, st, p, tasks)
         : p.out_fmt == MCEMU_FP16 ? launch_early(empty_kernel<__half>, grid, block, 0, st, p, tasks)
                                   : launch_early(empty_kernel<__nv_bfloat16>, grid, block, 0, st, p, tasks);
}

// Parts of K (a cluster's CTAs) and blocks of 128 to each: what takes the fewest blocks in a row, with two
// more for each unit's joining.  How many clusters run at a time is what a GB300 of 152 multiprocessors reports.
Fp8Plan few_plan(int64_t busy, int64_t units, int width, int blocks) {
  constexpr int kClusters[9] = {0, 152, 76, 46, 36, 28, 23, 15, 15};
  Fp8Plan best{true, width, units, 1, blocks, kClusters[1]};
  int64_t least = 0;
  for (int parts = 1; parts <= 8 && parts <= blocks; parts++) {
    const int per = (blocks + parts - 1) / parts;
    if (per * (parts - 1) >= blocks) continue;                  // a part would be empty
    const int64_t rounds = (busy + kClusters[parts] - 1) / kClusters[parts], steps = rounds * (per + (parts > 1 ? 2 : 1));
    if (parts == 1 || steps < least) {
      best = Fp8Plan{true, width, units, parts, per, kClusters[parts]};
      least = steps;
    }
  }
  return best;
}

Fp8Plan plan_of(const Fp8Product &p) {
  const int blocks = (p.K + kBlock - 1) / kBlock;
  const int64_t groups = p.by_k ? 1 : p.E, rows = ((int64_t)p.a.rows + groups - 1) / groups;
  if (!p.by_k && rows <= 128) {
    // a group's rows differ: tiles that hold half as many again, so that few weights are read twice
    const int64_t fit = p.offsets ? rows + rows / 2 : rows;
    const int width = fit <= 16 ? 16 : fit <= 32 ? 32 : fit <= 64 ? 64 : 128;
    const int64_t tiles_b = ((int64_t)p.b.rows + 127) / 128, filled = p.a.rows < groups ? p.a.rows : groups;
    return few_plan(filled * tiles_b, ((int64_t)p.a.rows / width + filled) * tiles_b, width, blocks);
  }
  const int width = 224;
  const int64_t tiles_b = ((int64_t)p.b.rows + width - 1) / width;
  const int64_t tiles_a = p.by_k ? ((int64_t)p.a.rows + 255) / 256 * p.E : (int64_t)p.a.rows / 256 + groups;
  return Fp8Plan{false, width, tiles_a * tiles_b, 1, blocks, 0};
}

}  // namespace

size_t fp8_product_workspace(int rows_a, int rows_b, int matrices_b, int K, bool a_rows, bool b_rows) {
  return (size_t)((a_rows ? 0 : aligned_bytes(rows_a, 1, K)) + (b_rows ? 0 : aligned_bytes(rows_b, matrices_b, K)));
}

int launch_fp8_product(const Fp8Product &given, bool a_rows, bool b_rows, void *ws, void *stream) {
  cudaStream_t st = (cudaStream_t)stream;
  Fp8Product p = given;
  if (p.K == 0) return launch_empty(p, st);
  const Fp8Plan plan = plan_of(p);
  if (plan.units > INT32_MAX / 2) return MCEMU_ERR_UNSUPPORTED;
  const int ld = (p.K + 15) & ~15, matrices = p.by_k ? 1 : p.E;
  uint8_t *to = (uint8_t *)ws;
  if (!a_rows) {
    const int rc = align(p.a, 1, p.K, to, st);
    if (rc != MCEMU_OK) return rc;                              // the operand would be whatever the workspace held
    p.a.q = to, p.a.ld = ld;
    to += aligned_bytes(p.a.rows, 1, p.K);
  }
  if (!b_rows) {
    const int rc = align(p.b, matrices, p.K, to, st);
    if (rc != MCEMU_OK) return rc;
    p.b.q = to, p.b.ld = ld, p.b.stride = (int64_t)p.b.rows * ld;
  }
  return plan.few ? launch_fp8_few(p, plan, stream) : launch_fp8_pair(p, plan, stream);
}

}  // namespace mcemu
