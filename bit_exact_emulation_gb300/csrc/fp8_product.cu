// fp8_product.cu -- FP8 products: which form a call takes, operands whose rows the copy engine
// cannot read, and sums of nothing.
#include "fp8_plan.h"
#include "ops_common.cuh"

namespace mcemu {
namespace {

constexpr int kBlock = MCEMU_FP8_BLOCK;

// Rows at any address to rows on 16-byte boundaries, sixteen bytes a thread; both operands by one kernel.
struct Copy {
  const uint8_t *from;
  int64_t ld, stride, tasks;
  int rows;
  uint8_t *to;
};
__global__ void __launch_bounds__(256) align_kernel(const Copy a, const Copy b, int K, int units) {
  grid_go();
  int64_t task = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const bool second = task >= a.tasks;
  if (second) task -= a.tasks;
  const Copy &c = second ? b : a;
  if (task >= c.tasks) return;
  const int64_t row = task / units, matrix = row / c.rows;
  const int k = (int)(task - row * units) * 16;
  *(uint4 *)(c.to + task * 16) = row16((const int8_t *)c.from + matrix * c.stride + (row - matrix * c.rows) * c.ld, k, K, false);
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

// Which form, and how it is cut: what ends soonest by these estimates in microseconds, whose constants are fitted
// to the following (bf16 results, operands in L2; `few` with the parts of K that it prefers):
//
//   M x N x K            few   pairs, 224   pairs, 128
//   16 x 1024 x 1024     4.5       7.2          6.2
//   512 x 1024 x 1024   10.2       8.6          7.2
//   16 x 4096 x 4096     5.5      13.0         13.4
//   128 x 4096 x 4096   12.5      14.2         11.4
//   512 x 4096 x 4096   12.8      14.8         12.9
//   1024 x 4096 x 4096  20.9      16.7         20.1
//   64 x 16384 x 4096    9.1      15.6         17.9
//   256 x 16384 x 4096  22.3      16.7         20.0
//   256 x 1024 x 8192   12.3      21.3         16.2
//   64 x 8192 x 8192    16.1      24.5         17.9
//   256 x 8192 x 8192   22.3      22.1         19.6
//   1024 x 8192 x 8192  72.1      42.8         61.9
//
// `busy` tiles are expected and `most` possible (a group's rows are known on the device alone).
constexpr int kPairs = 76;
struct Choice {
  Fp8Plan plan;
  double us;
};
Choice pair_choice(int width, double busy, int64_t most, int blocks) {
  const double full = busy < kPairs ? busy / kPairs : 1.0, rounds = (double)(int64_t)((busy + kPairs - 1) / kPairs);
  const double block = width == 224 ? 0.22 + 0.06 * full : 0.147 + 0.08 * full;
  return {Fp8Plan{false, width, most, 1, blocks, 0}, (width == 224 ? 6.7 : 5.4) + rounds * (blocks * block + 0.4)};
}
// Parts of K (a cluster's CTAs): how many clusters run at a time is what a GB300 of 152 multiprocessors reports.
// A join's time goes by the tokens of a tile; by 4096 x 4096, one part and four: 16 tokens 7.6 and 5.4 us, 64
// tokens 8.6 and 7.4, 80 tokens 11.2 and 9.2, 128 tokens 11.2 and 11.6.
Choice few_choice(int width, int64_t tokens, double busy, int64_t most, int blocks) {
  constexpr int kClusters[9] = {0, 152, 76, 46, 36, 28, 23, 15, 15};
  const double n = (double)(tokens < width ? tokens : width), join = 0.3 + n * n / 3400;
  const double start = width == 128 ? 5.2 : 4.1 + width * 0.005;
  Choice best{};
  for (int parts = 1; parts <= 8 && parts <= blocks; parts++) {
    const int per = (blocks + parts - 1) / parts;
    if (per * (parts - 1) >= blocks) continue;                  // a part would be empty
    if (parts > 1 && width > 32 && most > kClusters[parts]) continue;          // see fp8_few.cuh
    const double full = busy * parts < 152 ? busy * parts / 152 : 1.0;
    const double block = width == 128 ? 0.17 + 0.07 * full : width == 64 ? 0.12 + 0.03 * full : 0.11;
    const double rounds = (double)(int64_t)((busy + kClusters[parts] - 1) / kClusters[parts]);
    const double us = start + rounds * (per * block + (parts > 1 ? join : 0.2));
    // fewer parts where that costs nothing (128 rows of 32 experts of 2048 x 4096: one 43.6 us, two 47.5)
    if (parts == 1 || us < 0.97 * best.us) best = {Fp8Plan{true, width, most, parts, per, kClusters[parts]}, us};
  }
  return best;
}

Fp8Plan plan_of(const Fp8Product &p) {
  const int blocks = (p.K + kBlock - 1) / kBlock;
  // sums over groups of blocks: a group's share of them is one unit's work
  const int64_t groups = p.E, filled = p.by_k || p.a.rows > groups ? groups : p.a.rows;
  const int each = p.by_k ? (int)((blocks + groups - 1) / groups) : blocks;
  const auto tiles = [](int64_t rows, int tile) { return (rows + tile - 1) / tile; };
  Choice best{};
  for (int width : {224, 128}) {
    const int64_t across = tiles(p.b.rows, width);
    // a group's last tile is half empty on average
    const double high = p.by_k ? (double)groups * tiles(p.a.rows, 256)
                        : p.offsets ? p.a.rows / 256.0 + filled * 0.5
                                    : (double)tiles(p.a.rows, 256);
    const int64_t most = (p.by_k ? groups * tiles(p.a.rows, 256) : p.offsets ? p.a.rows / 256 + groups : tiles(p.a.rows, 256)) * across;
    const Choice c = pair_choice(width, high * across, most, each);
    if (width == 224 || c.us < best.us) best = c;
  }
  if (p.by_k) return best.plan;
  const int64_t across = tiles(p.b.rows, 128), mean = tiles(p.a.rows, (int)filled);
  for (int width : {16, 32, 64, 128}) {
    if (width < 128 && width < (p.offsets ? mean + mean / 2 : mean)) continue;       // would read most weights twice
    const double high = p.offsets ? p.a.rows / (double)width + filled * 0.5 : (double)tiles(p.a.rows, width);
    const int64_t most = (p.offsets ? p.a.rows / width + filled : tiles(p.a.rows, width)) * across;
    const Choice c = few_choice(width, mean, (high > filled ? high : (double)filled) * across, most, blocks);
    if (c.us < best.us) best = c;
  }
  return best.plan;
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
  if (!a_rows || !b_rows) {
    const int ld = (p.K + 15) & ~15, matrices = p.by_k ? 1 : p.E;
    uint8_t *to_a = (uint8_t *)ws, *to_b = to_a + (a_rows ? 0 : aligned_bytes(p.a.rows, 1, p.K));
    const Copy a{p.a.q, p.a.ld, 0, a_rows ? 0 : (int64_t)p.a.rows * (ld / 16), p.a.rows, to_a};
    const Copy b{p.b.q, p.b.ld, p.b.stride, b_rows ? 0 : (int64_t)p.b.rows * matrices * (ld / 16), p.b.rows, to_b};
    const int64_t blocks = (a.tasks + b.tasks + 255) / 256;
    if (blocks > INT32_MAX) return MCEMU_ERR_UNSUPPORTED;
    align_kernel<<<(unsigned)blocks, 256, 0, st>>>(a, b, p.K, ld / 16);
    const int rc = launch_status();
    if (rc != MCEMU_OK) return rc;                              // the operands would be whatever the workspace held
    if (!a_rows) p.a.q = to_a, p.a.ld = ld;
    if (!b_rows) p.b.q = to_b, p.b.ld = ld, p.b.stride = (int64_t)p.b.rows * ld;
  }
  return plan.few ? launch_fp8_few(p, plan, stream) : launch_fp8_pair(p, plan, stream);
}

}  // namespace mcemu
