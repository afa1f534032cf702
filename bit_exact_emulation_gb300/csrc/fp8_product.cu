// fp8_product.cu -- FP8 products: which form a call takes, operands whose rows the copy engine
// cannot read, and sums of nothing.
#include <utility>

#include "fp8_plan.h"
#include "ops_common.cuh"

namespace mcemu {
namespace {

constexpr int kBlock = MCEMU_FP8_BLOCK;

// Sixteen bytes of a row of K from k on, zeros beyond its end, at any alignment: out of the four or five words that hold
// them (of which three bytes may lie beside the row).  Without a branch, so that several are under way at once.
__device__ __forceinline__ uint4 bytes16(const uint8_t *row, int k, int K) {
  const uintptr_t p = (uintptr_t)(row + k);
  const uint32_t *from = (const uint32_t *)(p & ~(uintptr_t)3);
  const int off = (int)(p & 3), left = K - k;
  uint32_t w[5], v[4];
#pragma unroll
  for (int i = 0; i < 5; i++) w[i] = 4 * i - off < left && left > 0 && (i < 4 || off) ? __ldg(from + i) : 0u;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    v[i] = __funnelshift_r(w[i], w[i + 1], 8 * off);
    const int n = left - 4 * i;               // bytes that count
    if (n < 4) v[i] = n <= 0 ? 0u : v[i] & 0xFFFFFFFFu >> (32 - 8 * n);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// Rows at any address to rows on 16-byte boundaries, sixteen bytes a thread, kCopies times; both operands by one
// kernel.  Of matrices for groups only those whose group has rows (or may have: an offset above the one before).
constexpr int kCopies = 4, kBlockTasks = 256 * kCopies;
struct Copy {
  const uint8_t *from;
  int64_t ld, stride;
  int rows, blocks;          // of one matrix: rows, and blocks of threads (0: no copy)
  uint8_t *to;
};
__global__ void __launch_bounds__(256) align_kernel(const Copy a, const Copy b, int K, int units, const int32_t *offsets, int T) {
  grid_go();
  int block = blockIdx.x, matrix = 0;
  const bool second = block >= a.blocks;
  if (second) {
    matrix = (block - a.blocks) / b.blocks;
    block = block - a.blocks - matrix * b.blocks;
    if (offsets && min(__ldg(offsets + matrix + 1), T) <= max(__ldg(offsets + matrix), 0)) return;
  }
  const int rows = second ? b.rows : a.rows;
  const int64_t ld = second ? b.ld : a.ld;
  const uint8_t *from = second ? b.from + matrix * b.stride : a.from;
  uint8_t *to = second ? b.to + (int64_t)matrix * rows * units * 16 : a.to;
  const int64_t first = (int64_t)block * kBlockTasks, row0 = first / units;
  const int skip = (int)(first - row0 * units);
  uint4 v[kCopies];
  int64_t place[kCopies];
#pragma unroll
  for (int n = 0; n < kCopies; n++) {
    const int at = skip + n * 256 + (int)threadIdx.x, down = at / units, unit = at - down * units;
    const int64_t row = row0 + down;
    place[n] = row < rows ? row * units + unit : -1;
    v[n] = bytes16(from + (row < rows ? row : 0) * ld, unit * 16, row < rows ? K : 0);
  }
#pragma unroll
  for (int n = 0; n < kCopies; n++)
    if (place[n] >= 0) *(uint4 *)(to + place[n] * 16) = v[n];
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
// `busy` tiles are expected and `most` possible (a group's rows are known on the device alone).  `out` is what a tile
// costs beside its blocks: turned (fp8_pair.cuh) 0.4, else in 16 bits 0.55 and in fp32 1.1 (weight gradients of 8
// experts, 2048 x 4096 each: 16 rounds of tiles 123 us, turned 17 rounds 119).  Sums of a few blocks wait for their results' way
// out, which this does not know: turned, 16 rounds of 17 blocks in fp32 are estimated at 89 us and take 113.
constexpr int kPairs = 76;
struct Choice {
  Fp8Plan plan;
  double us;
};
Choice pair_choice(int width, double busy, int64_t most, int blocks, double out) {
  const double full = busy < kPairs ? busy / kPairs : 1.0, rounds = (double)(int64_t)((busy + kPairs - 1) / kPairs);
  const double block = width == 224 ? 0.22 + 0.06 * full : 0.147 + 0.08 * full;
  return {Fp8Plan{false, width, most, 1, blocks, 0}, (width == 224 ? 6.7 : 5.4) + rounds * (blocks * block + out)};
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
  for (const bool turned : {false, true})
    for (int width : {224, 128}) {
      const int tile_a = turned ? width : 256;
      const int64_t across = tiles(p.b.rows, turned ? 256 : width);
      // a group's last tile is half empty on average
      const double high = p.by_k ? (double)groups * tiles(p.a.rows, tile_a)
                          : p.offsets ? p.a.rows / (double)tile_a + filled * 0.5
                                      : (double)tiles(p.a.rows, tile_a);
      const int64_t most = (p.by_k ? groups * tiles(p.a.rows, tile_a) : p.offsets ? p.a.rows / tile_a + groups : tiles(p.a.rows, tile_a)) * across;
      Choice c = pair_choice(width, high * across, most, each, turned ? 0.4 : p.out_fmt == MCEMU_FP32 ? 1.1 : 0.55);
      c.plan.turned = turned;
      if (best.us == 0 || c.us < best.us) best = c;
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
    const auto blocks = [&](int rows) { return ((int64_t)rows * (ld / 16) + kBlockTasks - 1) / kBlockTasks; };
    const int64_t blocks_a = a_rows ? 0 : blocks(p.a.rows), blocks_b = b_rows ? 0 : blocks(p.b.rows);
    const int64_t all = blocks_a + blocks_b * matrices;
    if (blocks_a > INT32_MAX || blocks_b > INT32_MAX || all > INT32_MAX) return MCEMU_ERR_UNSUPPORTED;
    const Copy a{p.a.q, p.a.ld, 0, p.a.rows, (int)blocks_a, to_a}, b{p.b.q, p.b.ld, p.b.stride, p.b.rows, (int)blocks_b, to_b};
    align_kernel<<<(unsigned)all, 256, 0, st>>>(a, b, p.K, ld / 16, p.by_k ? nullptr : p.offsets, p.T);
    const int rc = launch_status();
    if (rc != MCEMU_OK) return rc;                              // the operands would be whatever the workspace held
    if (!a_rows) p.a.q = to_a, p.a.ld = ld;
    if (!b_rows) p.b.q = to_b, p.b.ld = ld, p.b.stride = (int64_t)p.b.rows * ld;
  }
  if (plan.turned) {
    std::swap(p.a, p.b);
    p.turned = true;
  }
  return plan.few ? launch_fp8_few(p, plan, stream) : launch_fp8_pair(p, plan, stream);
}

}  // namespace mcemu
