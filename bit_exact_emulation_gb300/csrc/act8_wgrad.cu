// act8_wgrad.cu -- a linear layer's weight gradient from the 8-bit checkpoint of its input
// (include/mcemu_ops.h has the formula).
//
// A product of dY^T (N x T) and the checkpoint (T x K) over the tokens, bound by the matrix unit:
// 8192 x 4096 x 4096 takes 171 us, 15 of them the widening: 1.61 PFLOP/s, 0.84 of the measured bf16
// rate.  A code times its power-of-two scale is a bfloat16 number, so the checkpoint is widened
// once to a bfloat16 panel (3 bytes of traffic an element) and the product is the matrix
// unit's, with exact operands.  Both operands are read with the tokens outermost as they lie in
// memory (MN-major); dY needs no panel of its own unless its rows miss 16-byte boundaries.
#include "panel.cuh"

namespace mcemu {
namespace {

// The image of 64 tokens by 128 columns: two halves of 64 columns, 8 KB each, a token's 64
// columns in 128 bytes.  Where 16-byte unit u (of 16) of token t lies in it:
__device__ __forceinline__ int image_at(int t, int u) {
  return (u >> 3) * 8192 + (t >> 3) * 1024 + (t & 7) * 128 + (((u & 7) ^ (t & 7)) << 4);
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *(const uint32_t *)&v;
}

// Checkpoint to panel, one image (64 tokens by one block of 128) to a block of threads: 16 codes a
// thread, twice.
__global__ void __launch_bounds__(256) widen_kernel(const WgradArgs a, int ttiles, bool wide, uint8_t *__restrict__ to) {
  const int block = blockIdx.x / ttiles, tt = blockIdx.x - block * ttiles;
  grid_go();
  to += (int64_t)blockIdx.x * panel::kTileBytes;
  const int piece = threadIdx.x & 7, r0 = threadIdx.x >> 3, k = block * 128 + 16 * piece;
  uint4 v[2];
  float s[2];
#pragma unroll
  for (int j = 0; j < 2; j++) {
    const int t = tt * 64 + r0 + 32 * j;
    v[j] = make_uint4(0, 0, 0, 0);
    s[j] = 0.f;
    if (t < a.T && k < a.K) {
      v[j] = row16(a.q + (int64_t)t * a.ldq, k, a.K, wide);
      s[j] = act8_scale(a.e[(int64_t)t * a.lde + block]);
    }
  }
#pragma unroll
  for (int j = 0; j < 2; j++) {
    const int r = r0 + 32 * j;
    float f[16];
    Vec<int8_t, 16> q;
    *(uint4 *)&q = v[j];
    bytes_to_f<16>(q, f);
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; i++) o[i] = bf16x2(f[2 * i] * s[j], f[2 * i + 1] * s[j]);
    // the swizzle keeps the 32 bytes in one sector, their halves exchanged in odd rows
    const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
    store32(to + (image_at(r, 2 * piece) & ~31), r & 1 ? hi : lo, r & 1 ? lo : hi);
  }
}

// dY to a panel, for rows that the copy engine cannot read: eight elements a thread, four times.
__global__ void __launch_bounds__(256) copy_kernel(const WgradArgs a, int ttiles, uint8_t *__restrict__ to) {
  const int64_t tile = blockIdx.x;
  const int block = (int)(tile / ttiles), tt = (int)(tile - (int64_t)block * ttiles);
  grid_go();
  to += tile * panel::kTileBytes;
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const int unit = threadIdx.x & 15, r = (threadIdx.x >> 4) + 16 * j, t = tt * 64 + r, n = block * 128 + 8 * unit;
    uint32_t o[4] = {0, 0, 0, 0};
    if (t < a.T) {
      const uint16_t *p = a.dy + (int64_t)t * a.lddy + n;
#pragma unroll
      for (int i = 0; i < 8; i++)
        if (n + i < a.N) o[i >> 1] |= (uint32_t)__ldg(p + i) << (16 * (i & 1));
    }
    *(uint4 *)(to + image_at(r, unit)) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

__device__ __forceinline__ void put(const WgradArgs &a, int64_t at, float v) {
  if (a.out_fmt == MCEMU_FP32) ((float *)a.dW)[at] = a.accumulate ? ((float *)a.dW)[at] + v : v;
  else ((__nv_bfloat16 *)a.dW)[at] = __float2bfloat16_rn(v);
}

struct WgradEp {
  using Sum = float;
  WgradArgs a;
  float *parts;              // of the shared tiles: [slot][BN][256]
  int bn;
  static __device__ __forceinline__ void add(float &s, float v) { s += v; }
  __device__ __forceinline__ void store(const panel::Unit &w, int k, int n0, const float *sum) const {
    if (w.slot >= 0) {
      float *p = parts + ((int64_t)w.slot * bn + n0 - w.tb * bn) * 256 + k - w.ta * 256;
#pragma unroll
      for (int x = 0; x < 16; x++) p[x * 256] = sum[x];
    } else if (k < a.K) {
#pragma unroll
      for (int x = 0; x < 16; x++)
        if (n0 + x < a.N) put(a, (int64_t)(n0 + x) * a.lddw + k, sum[x]);
    }
  }
};

// The shared tiles' parts, added in order: four rows of a tile to a block, four columns a thread.
__global__ void __launch_bounds__(256) join_kernel(const WgradArgs a, const panel::Args g, int bn,
                                                   const float *__restrict__ parts) {
  const int per = bn / 4, t = blockIdx.x / per, row = (blockIdx.x - t * per) * 4 + (threadIdx.x >> 6);
  const int col = (threadIdx.x & 63) * 4;
  int ta, tb;
  panel::tile_at(g, g.full + t, ta, tb);
  const int n = tb * bn + row, k = ta * 256 + col;
  grid_wait();
  if (n >= a.N || k >= a.K) return;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int p = 0; p < g.parts; p++) {
    const float4 v = *(const float4 *)(parts + ((int64_t)(p * g.rest + t) * bn + row) * 256 + col);
    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
  }
  const float o[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
  for (int i = 0; i < 4; i++)
    if (k + i < a.K) put(a, (int64_t)n * a.lddw + k + i, o[i]);
}

// No tokens: a gradient of zeros.
__global__ void __launch_bounds__(256) zero_kernel(const WgradArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < (int64_t)a.N * a.K) put(a, i / a.K * a.lddw + i % a.K, 0.f);
}

// 64-token tiles between two drains.  Relative error of 8192 x 4096 x 4096 against 64 bits, for activations
// with a few large channels (and for normal ones), and time: 4 tiles 1.4e-7 (1.2e-7), 178 us; 8 tiles
// 2.0e-7 (1.2e-7), 171 us; 16 tiles 4.3e-7 (1.8e-7), 169 us; 64 tiles 2.3e-6 (9.5e-7), 168 us.  A
// library's fp32 product of the same numbers: 5.1e-7 (2.9e-7).
constexpr int kChunk = 8;

struct Layout {
  int ttiles, blocks_k, blocks_n;
  panel::Plan cut;
  int64_t panel_x, panel_dy, parts;          // bytes
};
Layout layout_of(int T, int N, int K, bool direct) {
  Layout p;
  p.ttiles = (T + 63) / 64;
  p.blocks_k = (K + 255) / 256 * 2;
  p.blocks_n = (N + 255) / 256 * 2;
  p.cut = panel::plan_of(K, N, p.ttiles, true);
  p.panel_x = (int64_t)p.blocks_k * p.ttiles * panel::kTileBytes;
  p.panel_dy = direct ? 0 : (int64_t)p.blocks_n * p.ttiles * panel::kTileBytes;
  p.parts = (int64_t)p.cut.rest * p.cut.parts * 256 * p.cut.bn * 4;
  return p;
}

}  // namespace

int act8_wgrad_timeouts(cudaStream_t st, unsigned int *got) { return tc::take_timeouts(st, got); }

size_t act8_wgrad_workspace(int T, int N, int K, bool direct) {
  const Layout p = layout_of(T, N, K, direct);
  return (size_t)(p.panel_x + p.panel_dy + p.parts) + kPanelPad;
}

int launch_act8_wgrad(const WgradArgs &a, bool direct, void *ws, void *stream) {
  cudaStream_t st = (cudaStream_t)stream;
  const int64_t size = (int64_t)a.N * a.K, blocks = (size + 255) / 256;
  if (blocks > INT32_MAX) return MCEMU_ERR_UNSUPPORTED;
  if (a.T == 0) {
    zero_kernel<<<(unsigned)blocks, 256, 0, st>>>(a);
    return launch_status();
  }
  const Layout p = layout_of(a.T, a.N, a.K, direct);
  if (!panel::panel_fits(p.blocks_k, p.ttiles) || !panel::panel_fits(p.blocks_n, p.ttiles)) return MCEMU_ERR_UNSUPPORTED;
  uint8_t *px = panels_in(ws), *pdy = px + p.panel_x;
  float *parts = (float *)(pdy + p.panel_dy);
  widen_kernel<<<(unsigned)(p.blocks_k * p.ttiles), 256, 0, st>>>(a, p.ttiles, rows16(a.q, a.ldq, 1), px);
  int rc = launch_status();
  if (rc == MCEMU_OK && !direct) {
    copy_kernel<<<(unsigned)(p.blocks_n * p.ttiles), 256, 0, st>>>(a, p.ttiles, pdy);
    rc = launch_status();
  }
  if (rc != MCEMU_OK) return rc;              // the panels would be whatever the workspace held
  rc = panel::launch<WgradEp, 1, 1>(p.cut, px, a.K, pdy, a.N, direct ? a.dy : nullptr, a.lddy, a.T, p.ttiles,
                                              kChunk, WgradEp{a, parts, p.cut.bn}, st);
  if (rc != MCEMU_OK || !p.cut.rest) return rc;
  const panel::Args g{p.ttiles, p.blocks_k / 2, (a.N + p.cut.bn - 1) / p.cut.bn, p.cut.full, p.cut.rest, p.cut.parts,
                      p.cut.per_part, kChunk};
  return launch_early(join_kernel, dim3(p.cut.rest * p.cut.bn / 4), dim3(256), 0, st, a, g, p.cut.bn, (const float *)parts);
}

}  // namespace mcemu
