// fp8_tc.cuh -- what the FP8 products' kernels share: sm_103a's block-scaled matrix instruction
// and its operands, exponents on their way to tensor memory, the groups' place in the work.
//
// Operands lie in shared memory as rows of 128 codes (one block of a row) in the 128-byte swizzle,
// 1024 bytes to eight rows, as the copy engine makes them.  The matrix unit multiplies 32 codes of a
// row at a time and scales the products by two exponents of eight bits (2^(byte - 127), 255: NaN; the
// stored exponent plus 127) out of tensor memory.  There a 32-bit word holds four bytes of
// one row, and a column of 32 lanes 32 rows: here the four bytes are four blocks of 128 along k, and
// each matrix instruction names the byte that it takes.  Four blocks' exponents of 128 rows lie in shared
// memory as 32 rows of 16 bytes: word i of row l belongs to the operand's row l + 32 i.
#pragma once
#include "fp8.h"
#include "ops_common.cuh"
#include "tc.cuh"

namespace mcemu {
namespace fp8 {

constexpr int kBlock = MCEMU_FP8_BLOCK;
constexpr int kTileBytes = 128 * kBlock;      // 128 rows of a block
// Blocks along k between two drains of few rows' accumulators: the matrix unit truncates what it adds up.
constexpr int kChunk = 4;
constexpr int kScaleBytes = 512;              // four blocks' exponents of 128 rows

// Tensor map of row-major matrices, boxes of `wide` columns by `high` rows; of codes (fmt < 0) in the 128-byte
// swizzle, of results plainly.
inline int tensor_map(CUtensorMap *map, int fmt, const void *base, uint64_t cols, uint64_t rows, uint64_t ld,
                      uint64_t matrices, uint64_t stride, uint32_t wide, uint32_t high) {
  using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static std::atomic<void *> known{nullptr};
  void *f = known.load();
  if (!f) {
    cudaDriverEntryPointQueryResult how;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &how) != cudaSuccess ||
        how != cudaDriverEntryPointSuccess || !f)
      return MCEMU_ERR_CUDA;
    known.store(f);
  }
  const int size = fmt < 0 ? 1 : fmt == MCEMU_FP32 ? 4 : 2;
  const CUtensorMapDataType type = fmt < 0             ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : fmt == MCEMU_FP32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : fmt == MCEMU_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                       : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint64_t dims[3] = {cols, rows, matrices}, strides[2] = {ld * size, (matrices > 1 ? stride : ld) * size};
  const cuuint32_t boxes[3] = {wide, high, 1}, ones[3] = {1, 1, 1};
  return ((Encode)f)(map, type, 3, const_cast<void *>(base), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     fmt < 0 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? MCEMU_OK
             : MCEMU_ERR_CUDA;
}

// ---- copies and barriers -------------------------------------------------------
// A box from (x, y, z) on into this CTA's shared memory, its bytes counted on this CTA's barrier; by one elected
// lane of the calling warp (all lanes call): alone in a branch it takes two to four times as long, 130 cycles and more.
__device__ __forceinline__ void box_load(uint32_t to, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "{\n.reg .pred q;\nelect.sync _|q, 0xFFFFFFFF;\n"
      "@q cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n}" ::"r"(to),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// The same for a pair of CTAs that issue matrix instructions as one: counted on `bar`, an address in the
// cluster (at_rank).
__device__ __forceinline__ void box_load_pair(uint32_t to, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "{\n.reg .pred q;\nelect.sync _|q, 0xFFFFFFFF;\n"
      "@q cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
      "%4}], [%5];\n}" ::"r"(to),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// This CTA's shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t at_rank(uint32_t addr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
// A box of shared memory to global memory, or added to what is there (fp32); by one thread, which also counts
// them in groups.  Rows outside the tensor are not written; a row is, with zeros, up to the end of its last 16 bytes, which
// is for the caller to avoid.
__device__ __forceinline__ void box_store(const CUtensorMap *map, uint32_t from, int x, int y, int z, bool add) {
  if (add)
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
                 "r"(x), "r"(y), "r"(z), "r"(from)
                 : "memory");
  else
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x),
                 "r"(y), "r"(z), "r"(from)
                 : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Fetches a tensor map ahead of its first use, which waits 600 cycles for it otherwise.
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// `bytes` of this CTA's shared memory to the address `to` in the cluster, counted on the barrier `bar` of the
// same CTA; by one thread.  That count is all that tells when the bytes have been read: the sender's own groups
// (boxes_left) hold only copies without a barrier.
__device__ __forceinline__ void bulk_push(uint32_t to, uint32_t from, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to), "r"(from),
               "r"(bytes), "r"(bar)
               : "memory");
}
// Until all of the calling thread's boxes have left shared memory, or are written.
__device__ __forceinline__ void boxes_left() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void boxes_written() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// Arrives on the barrier at the same offset in CTA `rank` of the cluster; what this thread has written is
// visible to who waits there at cluster scope.
__device__ __forceinline__ void mbar_arrive_at(uint32_t bar, uint32_t rank) {
  asm volatile(
      "{\n.reg .b32 a;\nmapa.shared::cluster.u32 a, %0, %1;\n"
      "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [a];\n}" ::"r"(bar),
      "r"(rank)
      : "memory");
}
__device__ __forceinline__ bool mbar_try_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// tc::mbar_wait_warp, at cluster scope: a bounded wait by a whole warp.
static __device__ __forceinline__ void mbar_wait_warp_cluster(uint32_t bar, uint32_t parity, bool &dead) {
  tc::mbar_wait_warp(bar, parity, dead);
  if (!dead) (void)mbar_try_cluster(bar, parity);        // the phase is over: this one only orders
}

// ---- matrix instruction -----------------------------------------------------------
// Instruction word of kind::mxf8f6f4: fp32 accumulators, E4M3 (0) or E5M2 (1) operands, both K-major,
// exponents in UE8M0, their bytes 0 of each word.
__host__ __device__ constexpr uint32_t instruction(int m, int n, int fmt_a, int fmt_b) {
  return (uint32_t)(fmt_a == MCEMU_E5M2) << 7 | (uint32_t)(fmt_b == MCEMU_E5M2) << 10 | (uint32_t)(n >> 3) << 17 |
         1u << 23 | (uint32_t)(m >> 4) << 24;
}
constexpr uint32_t kNextByte = 1u << 29 | 1u << 4;        // the same with the next byte of both words

// One matrix instruction over 32 of k, by one elected lane of the calling warp (all lanes call).
template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t ins, uint32_t scale_a,
                                    uint32_t scale_b, bool add) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.u32 p, %4, 0;\nelect.sync _|q, 0xFFFFFFFF;\n"
        "@q tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(ins), "r"((uint32_t)add), "r"(scale_a), "r"(scale_b)
        : "memory");
  else
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.u32 p, %4, 0;\nelect.sync _|q, 0xFFFFFFFF;\n"
        "@q tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(ins), "r"((uint32_t)add), "r"(scale_a), "r"(scale_b)
        : "memory");
}
// Four blocks' exponents of 128 rows from shared memory to four columns of tensor memory, in both CTAs for
// CG 2; ordered before the matrix instructions that the same thread issues after it.
template <int CG>
__device__ __forceinline__ void copy_scales(uint32_t to, uint32_t from) {
  // rows of 16 bytes, eight of them 128 bytes from the next eight, no swizzle
  const uint64_t desc = (uint64_t)((from & 0x3FFFF) >> 4) | 8ull << 16 | 8ull << 32 | 1ull << 46;
  if constexpr (CG == 1)
    asm volatile("{\n.reg .pred q;\nelect.sync _|q, 0xFFFFFFFF;\n@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n}" ::"r"(to),
                 "l"(desc)
                 : "memory");
  else
    asm volatile("{\n.reg .pred q;\nelect.sync _|q, 0xFFFFFFFF;\n@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n}" ::"r"(to),
                 "l"(desc)
                 : "memory");
}

// ---- exponents -----------------------------------------------------------------
// The exponents of rows `first` + lane + 32 i of an operand, on their way from memory to shared memory by a
// warp.
template <int R>
struct Scales {
  const int8_t *row[R];                       // null: the operand has no such row

  __device__ __forceinline__ void rows(const Fp8Operand &o, int matrix, int first) {
#pragma unroll
    for (int i = 0; i < R; i++) {
      const int r = first + (int)(threadIdx.x & 31) + 32 * i;
      row[i] = r < o.rows ? o.e + matrix * o.stride_e + (int64_t)(r >> o.tile) * o.lde : nullptr;
    }
  }
  // Those of blocks kb .. kb + 4 W - 1 of rows i0 .. i0 + 3, of which the ones before `end` count, as the matrix
  // unit takes them: 2^0 for rows that there are not and blocks from `end` on, whose codes are zeros or whose
  // sums nobody stores.  Read in aligned words, so that up to three bytes beside a row are read and not used.
  template <int W>
  __device__ __forceinline__ void load(int i0, int kb, int end, uint32_t (&w)[W][4]) const {
    uint32_t raw[4][W + 1];
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int j = 0; j <= W; j++) {
        raw[i][j] = 0;
        if (i0 + i >= R) continue;
        const uintptr_t p = (uintptr_t)(row[i0 + i] + kb);
        if (row[i0 + i] && kb + 4 * j - (int)(p & 3) < end && (j < W || (p & 3)))
          raw[i][j] = __ldg((const uint32_t *)(p & ~(uintptr_t)3) + j);
      }
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int j = 0; j < W; j++) {
        w[j][i] = 0x7F7F7F7Fu;
        if (i0 + i >= R) continue;
        uint32_t v = __funnelshift_r(raw[i][j], raw[i][j + 1], 8 * (int)((uintptr_t)(row[i0 + i] + kb) & 3));
        const int left = end - kb - 4 * j;    // blocks from here on
        if (left < 4) v = left <= 0 ? 0u : v & 0xFFFFFFFFu >> (32 - 8 * left);
        if (row[i0 + i]) w[j][i] = __vadd4(v, 0x7F7F7F7Fu);
      }
  }
};
// Words of rows l, l + 32, l + 64, l + 96 of 128, by lane l, to shared memory.
__device__ __forceinline__ void store_scales(uint32_t to, const uint32_t (&w)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + (threadIdx.x & 31) * 16), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3])
               : "memory");
}

// ---- groups ---------------------------------------------------------------------
// Where each group's rows (blocks) begin and how many tiles of `tile` rows come before it; by one warp.
// at[g] .. at[g + 1] are group g's rows, or with by_k its blocks of 128 along k; before[] as many entries.
// Offsets count as at most T and as no less than the one before.
__device__ __forceinline__ void place_groups(const Fp8Product &p, int tile, int *at, int *before) {
  const int lane = threadIdx.x & 31;
  if (!p.offsets) {
    if (lane == 0) at[0] = 0, at[1] = p.T, before[0] = 0, before[1] = (p.T + tile - 1) / tile;
    return;
  }
  int most = 0, blocks = 0, tiles = 0;        // of the groups before these 32
  for (int g0 = 0; g0 <= p.E; g0 += 32) {
    const int g = g0 + lane;
    int o = g <= p.E ? min(max(__ldg(p.offsets + g), 0), p.T) : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int other = __shfl_up_sync(0xFFFFFFFFu, o, d);
      if (lane >= d) o = max(o, other);
    }
    o = max(o, most);
    int last = __shfl_up_sync(0xFFFFFFFFu, o, 1);
    if (lane == 0) last = g0 ? most : o;
    // what ends at this offset: the group before it
    int b = g <= p.E ? (o - last + kBlock - 1) / kBlock : 0, t = g <= p.E ? (o - last + tile - 1) / tile : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int ob = __shfl_up_sync(0xFFFFFFFFu, b, d), ot = __shfl_up_sync(0xFFFFFFFFu, t, d);
      if (lane >= d) b += ob, t += ot;
    }
    if (g <= p.E) at[g] = p.by_k ? min(blocks + b, p.T / kBlock) : o, before[g] = tiles + t;
    most = __shfl_sync(0xFFFFFFFFu, o, 31);
    blocks += __shfl_sync(0xFFFFFFFFu, b, 31);
    tiles += __shfl_sync(0xFFFFFFFFu, t, 31);
  }
}

// ---- results ---------------------------------------------------------------------
// One result, added to what is there when fp32 and `accumulate`.  Volatile, so that nothing is read otherwise.
template <class T>
__device__ __forceinline__ void put_as(T *y, T v, int accumulate) {
  if constexpr (sizeof(T) == 4) {
    if (accumulate) v += *(volatile const T *)y;
  }
  *y = v;
}
template <class T>
__device__ __forceinline__ void put(T *y, float v, int accumulate) { put_as(y, from_f<T>(v), accumulate); }

// One result to shared memory.
template <class T>
__device__ __forceinline__ void put_shared(uint32_t to, float sum) {
  const T v = from_f<T>(sum);
  if constexpr (sizeof(T) == 4) asm volatile("st.shared.f32 [%0], %1;" ::"r"(to), "f"(v) : "memory");
  else asm volatile("st.shared.u16 [%0], %1;" ::"r"(to), "h"(*(const uint16_t *)&v) : "memory");
}
// Eight sums, or four of fp32, as they lie in memory.
template <class T>
__device__ __forceinline__ uint4 pack16(const float *sum) {
  uint32_t o[4];
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; i++) o[i] = __float_as_uint(sum[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float f[2] = {sum[2 * i], sum[2 * i + 1]};
      const Vec<T, 2> v = pack<T, 2>(f);
      o[i] = *(const uint32_t *)&v;
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace fp8
}  // namespace mcemu
