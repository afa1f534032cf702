// tc.cuh -- PTX of sm_103a's fifth-generation tensor cores as the 8-bit layer products use
// it: mbarriers with bounded waits, tensor memory, the matrix instruction and its shared-memory
// operands in the 128-byte swizzle.  CG is the number of CTAs (1 or 2) that issue as one.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "../../include/mcemu_ops.h"

namespace mcemu {
namespace tc {

// Waits that gave up (one count to a translation unit, as is all that touches it: hence static).
static __device__ unsigned int g_timeouts = 0;

// How many gave up on the current device, as of the end of `st`, since the last question.  The count
// only grows, so that one that gives up on another stream meanwhile is there for the next question.
static inline int take_timeouts(cudaStream_t st, unsigned int *got) {
  static std::mutex alone;
  static unsigned int known[64];
  unsigned int now = 0, none = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess) return MCEMU_ERR_CUDA;
  const std::lock_guard<std::mutex> lock(alone);
  if (cudaMemcpyFromSymbolAsync(&now, g_timeouts, sizeof now, 0, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return MCEMU_ERR_CUDA;
  unsigned int &last = dev < 64 ? known[dev] : none;
  *got = now < last ? now : now - last;       // less than before: the device was reset
  last = now;
  return MCEMU_OK;
}

// Tensor map of a row-major matrix of 16-bit elements: `cols` x `rows`, `ld` elements between
// rows (a multiple of 8, as is the base of 16 bytes), boxes of 64 columns by `box` rows, stored
// plainly or in the 128-byte swizzle.  The driver's encoder is looked up once.
inline int tensor_map(CUtensorMap *map, const void *base, uint64_t cols, uint64_t rows, uint64_t ld, uint32_t box,
                      bool swizzle) {
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
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {ld * 2};
  const cuuint32_t boxes[2] = {64, box}, ones[2] = {1, 1};
  return ((Encode)f)(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void *>(base), dims, strides, boxes, ones,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? MCEMU_OK
             : MCEMU_ERR_CUDA;
}

// Moves the registers of a block of three warpgroups, 168 a thread at launch, from the third
// to the two that hold sums: 2 * 224 + 56 = 3 * 168.
__device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 224;"); }
__device__ __forceinline__ void give_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 56;"); }

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Sixteen bytes of the shared memory of CTA `rank` of the cluster, at this CTA's address `addr`.
__device__ __forceinline__ int4 load_peer(uint32_t addr, uint32_t rank) {
  uint32_t at;
  int4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---- mbarriers ---------------------------------------------------------------
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_init_fence() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Arrives on the barrier at the same offset in CTA 0 of the pair.  Relaxed: it orders no memory
// accesses, and has none to order.  What it announces are tensor-memory reads, which are complete
// (tmem_wait); the PTX manual's pattern for handing tensor memory to another thread after such is the
// fence before a thread synchronisation, a relaxed arrival at cluster scope, the wait, and the fence
// after it.  With a release in its place int8 8192 x 8192 x 4096 takes 332 us, 319 without.
__device__ __forceinline__ void mbar_arrive_lead(uint32_t bar) {
  asm volatile(
      "{\n.reg .b32 a;\nmapa.shared::cluster.u32 a, %0, 0;\n"
      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [a];\n}" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits for the phase of `parity` to end.  Gives up after two seconds: `dead` is then set, it is
// counted, and later waits return at once, so that the kernel runs to its end on what it has.
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
static __device__ __forceinline__ bool mbar_wait_long(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = now_ns();
  for (int i = 0; i < 1 << 26; i++) {
    if (mbar_try(bar, parity)) return true;
    if ((i & 63) == 63 && now_ns() - t0 > 2000000000ull) break;
  }
  atomicAdd(&g_timeouts, 1u);
  return false;
}
static __device__ __forceinline__ void mbar_wait(uint32_t bar, uint32_t parity, bool &dead) {
  if (dead) return;
#pragma unroll 1
  for (int i = 0; i < 64; i++)
    if (mbar_try(bar, parity)) return;
  dead = !mbar_wait_long(bar, parity);
}

// Copies a box of a two-dimensional tensor map, from element (x, y) on, into this CTA's shared
// memory and counts its bytes on the barrier at the same offset in CTA 0 of the pair.  Elements
// outside the tensor read as zeros and count too.
__device__ __forceinline__ void box_load_pair(uint32_t to, const CUtensorMap *map, int x, int y, uint32_t bar) {
  asm volatile(
      "{\n.reg .b32 b;\nmapa.shared::cluster.u32 b, %4, 0;\n"
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[b];\n}" ::"r"(to),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// The same by a whole warp, its verdict known to be common to all lanes: what the issuing warp
// does with it stays in uniform registers, which is what the matrix instruction reads.  (One lane
// alone in a branch moves every operand there anew: 120 cycles an instruction.)
static __device__ __forceinline__ void mbar_wait_warp(uint32_t bar, uint32_t parity, bool &dead) {
  if (dead) return;
#pragma unroll 1
  for (int i = 0; i < 64; i++)
    if (__any_sync(0xFFFFFFFFu, mbar_try(bar, parity))) return;
  dead = !__any_sync(0xFFFFFFFFu, mbar_wait_long(bar, parity));
}
// The warp's number in its block, known to be uniform.
__device__ __forceinline__ int warp_number() { return __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0); }

// ---- fences ------------------------------------------------------------------
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// ---- tensor memory (whole warps) ------------------------------------------------
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t where, uint32_t cols) {
  if constexpr (CG == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(where), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(where), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t cols) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols) : "memory");
}
// 16 consecutive columns of the warp's 32 lanes; complete after tmem_wait().
__device__ __forceinline__ void tmem_load16(uint32_t at, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(at));
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// ---- matrix instruction ------------------------------------------------------
// Shared-memory operand in 128-byte swizzle: rows of 128 bytes, eight to an atom of 1024.
// K-major (a row is 64 elements of K): `far` unused, `near` = 1024 between groups of eight
// rows.  MN-major (a row is 64 elements of M or N, eight k to an atom): `far` from one 64 of
// M or N to the next, `near` from one eight of k to the next.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t far, uint32_t near) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)(far >> 4) << 16 | (uint64_t)(near >> 4) << 32 | 1ull << 46 |
         2ull << 61;
}
// Instruction word of kind::f16: fp32 accumulators, binary16 (0) or bfloat16 (1) operands,
// each K-major (0) or MN-major (1).
__host__ __device__ constexpr uint32_t instruction(int m, int n, int bf16, int a_mn, int b_mn) {
  return 1u << 4 | (uint32_t)bf16 << 7 | (uint32_t)bf16 << 10 | (uint32_t)a_mn << 15 | (uint32_t)b_mn << 16 |
         (uint32_t)(n >> 3) << 17 | (uint32_t)(m >> 4) << 24;
}
// One matrix instruction, by one elected lane of the calling warp (all lanes call).
template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t ins, bool add) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.u32 p, %4, 0;\nelect.sync _|q, 0xFFFFFFFF;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(ins), "r"((uint32_t)add)
        : "memory");
  else
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.u32 p, %4, 0;\nelect.sync _|q, 0xFFFFFFFF;\n"
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(ins), "r"((uint32_t)add)
        : "memory");
}
// Arrives on `bar` (of both CTAs for CG 2) once every matrix instruction issued so far by the
// elected lane is done (all lanes call).
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n.reg .pred q;\nelect.sync _|q, 0xFFFFFFFF;\n"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar)
        : "memory");
  else
    asm volatile(
        "{\n.reg .pred q;\nelect.sync _|q, 0xFFFFFFFF;\n"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
// The same on this CTA's barrier alone.
template <int CG>
__device__ __forceinline__ void commit_here(uint32_t bar) {
  if constexpr (CG == 1) commit<1>(bar);
  else
    asm volatile(
        "{\n.reg .pred q;\nelect.sync _|q, 0xFFFFFFFF;\n"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar)
        : "memory");
}

}  // namespace tc
}  // namespace mcemu
