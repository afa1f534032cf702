// norm_rows.cuh -- rows that no vector fits, on their way to shared memory (rmsnorm.cu,
// rmsnorm_grad_single.cu).
#pragma once
#include "ops_common.cuh"

namespace mcemu {

// One operand's rows, every `step` bytes, copied a row at a time to shared memory in aligned 16-byte
// units: a row's first byte then lies `off` behind the copy's.  Places beyond the row are
// zeros; up to 15 bytes before it are read with its first unit.
template <int TX, int PER, int BYTES>          // of an element, PER of which are a thread's
struct Rows {
  static constexpr int kPitch = PER * TX * BYTES + 16, kUnits = (PER * BYTES + 15) / 16;
  const uint8_t *row;
  int64_t step;
  int bytes, off;
  __device__ __forceinline__ Rows(const void *p, int64_t ld, int H)
      : row((const uint8_t *)p + blockIdx.x * ld * BYTES), step(gridDim.x * ld * BYTES), bytes(H * BYTES), off(0) {}
  __device__ __forceinline__ void unit(uint8_t *to, int u, int end) const {
    const uint32_t s = (uint32_t)__cvta_generic_to_shared(to + u);
    const int n = max(0, min(16, end - u));
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(s), "l"(row - off + (n ? u : 0)), "r"(n)
                 : "memory");
  }
  // Copies the next row.
  __device__ __forceinline__ void fetch(uint8_t *to) {
    off = (int)((uintptr_t)row & 15);
    const int end = off + bytes;
#pragma unroll
    for (int j = 0; j < kUnits; j++)
      if (j * TX * 16 + (int)threadIdx.x * 16 < kPitch) unit(to, (j * TX + (int)threadIdx.x) * 16, end);
    if (kPitch - 16 == kUnits * TX * 16 && threadIdx.x == 0) unit(to, kPitch - 16, end);
    row += step;
  }
};

}  // namespace mcemu
