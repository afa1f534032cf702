// fp8_few.cu -- the products of few rows (fp8_few.cuh) for each type of result.
#include "fp8_few.cuh"
#include "fp8_plan.h"

namespace mcemu {

int fp8_few_timeouts(cudaStream_t st, unsigned int *got) { return tc::take_timeouts(st, got); }

namespace {
template <class T>
int go(const Fp8Product &p, const Fp8Plan &plan, const CUtensorMap &ma, const CUtensorMap &mb, cudaStream_t st) {
  switch (plan.width) {
    case 16: return fp8::launch_few<T, 16>(p, ma, mb, plan.units, plan.parts, plan.per, plan.clusters, st);
    case 32: return fp8::launch_few<T, 32>(p, ma, mb, plan.units, plan.parts, plan.per, plan.clusters, st);
    case 64: return fp8::launch_few<T, 64>(p, ma, mb, plan.units, plan.parts, plan.per, plan.clusters, st);
    default: return fp8::launch_few<T, 128>(p, ma, mb, plan.units, plan.parts, plan.per, plan.clusters, st);
  }
}
}  // namespace

int launch_fp8_few(const Fp8Product &p, const Fp8Plan &plan, void *stream) {
  CUtensorMap ma, mb;
  int rc = fp8::tensor_map(&ma, -1, p.a.q, p.K, p.a.rows, p.a.ld, 1, 0, 128, plan.width);
  if (rc == MCEMU_OK) rc = fp8::tensor_map(&mb, -1, p.b.q, p.K, p.b.rows, p.b.ld, p.E, p.b.stride, 128, 128);
  if (rc != MCEMU_OK) return rc;
  cudaStream_t st = (cudaStream_t)stream;
  return p.out_fmt == MCEMU_FP32   ? go<float>(p, plan, ma, mb, st)
         : p.out_fmt == MCEMU_FP16 ? go<__half>(p, plan, ma, mb, st)
                                   : go<__nv_bfloat16>(p, plan, ma, mb, st);
}

}  // namespace mcemu
