// fp8_pair.cu -- the pairs' products (fp8_pair.cuh) for each type of result.
#include "fp8_pair.cuh"
#include "fp8_plan.h"

namespace mcemu {

int fp8_pair_timeouts(cudaStream_t st, unsigned int *got) { return tc::take_timeouts(st, got); }

namespace {
template <class T>
int go(const Fp8Product &p, const Fp8Plan &plan, const CUtensorMap &ma, const CUtensorMap &mb, cudaStream_t st) {
  if (p.turned)
    return plan.width == 224 ? fp8::launch_pair<T, 224, true>(p, ma, mb, plan.units, st)
                             : fp8::launch_pair<T, 128, true>(p, ma, mb, plan.units, st);
  return plan.width == 224 ? fp8::launch_pair<T, 224, false>(p, ma, mb, plan.units, st)
                           : fp8::launch_pair<T, 128, false>(p, ma, mb, plan.units, st);
}
}  // namespace

int launch_fp8_pair(const Fp8Product &p, const Fp8Plan &plan, void *stream) {
  CUtensorMap ma, mb;
  const int of_a = p.turned && !p.by_k ? p.E : 1, of_b = p.turned || p.by_k ? 1 : p.E;      // matrices
  int rc = fp8::tensor_map(&ma, -1, p.a.q, p.K, p.a.rows, p.a.ld, of_a, p.a.stride, 128, 128);
  if (rc == MCEMU_OK) rc = fp8::tensor_map(&mb, -1, p.b.q, p.K, p.b.rows, p.b.ld, of_b, p.b.stride, 128, plan.width / 2);
  if (rc != MCEMU_OK) return rc;
  cudaStream_t st = (cudaStream_t)stream;
  return p.out_fmt == MCEMU_FP32   ? go<float>(p, plan, ma, mb, st)
         : p.out_fmt == MCEMU_FP16 ? go<__half>(p, plan, ma, mb, st)
                                   : go<__nv_bfloat16>(p, plan, ma, mb, st);
}

}  // namespace mcemu
