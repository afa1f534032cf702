"""The bounded waits of the 8-bit products' kernels, made to run out: a barrier that nothing arrives at."""
import ctypes
import subprocess
import time

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

SOURCE = r"""
#include "%s/tc.cuh"
using namespace mcemu::tc;
static __global__ void __launch_bounds__(64) wait_kernel(unsigned *gave_up) {
  __shared__ __align__(8) uint64_t bars[2];
  if (threadIdx.x == 0) {
    mbar_init(smem_addr(&bars[0]), 1);
    mbar_init(smem_addr(&bars[1]), 1);
    mbar_init_fence();
  }
  __syncthreads();
  bool dead = false;
  if (threadIdx.x == 0) mbar_wait(smem_addr(&bars[0]), 0, dead);
  if (threadIdx.x >= 32)
    for (int i = 0; i < 5; i++) mbar_wait_warp(smem_addr(&bars[1]), 0, dead);    // later ones return at once
  gave_up[threadIdx.x] = dead;
}
extern "C" int start(unsigned *gave_up, cudaStream_t st) {
  wait_kernel<<<1, 64, 0, st>>>(gave_up);
  return cudaGetLastError();
}
extern "C" int take(unsigned *got, cudaStream_t st) { return take_timeouts(st, got); }
"""


def test_a_wait_that_runs_out_is_counted_and_the_kernel_ends(tmp_path):
    from bit_exact_emulation_gb300 import build as B
    src, so = tmp_path / "waits.cu", tmp_path / "waits.so"
    src.write_text(SOURCE % B.CSRC)
    subprocess.run([B._nvcc(), *B.ARCH, *B.FLAGS, "-shared", str(src), "-o", str(so)], check=True)
    L = ctypes.CDLL(str(so))
    L.start.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    L.take.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    gave_up = torch.full((64,), 7, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    st = torch.cuda.current_stream().cuda_stream
    got = ctypes.c_uint(9)

    def take():
        assert L.take(ctypes.byref(got), st) == 0
        return got.value

    assert take() == 0
    t = time.monotonic()
    assert L.start(gave_up.data_ptr(), st) == 0
    assert take() >= 2 and take() == 0                 # one thread's and one warp's; once
    assert 1.5 < time.monotonic() - t < 10
    assert gave_up.cpu().tolist() == [1] + [0] * 31 + [1] * 32
    assert torch.ones(4, device="cuda").sum().item() == 4
