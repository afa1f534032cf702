"""The host side of the 8-bit layer operators on a stand-in for the CUDA runtime (no GPU)."""
import ctypes
import os
import subprocess

import pytest

pytest.importorskip("torch")
from bit_exact_emulation_gb300 import build as B
from bit_exact_emulation_gb300 import ops

HERE = os.path.dirname(os.path.abspath(__file__))
OBJECTS = ["ops_api", "rmsnorm", "rmsnorm_grad", "rmsnorm_grad_single", "act8", "int8_linear", "act8_wgrad"]
FP16, BF16, XF32, FP32, E4M3, E5M2, INT8, UINT8, INT32 = range(9)
OK, CUDA_ERROR, TIMEOUT = 0, 5, 6
P = 0x10000                                        # a pointer that is never followed


def on_stand_in(objects, folder):
    so = str(folder / "libfake.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(B._nvcc()))), "include")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-Wl,-Bsymbolic", "-I", cuda, os.path.join(HERE, "fake_cudart.cpp"),
                    *objects, "-o", so], check=True)
    return ctypes.CDLL(so)


@pytest.fixture(scope="module")
def F(tmp_path_factory):
    """The operators' objects as they were built, on the stand-in."""
    objects = [os.path.join(B.HERE, "_build", f + ".o") for f in OBJECTS]
    B.build(force=not all(map(os.path.exists, objects)))
    L = on_stand_in(objects, tmp_path_factory.mktemp("fake"))
    for name, (res, args) in ops.SYMBOLS.items():
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    L.fake_name.restype = ctypes.c_char_p
    return L


WS = (P, 1 << 50)
CALLS = {
    "norm": lambda L: L.mcemu_rmsnorm(BF16, BF16, INT8, 64, 512, P, 512, 0, 0, P, 1e-5, 0, 0, P, 512, P, P, None),
    "norm of odd rows": lambda L: L.mcemu_rmsnorm(BF16, BF16, INT8, 64, 511, P, 511, 0, 0, P, 1e-5, 0, 0, P, 511, P, P, None),
    "norm of many odd rows": lambda L: L.mcemu_rmsnorm(BF16, BF16, INT8, 640, 511, P, 511, 0, 0, P, 1e-5, 0, 0, P, 511, P, P, None),
    "norm of long rows": lambda L: L.mcemu_rmsnorm(BF16, BF16, INT8, 6, 40001, P, 40001, 0, 0, P, 1e-5, 0, 0, P, 40001, P, P, None),
    "norm gradients": lambda L: L.mcemu_rmsnorm_backward(BF16, BF16, 64, 512, P, 512, 0, 0, P, 512, 0, 0, 0, 0, P, P, P, 512, P, *WS, None),
    "norm gradients of odd rows": lambda L: L.mcemu_rmsnorm_backward(BF16, BF16, 64, 511, P, 511, 0, 0, P, 511, 0, 0, 0, 0, P, P, P, 511, P,
                                                                     *WS, None),
    "norm gradients of long rows": lambda L: L.mcemu_rmsnorm_backward(BF16, BF16, 6, 9001, P, 9001, 0, 0, P, 9001, 0, 0, 0, 0, P, P, P, 9001,
                                                                      P, *WS, None),
    "compress": lambda L: L.mcemu_act8_compress(BF16, 64, 512, P, 512, P, 512, P, 4, None),
    "compress odd rows": lambda L: L.mcemu_act8_compress(BF16, 64, 511, P, 511, P, 511, P, 4, None),
    "expand": lambda L: L.mcemu_act8_expand(BF16, 64, 512, P, 512, P, 4, P, 512, None),
    "product, few tokens": lambda L: L.mcemu_int8_linear(4, 512, 512, P, 512, P, P, 512, P, None, BF16, P, 512, None, 0, None),
    "product, batch": lambda L: L.mcemu_int8_linear(64, 8192, 512, P, 512, P, P, 512, P, None, BF16, P, 8192, None, 0, None),
    "product, panels": lambda L: L.mcemu_int8_linear(1300, 1800, 520, P, 520, P, P, 520, P, None, BF16, P, 1800, *WS, None),
    "weight gradient": lambda L: L.mcemu_act8_wgrad(512, 512, 512, P, 512, P, 512, P, 4, FP32, 0, P, 512, *WS, None),
    "weight gradient, shared tiles": lambda L: L.mcemu_act8_wgrad(5001, 520, 1000, P, 520, P, 1000, P, 8, BF16, 0, P, 1000, *WS, None),
    "weight gradient, odd rows": lambda L: L.mcemu_act8_wgrad(512, 511, 512, P, 511, P, 512, P, 4, FP32, 0, P, 512, *WS, None),
    "weight gradient, no tokens": lambda L: L.mcemu_act8_wgrad(0, 512, 512, P, 512, P, 512, P, 4, FP32, 0, P, 512, *WS, None),
}
LAUNCHES = {"norm gradients": 2, "norm gradients of odd rows": 2, "norm gradients of long rows": 3, "product, panels": 2,
            "weight gradient": 2, "weight gradient, shared tiles": 3, "weight gradient, odd rows": 3}


@pytest.mark.parametrize("name", CALLS)
def test_a_launch_that_fails_is_reported(F, name):
    """Whichever launch of a call fails, that call says so, launches nothing on top of it and leaves no
    error to the calls after it."""
    F.fake_reset(-1)
    assert CALLS[name](F) == OK
    n = F.fake_launches()
    assert n == LAUNCHES.get(name, 1), [F.fake_name(i) for i in range(n)]
    for k in range(n):
        F.fake_reset(k)
        assert CALLS[name](F) == CUDA_ERROR, (k, F.fake_name(k))
        assert F.fake_launches() == k + 1
        assert F.cudaGetLastError() == 0


def test_check_reports_each_wait_that_gave_up_once(F):
    """Of either product's file; also one that gives up on another stream while the call reads."""
    assert F.fake_words() == 2 and F.mcemu_ops_check(None) == OK
    for i in (0, 1):
        F.fake_raise(i, 0)
        assert F.mcemu_ops_check(None) == TIMEOUT
        assert F.mcemu_ops_check(None) == OK
        F.fake_raise(i, 1)                         # grows after the first copy
        assert TIMEOUT in (F.mcemu_ops_check(None), F.mcemu_ops_check(None))
        assert F.mcemu_ops_check(None) == OK


def test_each_file_has_a_flag_of_its_own(tmp_path):
    """Without inlining too, where one copy of a function of two files would serve both."""
    objects = []
    for name in "ab":
        src, obj = tmp_path / f"{name}.cu", tmp_path / f"{name}.o"
        src.write_text(f'#include "{B.CSRC}/tc.cuh"\n'
                       f'extern "C" int take_{name}(unsigned *got) {{ return mcemu::tc::take_timeouts(nullptr, got); }}\n'
                       "static __global__ void user(uint32_t bar, bool dead) { mcemu::tc::mbar_wait(bar, 0, dead); }\n")
        subprocess.run([B._nvcc(), *B.ARCH, "-O0", "-std=c++17", "-Xcompiler", "-fPIC", "-c", str(src), "-o", str(obj)], check=True)
        objects.append(str(obj))
    L = on_stand_in(objects, tmp_path)
    got = ctypes.c_uint()

    def take(f):
        assert f(ctypes.byref(got)) == OK
        return got.value

    assert L.fake_words() == 2
    L.fake_raise(0, 0)
    seen = [take(L.take_a), take(L.take_b)]
    L.fake_raise(1, 0)
    assert [seen, [take(L.take_a), take(L.take_b)]] in ([[1, 0], [0, 1]], [[0, 1], [1, 0]])
