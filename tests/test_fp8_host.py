"""The host side of the FP8 layer operators on a stand-in for the CUDA runtime (no GPU)."""
import ctypes
import os

import pytest

pytest.importorskip("torch")
from bit_exact_emulation_gb300 import build as B
from bit_exact_emulation_gb300 import fp8
from test_ops_host import on_stand_in

OBJECTS = ["fp8_api", "fp8_quant", "fp8_product", "fp8_pair", "fp8_few"]
FP16, BF16, XF32, FP32, E4M3, E5M2 = range(6)
OK, CUDA_ERROR, TIMEOUT = 0, 5, 6
P = 0x10000                                        # a pointer that is never followed
WS = (P, 1 << 50)


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    """The operators' objects as they were built, on the stand-in."""
    objects = [os.path.join(B.HERE, "_build", f + ".o") for f in OBJECTS]
    B.build(force=not all(map(os.path.exists, objects)))
    L = on_stand_in(objects, tmp_path_factory.mktemp("fake"))
    for name, (res, args) in fp8.SYMBOLS.items():
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    L.fake_name.restype = ctypes.c_char_p
    return L


def linear(L, M, N, K, ld=None, out=BF16, acc=0):
    ld, b = ld or K, -(-K // 128)
    return L.mcemu_fp8_linear(M, N, K, E4M3, P, ld, P, b, E4M3, P, ld, P, b, 0, 0, out, acc, P, N, *WS, None)


def grouped(L, T, E, N, K, out=BF16):
    b = -(-K // 128)
    return L.mcemu_fp8_grouped_linear(T, E, N, K, E4M3, P, K, P, b, E5M2, P, K, N * K, P, P, out, P, N, *WS, None)


def wgrad(L, Pc, E, N, K, out=FP32, acc=0):
    return L.mcemu_fp8_grouped_wgrad(Pc, E, N, K, E4M3, P, Pc, P, Pc // 128, E4M3, P, Pc, P, Pc // 128, P, out, acc, P, K, N * K, *WS, None)


# name: (call, the launches that it makes)
CALLS = {
    "rows": (lambda L: L.mcemu_fp8_quantize(BF16, E4M3, 64, 512, P, 512, P, 512, P, 4, 0, 0, 0, 0, 0, 0, None), ["rows_kernel"]),
    "odd rows": (lambda L: L.mcemu_fp8_quantize(FP32, E5M2, 64, 511, P, 511, P, 511, P, 4, 0, 0, 0, 0, 0, 0, None), ["rows_kernel"]),
    "columns": (lambda L: L.mcemu_fp8_quantize(FP16, E4M3, 64, 512, P, 512, P, 512, P, 4, P, 128, P, 1, 0, 0, None), ["columns_kernel"]),
    "columns of groups": (lambda L: L.mcemu_fp8_quantize(BF16, E4M3, 64, 512, P, 512, 0, 0, 0, 0, P, 512, P, 4, 4, P, None), ["columns_kernel"]),
    "columns of no rows": (lambda L: L.mcemu_fp8_quantize(BF16, E4M3, 0, 512, 0, 512, 0, 0, 0, 0, P, 512, P, 4, 4, P, None), ["columns_kernel"]),
    "weight": (lambda L: L.mcemu_fp8_quantize_weight(BF16, E4M3, 3, 64, 512, P, 512, 32768, P, 512, 32768, P, P, 64, 32768, P, None),
               ["weight_kernel"]),
    "few rows": (lambda L: linear(L, 4, 4096, 4096), ["few_kernel"]),
    "few odd rows": (lambda L: linear(L, 4, 4096, 4097), ["align_kernel", "few_kernel"]),
    "many rows": (lambda L: linear(L, 4096, 4096, 4096), ["pair_kernel"]),
    "many odd rows": (lambda L: linear(L, 4096, 4096, 4097, out=FP32, acc=1), ["align_kernel", "pair_kernel"]),
    "nothing to add up": (lambda L: linear(L, 4, 8, 0), ["empty_kernel"]),
    "nothing to add": (lambda L: linear(L, 4, 8, 0, out=FP32, acc=1), []),
    "few rows of experts": (lambda L: grouped(L, 64, 32, 2048, 4096), ["few_kernel"]),
    "many rows of experts": (lambda L: grouped(L, 16384, 16, 4096, 2048), ["pair_kernel"]),
    "experts of odd sizes": (lambda L: grouped(L, 1003, 7, 1000, 1111, FP32), ["align_kernel", None]),
    "weight gradients": (lambda L: wgrad(L, 2048, 8, 512, 512, acc=1), ["pair_kernel"]),
    "weight gradients of no rows": (lambda L: wgrad(L, 0, 8, 512, 512), ["empty_kernel"]),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_launch_that_fails_is_reported(L, name):
    """Whichever launch of a call fails, that call says so, launches nothing on top of it and leaves no
    error to the calls after it."""
    call, kernels = CALLS[name]
    L.fake_reset(-1)
    assert call(L) == OK
    names = [L.fake_name(i).decode() for i in range(L.fake_launches())]
    assert len(names) == len(kernels) and all(k is None or k in n for k, n in zip(kernels, names)), names
    for k in range(len(kernels)):
        L.fake_reset(k)
        assert call(L) == CUDA_ERROR, names[k]
        assert L.fake_launches() == k + 1
        assert L.cudaGetLastError() == 0


def test_products_that_would_not_fit_a_grid_are_refused(L):
    """Tiles are counted in 32 bits."""
    L.fake_reset(-1)
    assert linear(L, 2 ** 31 - 70000, 2 ** 31 - 70000, 16) == 2 and L.fake_launches() == 0
    assert grouped(L, 2 ** 31 - 70000, 1024, 2 ** 31 - 70000, 16) == 2 and L.fake_launches() == 0
    assert wgrad(L, 128, 1024, 2 ** 30, 2 ** 30) == 2 and L.fake_launches() == 0


def test_check_reports_each_wait_that_gave_up_once(L):
    """Of either product's file; also one that gives up on another stream while the call reads."""
    assert L.fake_words() == 2 and L.mcemu_fp8_check(None) == OK
    for i in (0, 1):
        L.fake_raise(i, 0)
        assert L.mcemu_fp8_check(None) == TIMEOUT
        assert L.mcemu_fp8_check(None) == OK
        L.fake_raise(i, 1)                         # grows after the first copy
        assert TIMEOUT in (L.mcemu_fp8_check(None), L.mcemu_fp8_check(None))
        assert L.mcemu_fp8_check(None) == OK


@pytest.mark.parametrize("N,K,ldd,ldx", [(1, 32, 257, 256), (32, 1, 256, 257), (1, 1, 999, 257)])
def test_single_columns_of_a_weight_gradient_are_read_in_place(L, N, K, ldd, ldx):
    """A single row of an operand has no next one: its pointer decides, as in the other products.  Where that is
    odd, the row is copied."""
    def call(d, x, ws=0, nws=0):
        L.fake_reset(-1)
        st = L.mcemu_fp8_grouped_wgrad(256, 3, N, K, E4M3, d, ldd, P, 2, E4M3, x, ldx, P, 2, P, FP32, 0, P, K, N * K, ws, nws, None)
        return st, [L.fake_name(i).decode() for i in range(L.fake_launches())]

    assert L.mcemu_fp8_grouped_wgrad_workspace(256, 3, N, K, 1, 1) == 0
    st, names = call(P, P)
    assert st == OK and len(names) == 1 and "pair_kernel" in names[0]
    assert call(P + 1, P) == (7, [])
    st, names = call(P + 1, P, P, L.mcemu_fp8_grouped_wgrad_workspace(256, 3, N, K, 0, 1))
    assert st == OK and len(names) == 2 and "align_kernel" in names[0]
