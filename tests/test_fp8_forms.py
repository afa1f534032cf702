"""Which kernel an FP8 product runs, and how it is cut, on a stand-in for the CUDA runtime (no GPU): the sizes that the tests
on the GPU take for a path of a kernel do take it."""
import ctypes
import os
import re

import pytest

pytest.importorskip("torch")
from bit_exact_emulation_gb300 import build as B
from bit_exact_emulation_gb300 import fp8
from test_fp8_host import E4M3, OBJECTS, OK, P, WS
from test_ops_host import on_stand_in

FMT = {"fp16": 0, "bf16": 1, "fp32": 3}


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    objects = [os.path.join(B.HERE, "_build", f + ".o") for f in OBJECTS]
    B.build(force=not all(map(os.path.exists, objects)))
    L = on_stand_in(objects, tmp_path_factory.mktemp("fake"))
    for name, (res, args) in fp8.SYMBOLS.items():
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    L.fake_name.restype = ctypes.c_char_p
    return L


def blocks(n):
    return -(-n // 128)


def last(L, status):
    """(kernel, tile, turned, CTAs that share K, how many such clusters) of the launch that multiplies."""
    assert status == OK
    i = L.fake_launches() - 1
    name, parts = L.fake_name(i).decode(), L.fake_cluster(i)
    kernel, tile = re.search(r"(few|pair)_kernelI.*?Li(\d+)E", name).groups()
    return kernel, int(tile), "Lb1E" in name, parts, L.fake_blocks(i) // parts


def linear(L, M, N, K, out="bf16", acc=0, ldy=0):
    L.fake_reset(-1)
    ld, b = blocks(K) * 128, blocks(K)
    return last(L, L.mcemu_fp8_linear(M, N, K, E4M3, P, ld, P, b, E4M3, P, ld, P, b, 0, 0, FMT[out], acc, P, ldy or N, *WS, None))


def grouped(L, T, E, N, K, out="bf16"):
    L.fake_reset(-1)
    ld, b = blocks(K) * 128, blocks(K)
    return last(L, L.mcemu_fp8_grouped_linear(T, E, N, K, E4M3, P, ld, P, b, E4M3, P, ld, N * ld, P, P, FMT[out], P, N, *WS, None))


# Clusters that share K and take several units: rows (or those of each group), N, K, tokens to a tile, CTAs that share K.
# Groups' counts change from one to the next, and with them the tokens that a CTA joins; some are empty.
JOINS = [
    (1, 20062, 1689, 16, 2), (4, 19638, 1698, 16, 2), (5, 9785, 2215, 16, 3), (2, 11964, 4586, 16, 4), (9, 6081, 5649, 16, 5),
    (19, 19611, 2551, 32, 2), (18, 10357, 2974, 32, 3), (20, 12425, 7521, 32, 4), (20, 6624, 6919, 32, 5),
    ([6, 5, 0, 2, 5, 4, 4, 0, 3, 6, 0, 0, 1, 1, 5, 3, 0, 2, 4, 4, 6, 4, 6, 1], 823, 1677, 16, 2),
    ([0, 17, 20, 0, 0, 7, 0, 19, 9, 11, 15, 0, 0, 19, 10, 4], 521, 2206, 16, 3),
    ([3, 4, 14, 2, 6, 7, 1, 1, 8, 4], 1199, 4503, 16, 4),
    ([10, 5, 7, 0, 7, 0, 18, 17, 0, 7, 0, 5, 12, 0, 12, 0, 18, 0, 19, 6, 6, 6, 19, 0], 200, 6330, 16, 5),
    ([31, 0, 19, 29, 1, 27, 24, 3, 15, 13, 10], 1676, 2191, 32, 2),
    ([10, 0, 10, 13, 17, 9, 14, 13, 14, 0, 12, 16, 20, 14, 17, 17, 20, 1, 5, 17, 5, 16, 12], 388, 2567, 32, 3),
    ([3, 29, 9, 10, 23, 23, 24, 2, 6, 0, 0, 6, 0, 24, 32, 28, 0, 16, 18, 18, 8, 12, 2, 30], 403, 5995, 32, 4),
    ([16, 12, 4, 13, 1, 10, 11, 18, 20, 4, 6, 8, 12, 5, 6, 20, 10, 0], 281, 5634, 32, 5)]


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,N,K,tile,parts", JOINS, ids=str)
def test_joins_take_several_units_to_a_cluster(L, rows, N, K, tile, parts, out):
    counts = [rows] if isinstance(rows, int) else rows
    got = linear(L, rows, N, K, out) if isinstance(rows, int) else grouped(L, sum(counts), len(counts), N, K, out)
    assert got[:2] == ("few", tile) and got[3] == parts
    assert sum(-(-n // tile) for n in counts) * blocks(N) > got[4]
