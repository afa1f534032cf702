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


# Pairs of CTAs: rows of b to a tile, operands exchanged or not.  With fewer tiles than pairs and with several to each; sums of
# one run of 1024 along k and of more.
LINEAR_PAIRS = [(104, 101, 2409, 128, True), (300, 700, 3000, 128, True), (2405, 924, 4534, 128, True), (3328, 1400, 4742, 128, False),
                (2738, 1313, 1346, 224, False), (918, 4147, 1390, 224, False), (4096, 4099, 1300, 224, False), (562, 4019, 802, 224, True),
                (2845, 2490, 412, 224, True), (2300, 2100, 2400, 224, True)]
# Of grouped rows: offsets, which leave rows outside, T, N, K.
GROUPED_PAIRS = [([1, 120, 120, 299], 300, 700, 3000, 128, True), ([0, 5, 60, 61, 61, 200, 260, 261, 400, 426], 426, 2173, 211, 128, True),
                 ([3, 2200, 2201, 6400, 8471], 8471, 269, 1543, 224, False), ([0, 900, 900, 901, 1300, 1301, 1700, 2100, 2300, 2450], 2458, 1037, 1392, 224, False),
                 ([7, 1000, 1400, 1400, 2700, 2704, 3900, 4500, 4660], 4672, 408, 791, 224, True),
                 ([3, 1000, 1001, 1001, 3303, 5000, 8991], 9000, 2064, 1300, 224, True), ([0, 700, 2000, 2000, 4099, 7777, 9000], 9000, 4099, 1100, 224, True)]
# Weight gradients: T, groups, N, K.
WGRAD_PAIRS = [(231, 9, 1146, 101, 128, False), (328, 4, 187, 2432, 128, False), (107, 2, 110, 114, 128, True), (107, 6, 129, 1563, 128, True),
               (5018, 5, 237, 1935, 224, False), (4978, 7, 2495, 273, 224, False), (2306, 5, 129, 1964, 224, True), (247, 9, 799, 874, 224, True)]
# Results that pairs of this form give in 16 bits alone: in fp32 a few rows' form takes the call.
SHORT = (3328, 1400, 4742)


@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
def test_pairs_take_the_sizes_of_their_tests(L, out):
    for M, N, K, tile, turned in LINEAR_PAIRS:
        if (M, N, K) != SHORT or out != "fp32":
            assert linear(L, M, N, K, out)[:3] == ("pair", tile, turned), (M, N, K)
    for offsets, T, N, K, tile, turned in GROUPED_PAIRS:
        assert grouped(L, T, len(offsets) - 1, N, K, out)[:3] == ("pair", tile, turned), (offsets, N, K)
    for T, E, N, K, tile, turned in WGRAD_PAIRS:
        L.fake_reset(-1)
        C = fp8.columns(T, E)
        got = last(L, L.mcemu_fp8_grouped_wgrad(C, E, N, K, E4M3, P, C, P, C // 128, E4M3, P, C, P, C // 128, P, FMT[out], 0, P, K, N * K, *WS, None))
        assert got[:3] == ("pair", tile, turned), (T, E, N, K)


# Products whose sums are held against the emulated unit's: M, N, K, kernel, tile, CTAs that share K.
SUMS = [(7, 300, 9000, "few", 16, 8), (20, 200, 3000, "few", 32, 6), (40, 200, 5000, "few", 64, 7), (600, 200, 2100, "few", 128, 1),
        (104, 101, 2409, "pair", 128, 1), (300, 700, 3000, "pair", 128, 1), (2738, 1313, 1346, "pair", 224, 1), (2300, 2100, 2400, "pair", 224, 1)]


@pytest.mark.parametrize("M,N,K,kernel,tile,parts", SUMS)
def test_sums_are_cut_as_their_test_says(L, M, N, K, kernel, tile, parts):
    got = linear(L, M, N, K, "fp32")
    assert got[:2] == (kernel, tile) and got[3] == parts


def test_the_form_goes_by_more_than_sizes(L):
    """By the width of the results and by groups, as the header says."""
    M, N, K = SHORT
    assert linear(L, M, N, K, "bf16")[0] == linear(L, M, N, K, "fp16")[0] == "pair" and linear(L, M, N, K, "fp32")[0] == "few"
    assert linear(L, 300, 700, 3000)[0] == "pair" and grouped(L, 300, 9, 700, 3000)[0] == "few"
    for out in ("bf16", "fp32"):                     # not by strides, addresses or what y holds
        forms = {linear(L, 300, 700, 3000, out, ldy=ldy)[:4] for ldy in (700, 701, 704)}
        assert len(forms) == 1
    assert linear(L, 300, 700, 3000, "fp32", acc=1) == linear(L, 300, 700, 3000, "fp32")
