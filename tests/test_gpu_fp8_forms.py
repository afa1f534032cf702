"""The FP8 products on the GPU in each form that they take, at sizes that take it (tests/test_fp8_forms.py holds them to
that), against plain implementations in 64 bits."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from test_fp8_forms import JOINS  # noqa: E402
from test_gpu_fp8 import DT, F, blocks, exps, gen, of_rows, of_tiles, raw, rounded, same, strided, whole  # noqa: E402,F401


def offsets_of(counts):
    return torch.tensor([0, *counts], device="cuda").cumsum(0).int()


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,N,K,tile,parts", JOINS, ids=str)
def test_joins_of_several_units_to_a_cluster(F, rows, N, K, tile, parts, out):
    """Every sum is different from its neighbours', and the same call gives the same bits."""
    counts = [rows] if isinstance(rows, int) else rows
    T, E, g = sum(counts), len(counts), gen(N + K)
    x, w = (strided(whole(g, shape, "e4m3"), -K % 16) for shape in ((T, K), (E, N, K)))
    ex, ew = exps(g, T, blocks(K)), exps(g, E, blocks(N), blocks(K))
    o = offsets_of(counts)
    call = ((lambda: F.linear(x, ex, w[0], ew[0], out=out)) if isinstance(rows, int) else
            (lambda: F.grouped_linear(x, ex, w, ew, o, out=out)))
    got = [call() for _ in range(6)]
    xv, at = of_rows(x, ex), o.tolist()
    want = torch.cat([rounded(xv[a:b] @ of_tiles(w[i], ew[i]).T, out) for i, (a, b) in enumerate(zip(at, at[1:]))])
    for y in got:
        assert same(y, want)
    F.check()


@pytest.mark.parametrize("N,K", [(1, 300), (300, 1), (1, 1)])
def test_single_columns_of_a_weight_gradient_are_read_in_place(F, N, K):
    """Of an operand of one row the leading dimension is that of no next row: any will do, without a workspace."""
    T, g = 300, gen(N + K)
    o = offsets_of([100, 0, 200])
    dy, x = (torch.randint(-2, 3, (T, n), generator=g, device="cuda").bfloat16() for n in (N, K))
    (_, _, dt, edt), (_, _, xt, ext) = (F.quantize(t, rows=False, columns=True, offsets=o) for t in (dy, x))
    P, dW = dt.shape[1], torch.full((3, N, K), 7.0, device="cuda")
    ld = lambda t: P + 1 if len(t) == 1 else P
    st = F.lib().mcemu_fp8_grouped_wgrad(P, 3, N, K, F.FMT["e4m3"], dt.data_ptr(), ld(dt), edt.data_ptr(), P // 128, F.FMT["e4m3"],
                                         xt.data_ptr(), ld(xt), ext.data_ptr(), P // 128, o.data_ptr(), F.FMT["fp32"], 0, dW.data_ptr(), K,
                                         N * K, None, 0, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    at = o.tolist()
    assert same(dW, rounded(torch.stack([dy[a:b].double().T @ x[a:b].double() for a, b in zip(at, at[1:])]), "fp32"))
    F.check()


def test_a_group_without_rows_keeps_what_it_adds_to(F):
    """To the last bit, negative zeros, subnormal numbers and NaNs' payloads too; in rows that the copy engine writes and in others."""
    N, K, g = 264, 300, gen(11)
    for lead, offsets in ((0, [0, 0, 200, 200, 200]), (0, [200, 200, 200, 200, 200]), (1, [0, 0, 77, 77, 200]), (0, [0, 130, 5, 130, 200])):
        o = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        dy, x = (torch.randint(-2, 3, (200, n), generator=g, device="cuda").bfloat16() for n in (N, K))
        (_, _, dt, edt), (_, _, xt, ext) = (F.quantize(t, rows=False, columns=True, offsets=o) for t in (dy, x))
        bits = torch.tensor([-2 ** 31, 1, -2 ** 31 + 5, 0x007FFFFF, 0x7FC00123, 0x7F800000, 0, 0x3F800000], dtype=torch.int32, device="cuda")
        was = bits[torch.randint(0, 8, (4, N, K), generator=g, device="cuda")].view(torch.float32)
        dW = strided(was, 0, lead)
        F.grouped_wgrad(dt, edt, xt, ext, o, dW=dW, accumulate=True)
        at = [max(offsets[:i + 1]) for i in range(5)]
        for i, (a, b) in enumerate(zip(at, at[1:])):
            if a == b:
                assert torch.equal(dW[i].contiguous().view(torch.int32), was[i].view(torch.int32)), (offsets, i)
    F.check()


# Rows of y that begin on 16-byte boundaries and end between two, in products by pairs of CTAs and by single ones.
@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,N,K", [(104, 97, 2409), (104, 101, 2409), (104, 103, 2409), (2738, 1313, 1346), (918, 4147, 1390), (562, 4019, 802),
                                   (5, 203, 700), (300, 230, 400)])
def test_nothing_is_written_beside_a_row_that_ends_between_boundaries(F, M, N, K, out):
    g = gen(M + N)
    x, w = (strided(whole(g, (r, K), "e4m3"), -K % 16) for r in (M, N))
    ex, ew = exps(g, M, blocks(K)), exps(g, N, blocks(K))
    product = of_rows(x, ex) @ of_rows(w, ew).T
    # subnormal numbers beside the rows, which even a zero added by the copy engine would change
    buf = torch.full((M + 2, -(-N // 8) * 8 + 8), 2.0 ** -24 if out == "fp16" else 2.0 ** -130, device="cuda").to(DT[out])
    was = buf.clone()
    y = buf[1:M + 1, :N]
    for accumulate in (False, True) if out == "fp32" else (False,):
        y.fill_(3.0)
        F.linear(x, ex, w, ew, out=out, y=y, accumulate=accumulate)
        assert same(y.contiguous(), rounded(product + 3.0 * accumulate, out))
        y.copy_(was[1:M + 1, :N])
        assert same(buf, was)
    offsets, E = [0, M // 3, M // 3, M], 3
    o = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    w = strided(torch.stack([raw(w)] * E).view(w.dtype), -K % 16)
    tiles = exps(g, E, blocks(N), blocks(K))
    F.grouped_linear(x, ex, w, tiles, o, out=out, y=y)
    for i, (a, b) in enumerate(zip(offsets, offsets[1:])):
        assert same(y[a:b].contiguous(), rounded(of_rows(x, ex)[a:b] @ of_tiles(w[i], tiles[i]).T, out))
    y.copy_(was[1:M + 1, :N])
    assert same(buf, was)
    F.check()


@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,N,K", [(200, 107, 113), (300, 129, 1563), (2000, 799, 874), (900, 264, 1)])
def test_nothing_is_written_beside_the_rows_of_a_weight_gradient(F, T, N, K, out):
    g, offsets = gen(T + N), [0, T // 2, T // 2, T - 7, T]
    o = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    dy, x = (torch.randint(-2, 3, (T, n), generator=g, device="cuda").bfloat16() for n in (N, K))
    (_, _, dt, edt), (_, _, xt, ext) = (F.quantize(t, rows=False, columns=True, offsets=o) for t in (dy, x))
    want = torch.stack([dy[a:b].double().T @ x[a:b].double() for a, b in zip(offsets, offsets[1:])])
    buf = torch.full((4, N + 2, -(-K // 8) * 8 + 8), 2.0 ** -24 if out == "fp16" else 2.0 ** -130, device="cuda").to(DT[out])
    was = buf.clone()
    dW = buf[:, 1:N + 1, :K]
    for accumulate in (False, True) if out == "fp32" else (False,):
        dW.fill_(3.0)
        F.grouped_wgrad(dt, edt, xt, ext, o, out=out, dW=dW, accumulate=accumulate)
        assert same(dW.contiguous(), rounded(want + 3.0 * accumulate, out))
        dW.copy_(was[:, 1:N + 1, :K])
        assert same(buf, was)
    F.check()
