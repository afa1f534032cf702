"""The FP8 products on the GPU in each form that they take, at sizes that take it (tests/test_fp8_forms.py holds them to
that), against plain implementations in 64 bits."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from test_fp8_forms import GROUPED_PAIRS, JOINS, LINEAR_PAIRS, SHORT, SUMS, WGRAD_PAIRS  # noqa: E402
from test_gpu_fp8 import CODE, DT, F, blocks, columns_host, exps, gen, of_rows, of_tiles, raw, rounded, rows_host, same  # noqa: E402,F401
from test_gpu_fp8 import strided, values, whole  # noqa: E402


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


# Rows that the copy engine can write, wholly or not, and rows that it cannot.
LAYOUTS = [("bf16", 0, 0), ("bf16", 3, 1), ("fp16", -1, 8), ("fp32", 5, 3), ("fp32", -1, 4)]


def padding(cols, pad):
    return -cols % 16 if pad < 0 else pad


@pytest.mark.parametrize("out,pad,lead", LAYOUTS)
@pytest.mark.parametrize("M,N,K,tile,turned", LINEAR_PAIRS)
def test_pairs(F, M, N, K, tile, turned, out, pad, lead):
    """With a bias at any address, and added to what is there."""
    if (M, N, K) == SHORT and out == "fp32":
        pytest.skip("another form's call")
    g, pad = gen(M + N + K), padding(N, pad)
    x, w = strided(whole(g, (M, K), "e4m3"), -K % 16), strided(whole(g, (N, K), "e5m2"), -K % 16)
    tiles = (M + lead) % 2 == 0
    ex, ew = exps(g, M, blocks(K)), exps(g, blocks(N) if tiles else N, blocks(K))
    bias = torch.randint(-8, 9, (N + 1,), generator=g, device="cuda").float()[lead % 2:][:N]
    product = of_rows(x, ex) @ (of_tiles(w, ew) if tiles else of_rows(w, ew)).T
    buf = torch.full((lead + M * (N + pad) + 16,), 7.0, dtype=DT[out], device="cuda")
    y = buf[lead:lead + M * (N + pad)].view(M, N + pad)[:, :N]
    assert F.linear(x, ex, w, ew, bias=bias, out=out, y=y).data_ptr() == y.data_ptr()
    assert same(y.contiguous(), rounded(product + bias.double(), out))
    assert same(F.linear(x, ex, w, ew, out=out), rounded(product, out))
    if out == "fp32":
        before = torch.randint(-9, 10, (M, N), generator=g, device="cuda").float()
        y.copy_(before)
        F.linear(x, ex, w, ew, out=out, y=y, accumulate=True)
        assert same(y.contiguous(), rounded(product + before.double(), out))
    y.fill_(7.0)
    assert torch.all(buf == 7.0)                     # nothing beside the rows was touched
    F.check()


@pytest.mark.parametrize("out,pad,lead", LAYOUTS)
@pytest.mark.parametrize("offsets,T,N,K,tile,turned", GROUPED_PAIRS, ids=str)
def test_pairs_of_groups(F, offsets, T, N, K, tile, turned, out, pad, lead):
    """Rows outside all groups, and what lies beside the rows, stay as they were."""
    E, g, pad = len(offsets) - 1, gen(T + N + K), padding(N, pad)
    x, w = strided(whole(g, (T, K), "e5m2"), -K % 16), strided(whole(g, (E, N, K), "e4m3"), -K % 16)
    ex, ew = exps(g, T, blocks(K)), exps(g, E, blocks(N), blocks(K))
    buf = torch.full((lead + T * (N + pad) + 16,), 7.0, dtype=DT[out], device="cuda")
    y = buf[lead:lead + T * (N + pad)].view(T, N + pad)[:, :N]
    F.grouped_linear(x, ex, w, ew, torch.tensor(offsets, dtype=torch.int32, device="cuda"), out=out, y=y)
    xv = of_rows(x, ex)
    for i, (a, b) in enumerate(zip(offsets, offsets[1:])):
        assert same(y[a:b].contiguous(), rounded(xv[a:b] @ of_tiles(w[i], ew[i]).T, out)), i
    y[offsets[0]:offsets[-1]] = 7.0
    assert torch.all(buf == 7.0)
    F.check()


@pytest.mark.parametrize("out,pad,lead", LAYOUTS)
@pytest.mark.parametrize("T,E,N,K,tile,turned", WGRAD_PAIRS)
def test_pairs_of_weight_gradients(F, T, E, N, K, tile, turned, out, pad, lead):
    g, pad = gen(T + N + K), padding(K, pad)
    ends = torch.randint(0, T + 1, (E - 1,), generator=g, device="cuda").sort().values
    o = torch.cat([ends.new_zeros(1), ends, ends.new_full((1,), T - 1)]).cummax(0).values.int()
    o[E // 2] = o[E // 2 + 1]                        # one without rows
    dy, x = (torch.randint(-2, 3, (T, n), generator=g, device="cuda").bfloat16() for n in (N, K))
    (_, _, dt, edt), (_, _, xt, ext) = (F.quantize(t, rows=False, columns=True, offsets=o, out=f) for t, f in ((dy, "e5m2"), (x, "e4m3")))
    buf = torch.full((lead + E * N * (K + pad) + 16,), 7.0, dtype=DT[out], device="cuda")
    dW, at = buf[lead:lead + E * N * (K + pad)].view(E, N, K + pad)[..., :K], o.tolist()
    want = torch.stack([dy[a:b].double().T @ x[a:b].double() for a, b in zip(at, at[1:])])
    F.grouped_wgrad(dt, edt, xt, ext, o, out=out, dW=dW)
    assert same(dW.contiguous(), rounded(want, out))
    if out == "fp32":
        F.grouped_wgrad(dt, edt, xt, ext, o, dW=dW, accumulate=True)
        assert same(dW.contiguous(), rounded(2 * want, out))
    dW.fill_(7.0)
    assert torch.all(buf == 7.0)
    F.check()


@pytest.mark.parametrize("pad,lead", [(1, 0), (-1, 16), (3, 5)])
@pytest.mark.parametrize("M,N,K,tile,turned", [(20, 200, 3001, 32, False), LINEAR_PAIRS[0], LINEAR_PAIRS[4], LINEAR_PAIRS[7]])
def test_operands_in_any_layout(F, M, N, K, tile, turned, pad, lead):
    """What lies beside rows and exponents is not finite, and in no sum."""
    g = gen(M + pad)
    x, w = whole(g, (M, K), "e4m3"), whole(g, (N, K), "e4m3")
    ex, ew = exps(g, M, blocks(K)), exps(g, N, blocks(K))

    def inside(t, fill, pad):
        n, cols = t.shape
        buf = torch.full((lead + n * (cols + pad) + 16,), fill, dtype=torch.uint8, device="cuda")
        v = buf[lead:lead + n * (cols + pad)].view(n, cols + pad)[:, :cols]
        v.copy_(raw(t))
        return v.view(t.dtype)

    y = F.linear(inside(x, 0x7F, padding(K, pad)), inside(ex, 0x80, abs(pad)), inside(w, 0x7F, padding(K, pad)), inside(ew, 0x80, abs(pad)))
    assert same(y, rounded(of_rows(x, ex) @ of_rows(w, ew).T, "bf16"))
    F.check()


@pytest.mark.parametrize("M,N,K,tile,turned", [LINEAR_PAIRS[1], LINEAR_PAIRS[4], LINEAR_PAIRS[7]])
def test_pairs_keep_what_is_not_finite_where_it_is(F, M, N, K, tile, turned):
    """A block, a row or a code that is not finite makes the sums that it belongs to so, and no other."""
    g = gen(M)
    x, w = strided(whole(g, (M, K), "e5m2"), -K % 16), strided(whole(g, (N, K), "e4m3"), -K % 16)
    ex, ew = exps(g, M, blocks(K)), exps(g, blocks(N), blocks(K))
    plain = F.linear(x, ex, w, ew, out="fp32")
    ex2, ew2 = ex.clone(), ew.clone()
    ex2[1, 3], ew2[2, blocks(K) - 1] = F.NAN, F.NAN
    y = F.linear(x, ex2, w, ew2, out="fp32")
    rows, cols = torch.arange(M, device="cuda") != 1, (torch.arange(N, device="cuda") // 128) != 2
    assert torch.isnan(y[1]).all() and torch.isnan(y[:, ~cols]).all()
    assert torch.equal(y[rows][:, cols], plain[rows][:, cols])
    x.view(torch.uint8)[M - 1, K - 1] = 0x7C         # infinity in E5M2, in the last block's last place
    x.view(torch.uint8)[3, 0] = 0x7E                 # NaN
    y = F.linear(x, ex, w, ew, out="fp32")
    assert not torch.isfinite(y[M - 1]).any() and torch.isnan(y[3]).all()
    rows = (torch.arange(M, device="cuda") != 3) & (torch.arange(M, device="cuda") != M - 1)
    assert torch.equal(y[rows], plain[rows])


@pytest.mark.parametrize("M,N,K,tile,turned", [LINEAR_PAIRS[1], LINEAR_PAIRS[4], LINEAR_PAIRS[7]])
def test_pairs_of_exponents_of_any_size(F, M, N, K, tile, turned):
    """Scales from 2^-127 to 2^127, sums down to subnormal numbers; what fp32 does not hold is infinite.  One block of
    K has numbers, any of them; the others zeros with exponents of any size."""
    g = gen(N)
    for n, (a, b) in enumerate([(-127, 127), (127, -127), (-60, -66), (-100, -27), (-70, -70), (-127, -20), (60, 60), (100, 27)]):
        k = (5 * n + 2) % (K // 128)
        (x, ex), (w, ew) = ((torch.zeros(r, blocks(K) * 128, device="cuda"), torch.randint(-127, 128, (r, blocks(K)), generator=g, device="cuda").to(torch.int8))
                            for r in (M, N))
        x[:, 128 * k:128 * k + 128] = w[:, 128 * k:128 * k + 128] = 1
        ex[:, k], ew[:, k] = a, b
        y = F.linear(x.to(CODE["e4m3"])[:, :K], ex, w.to(CODE["e4m3"])[:, :K], ew, out="fp32")
        assert torch.all(y == float("inf") if a + b + 7 > 127 else y == 2.0 ** (a + b + 7)), (a, b)


@pytest.mark.parametrize("fx,fw", [("e4m3", "e4m3"), ("e5m2", "e4m3")])
@pytest.mark.parametrize("M,N,K,kernel,tile,parts", SUMS)
def test_sums_are_the_emulated_units_of_one_cut(F, fx, fw, M, N, K, kernel, tile, parts):
    """Bit for bit, random codes, in the one way that the call's form adds up: runs of 512 along k in each CTA's share of
    the blocks, the CTAs' sums in their order; or runs of 1024.  Of large products the first and last rows and columns."""
    from bit_exact_emulation_gb300 import binding
    g = gen(M + K)
    x, w = (torch.randint(0, 256, (r, blocks(K) * 128), generator=g, device="cuda").to(torch.uint8).view(CODE[f]) for r, f in ((M, fx), (N, fw)))
    fix = lambda t: torch.where(torch.isfinite(t.float()), raw(t), torch.full_like(raw(t), 0x31)).view(t.dtype)[:, :K]
    x, w = fix(x), fix(w)
    zero = lambda r: torch.zeros(r, blocks(K), dtype=torch.int8, device="cuda")
    y = F.linear(x, zero(M), w, zero(N), out="fp32")
    some = lambda n: torch.arange(n, device="cuda") if n <= 700 else torch.cat([torch.arange(260, device="cuda"), torch.arange(n - 200, n, device="cuda")])
    r, c = some(M), some(N)
    x, w, C = x.view(torch.uint8)[r].view(x.dtype), w.view(torch.uint8)[c].view(w.dtype), torch.zeros(len(r), len(c), dtype=torch.int32, device="cuda")
    desc = binding.preset_desc("b200_fp8")
    desc.fmt_a, desc.fmt_b = binding.FMT[fx], binding.FMT[fw]
    unit = binding.Model(desc)

    def run(a, b):                                   # of blocks a to b - 1; the unit takes 32 of k at a time
        k = slice(128 * a, min(K, 128 * b))
        pad = lambda t: torch.nn.functional.pad(raw(t[:, k]), (0, -(k.stop - k.start) % 32)).view(t.dtype)
        return binding.tile_gemm(unit, binding.tile(0, 16, 16, 32, 8), pad(x), pad(w), C).view(torch.float32)

    length, per = (4, -(-blocks(K) // parts)) if kernel == "few" else (8, blocks(K))
    total = torch.zeros(C.shape, device="cuda")
    for a in range(0, blocks(K), per):
        part = torch.zeros(C.shape, device="cuda")
        for b in range(a, min(a + per, blocks(K)), length):
            part = part + run(b, min(b + length, a + per, blocks(K)))
        total = total + part
    assert torch.equal(y[r][:, c], total)


# Columns of more tiles of 128 x 128 than blocks of threads run at a time, so that each takes several: in fp32 one after the other
# along the rows and on to the next 128 places (304 blocks of threads), in 16 bits blocks of columns apart (from 1824 tiles on).  Rows of whole
# vectors and odd ones; groups of all sizes, some empty, rows outside them.
@pytest.mark.parametrize("fmt,out,T,H", [("fp32", "e4m3", 3000, 4096), ("fp32", "e5m2", 3000, 4099), ("fp32", "e4m3", 40000, 130), ("bf16", "e4m3", 4500, 7168),
                                         ("fp16", "e4m3", 4500, 7171), ("bf16", "e5m2", 30000, 1026)])
@pytest.mark.parametrize("ragged", [True, False])
def test_columns_of_more_tiles_than_run_at_a_time(F, fmt, out, T, H, ragged):
    x = values(T + H, T, H, fmt)
    offsets = [T // 9, T // 9, T // 9 + 1, T // 5, T // 5 + 128, T // 2, T // 2, T // 2 + 300, T - 200] if ragged else None
    o = torch.tensor(offsets, dtype=torch.int32, device="cuda") if ragged else None
    P = F.columns(T, len(offsets) - 1 if ragged else 1)
    assert P // 128 * blocks(H) >= 2 * (304 if fmt == "fp32" else 912)
    qt0, et0 = columns_host(x, out, offsets)
    q0, e0 = rows_host(x, out)
    x = x.cuda()
    for rows in (True, False):
        q, e, qt, et = F.quantize(x, out=out, rows=rows, columns=True, offsets=o)
        assert torch.equal(et.cpu(), et0) and same(qt.cpu(), qt0)
        assert not rows or (torch.equal(e.cpu(), e0) and same(q.cpu(), q0))


@pytest.mark.parametrize("less", [0, 3])
def test_rows_longer_than_two_dimensions_of_a_grid_hold(F, less):
    """65535 times sixteen blocks of 128 and more, against the same numbers in shorter rows."""
    H = 65535 * 2048 + 3 * 2048 + 5 * 128
    x = (torch.randn(H, generator=gen(less), device="cuda") * torch.exp2((torch.arange(H, device="cuda") // 128 % 19).float())).bfloat16()
    x[H - less:] = 0
    q, e, _, _ = F.quantize(x[None, :H - less])
    q0, e0, _, _ = F.quantize(x.view(-1, 128))
    assert torch.equal(e[0], e0[:, 0]) and torch.equal(raw(q)[0], raw(q0).view(-1)[:H - less])
