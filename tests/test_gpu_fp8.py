"""The FP8 layer operators on the GPU against plain implementations in 64 bits.

Operands of small whole numbers and powers of two have sums that every order of addition gives exactly,
so that the products are compared to the last bit; with values as a network has them they
are held to the matrix unit's error bound."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

CODE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
UNIT = {"fp32": 2.0 ** -24, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def F():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_exact_emulation_gb300 import build
    build.build()
    from bit_exact_emulation_gb300 import fp8
    return fp8


def blocks(n):
    return -(-n // 128)


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def raw(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def same(a, b):
    return a.shape == b.shape and a.dtype == b.dtype and torch.equal(raw(a), raw(b))


def strided(t, pad, lead=0):
    """The same tensor with `pad` more elements between rows and `lead` in front."""
    shape = (*t.shape[:-1], t.shape[-1] + pad)
    n = int(np.prod(shape))
    buf = torch.zeros(lead + n + 16, dtype=torch.uint8 if t.element_size() == 1 else t.dtype, device="cuda").view(t.dtype)
    v = buf[lead:lead + n].view(shape)[..., :t.shape[-1]]
    raw_v = v.view(torch.uint8) if t.element_size() == 1 else v
    raw_v.copy_(raw(t) if t.element_size() == 1 else t)
    return v


def whole(g, shape, fmt):
    """Codes of whole numbers from -2 to 2."""
    return torch.randint(-2, 3, shape, generator=g, device="cuda").float().to(CODE[fmt])


def exps(g, *shape):
    return torch.randint(-3, 4, shape, generator=g, device="cuda").to(torch.int8)


def of_rows(q, e):
    s = torch.exp2(e.double()).repeat_interleave(128, -1)[..., :q.shape[-1]]
    return q.double() * s


def of_tiles(q, e):
    return of_rows(q, e.repeat_interleave(128, -2)[..., :q.shape[-2], :])


def rounded(y64, out):
    """Sums that fp32 holds, rounded once.  A sum begins at +0, so that one of negative zeros alone is +0 (a
    library's sum of one product is the product, -0)."""
    assert torch.equal(y64.float().double(), y64)
    return (y64 + 0.0).float().to(DT[out])


# ---------------------------------------------------------------------------
# operands
# ---------------------------------------------------------------------------
def exponent(amax, out):
    """The definition, by comparison: the least e >= -120 with amax <= TOP * 2^e."""
    e = torch.full(amax.shape, -120, dtype=torch.int32)
    a = amax.double().cpu()
    for c in range(-120, 121):
        e[a > TOP[out] * 2.0 ** c] = c + 1
    e[~torch.isfinite(a)] = -128
    return e.to(torch.int8)


def code_host(x, e, out):
    """x * 2^-e (64 bits) to the format, and NaN's code where e says so.  torch rounds fp32 to the
    format to nearest, ties to even; x * 2^-e is exact in 64 bits, and in fp32 above 2^-126."""
    v = (x.double().cpu() * torch.exp2(-e.double())).float().to(CODE[out]).view(torch.uint8)
    return torch.where(e == -128, torch.tensor(0x7F, dtype=torch.uint8), v).view(CODE[out])


def rows_host(x, out):
    T, H = x.shape
    B = blocks(H)
    xp = torch.nn.functional.pad(x.float().cpu(), (0, B * 128 - H)).view(T, B, 128)
    e = exponent(xp.abs().amax(-1), out)
    return code_host(xp, e[..., None].expand(xp.shape), out).view(torch.uint8).view(T, B * 128)[:, :H].contiguous().view(CODE[out]), e


def canonical(offsets, T):
    got, most = [], 0
    for o in offsets:
        most = max(most, min(max(o, 0), T))
        got.append(most)
    return got


def columns_host(x, out, offsets):
    T, H = x.shape
    at = canonical(offsets, T) if offsets is not None else [0, T]
    P = (T + 127 * (len(at) - 1)) // 128 * 128
    xt = torch.zeros(H, P)
    first = 0
    for a, b in zip(at, at[1:]):
        xt[:, first:first + b - a] = x[a:b].float().cpu().T
        first += 128 * blocks(b - a)
    return rows_host(xt, out) if P else (torch.empty(H, 0).to(CODE[out]), torch.empty(H, 0, dtype=torch.int8))


def values(seed, T, H, fmt, special=True):
    """Normal values over many binades; values next to the exponents' borders, zeros, a block of zeros."""
    g = np.random.default_rng(seed)
    x = g.standard_normal((T, H)) * np.exp2(g.integers(-8, 8, (T, 1))) * np.exp(0.5 * g.standard_normal(H))
    if special and T * H > 4:
        x.flat[0] = 1.75 * 2 ** 6
        x.flat[T * H // 2] = np.nextafter(np.float32(1.75 * 2 ** 7), np.float32(1e9))
        x[T // 3, H // 2:] = 0
        x[T // 2:T // 2 + 1, :128] = 0
    return torch.from_numpy(x.astype(np.float32)).to(DT[fmt])


@pytest.mark.parametrize("T,H", [(1, 1), (1, 4096), (3, 7), (5, 128), (130, 129), (37, 1000), (300, 2050), (1, 33001)])
@pytest.mark.parametrize("fmt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("out", ["e4m3", "e5m2"])
def test_quantize_rows(F, T, H, fmt, out):
    x = values(T * 7 + H, T, H, fmt)
    q, e, qt, et = F.quantize(x.cuda(), out=out)
    q0, e0 = rows_host(x, out)
    assert qt is None and et is None
    assert torch.equal(e.cpu(), e0) and same(q.cpu(), q0)


GROUPS = [None, [0, 300], [0, 0, 5, 5, 135, 263, 300], [7, 8, 8, 200, 290], [300, 300, 300], [0, 128, 256, 300], [20, 10, 400, -5, 290]]


@pytest.mark.parametrize("offsets", GROUPS, ids=str)
@pytest.mark.parametrize("H", [1, 128, 136, 301])
@pytest.mark.parametrize("fmt,out", [("bf16", "e4m3"), ("fp16", "e5m2"), ("fp32", "e4m3")])
@pytest.mark.parametrize("rows", [True, False])
def test_quantize_columns(F, offsets, H, fmt, out, rows):
    x = values(H, 300, H, fmt)
    o = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    q, e, qt, et = F.quantize(x.cuda(), out=out, rows=rows, columns=True, offsets=o)
    qt0, et0 = columns_host(x, out, offsets)
    assert torch.equal(et.cpu(), et0) and same(qt.cpu(), qt0)
    if rows:
        q0, e0 = rows_host(x, out)
        assert torch.equal(e.cpu(), e0) and same(q.cpu(), q0)
    else:
        assert q is None and e is None


@pytest.mark.parametrize("E", [33, 200, 1024])
def test_quantize_columns_of_many_groups(F, E):
    """More groups than a warp has lanes, many of them empty."""
    r = np.random.default_rng(E)
    T = 500
    offsets = [0, *sorted(r.integers(0, T + 1, E - 1).tolist()), T]
    x = values(E, T, 40, "bf16")
    _, _, qt, et = F.quantize(x.cuda(), rows=False, columns=True, offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    qt0, et0 = columns_host(x, "e4m3", offsets)
    assert torch.equal(et.cpu(), et0) and same(qt.cpu(), qt0)


@pytest.mark.parametrize("pad,lead", [(0, 1), (3, 0), (8, 8), (24, 5)])
def test_quantize_strides_and_given_outputs(F, pad, lead):
    """Any strides and offsets; what lies around the outputs' rows is not touched."""
    T, H = 150, 200
    x = values(5, T, H, "bf16")
    want = F.quantize(x.cuda(), columns=True)
    P = want[2].shape[1]

    def room(rows, cols, dtype):
        buf = torch.full((lead + rows * (cols + pad) + 16,), 0xA5, dtype=torch.uint8, device="cuda")
        return buf, buf[lead:lead + rows * (cols + pad)].view(rows, cols + pad)[:, :cols].view(dtype)

    rooms = [room(T, H, torch.float8_e4m3fn), room(T, 2, torch.int8), room(H, P, torch.float8_e4m3fn), room(H, P // 128, torch.int8)]
    got = F.quantize(strided(x.cuda(), pad, lead), columns=True, **dict(zip(("q", "e", "qt", "et"), [v for _, v in rooms])))
    for (buf, v), g, w in zip(rooms, got, want):
        assert g.data_ptr() == v.data_ptr() and same(g, w)
        v.view(torch.uint8).fill_(0xA5)
        assert torch.all(buf == 0xA5)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("fmt", ["bf16", "fp16", "fp32"])
def test_a_block_that_is_not_finite_reads_back_as_nan(F, bad, fmt):
    x = values(9, 200, 300, fmt)
    x[130, 200] = bad
    q, e, qt, et = F.quantize(x.cuda(), columns=True)
    q0, e0 = rows_host(x, "e4m3")
    qt0, et0 = columns_host(x, "e4m3", None)
    assert e0[130, 1] == -128 and et0[200, 1] == -128
    assert torch.equal(e.cpu(), e0) and same(q.cpu(), q0) and torch.equal(et.cpu(), et0) and same(qt.cpu(), qt0)
    w, ew, _, _ = F.quantize_weight(x.cuda())
    assert ew[1, 1] == -128 and (ew == -128).sum() == 1
    assert torch.isnan(w[128:, 128:256].float()).all() and torch.isnan(w.float()).sum() == 72 * 128


@pytest.mark.parametrize("out", ["e4m3", "e5m2"])
def test_quantize_extreme_values(F, out):
    """Subnormals, the largest numbers of fp32, blocks at the least exponent."""
    m = np.float32(np.finfo(np.float32).max)
    x = torch.zeros(6, 128)
    x[0, :4] = torch.tensor([m, m / 2, 1.0, 1e-38])
    x[1, :3] = torch.tensor([1e-45, 3e-45, 1e-40])
    x[2, :3] = torch.tensor([TOP[out] * 2.0 ** -120, 2.0 ** -121, 2.0 ** -135])
    x[3, :2] = torch.tensor([TOP[out] * 2.0 ** -120 * (1 + 2.0 ** -23), 2.0 ** -125])
    x[4, :2] = torch.tensor([1e-30, -1e-36])
    q, e, _, _ = F.quantize(x.cuda(), out=out)
    q0, e0 = rows_host(x, out)
    assert torch.equal(e.cpu(), e0) and same(q.cpu(), q0)


def weight_host(w, out):
    N, K = w.shape
    n, k = blocks(N), blocks(K)
    p = torch.nn.functional.pad(w.float().cpu(), (0, k * 128 - K, 0, n * 128 - N)).view(n, 128, k, 128)
    e = exponent(p.abs().amax((1, 3)), out)
    q = code_host(p, e[:, None, :, None].expand(p.shape), out).view(torch.uint8).reshape(n * 128, k * 128)[:N, :K]
    return q.contiguous().view(CODE[out]), e


@pytest.mark.parametrize("shape", [(1, 1), (128, 128), (3, 130, 200), (2, 1, 300), (5, 129, 1), (1, 264, 523), (1000, 72)])
@pytest.mark.parametrize("fmt,out", [("bf16", "e4m3"), ("fp16", "e5m2"), ("fp32", "e4m3")])
@pytest.mark.parametrize("pad", [0, 3])
def test_quantize_weight(F, shape, fmt, out, pad):
    N, K = shape[-2:]
    E = shape[0] if len(shape) == 3 else 1
    w = torch.stack([values(i + N, N, K, fmt) for i in range(E)])
    given = strided(w.cuda(), pad, pad)
    q, e, qt, et = F.quantize_weight(given if len(shape) == 3 else given[0], out=out, transposed=True)
    only, eonly, none, _ = F.quantize_weight(given if len(shape) == 3 else given[0], out=out)
    assert same(only, q) and same(eonly, e) and none is None
    if len(shape) == 2:
        q, e, qt, et = (t[None] for t in (q, e, qt, et))
    for i in range(E):
        q0, e0 = weight_host(w[i], out)
        assert same(q[i].cpu(), q0) and torch.equal(e[i].cpu(), e0)
        assert same(qt[i].cpu(), q0.view(torch.uint8).T.contiguous().view(CODE[out])) and torch.equal(et[i].cpu(), e0.T)


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------
SHAPES = [(1, 1, 1), (1, 128, 128), (2, 5, 33), (3, 17, 130), (16, 4096, 512), (17, 300, 1000), (33, 129, 257), (64, 1000, 2048),
          (77, 5003, 2049), (128, 512, 4096), (129, 513, 640), (300, 500, 1111), (700, 230, 96), (1, 4096, 16384), (513, 1025, 513),
          (2048, 1000, 300), (1000, 2, 200), (1, 200, 128 * 67), (256, 224, 512), (257, 225, 513), (4000, 5000, 2700), (3000, 9000, 1024), (2304, 20000, 130)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("tiles", [True, False])
@pytest.mark.parametrize("fx,fw,out", [("e4m3", "e4m3", "bf16"), ("e5m2", "e4m3", "fp32"), ("e4m3", "e5m2", "fp16"), ("e5m2", "e5m2", "fp32")])
def test_linear_is_exact_where_fp32_is(F, M, N, K, tiles, fx, fw, out):
    g = gen(M * 31 + N * 7 + K)
    x, w = whole(g, (M, K), fx), whole(g, (N, K), fw)
    ex, ew = exps(g, M, blocks(K)), exps(g, blocks(N) if tiles else N, blocks(K))
    bias = torch.randint(-8, 9, (N,), generator=g, device="cuda").float() if (M + N) % 2 else None
    y = F.linear(x, ex, w, ew, bias=bias, out=out)
    want = of_rows(x, ex) @ (of_tiles(w, ew) if tiles else of_rows(w, ew)).T
    if bias is not None:
        want = want + bias.double()
    assert same(y, rounded(want, out))
    F.check()


def counts_of(offsets, T):
    at = canonical(offsets, T)
    return list(zip(at, at[1:]))


GROUPED = [(300, [0, 0, 5, 5, 135, 263, 300]), (300, [7, 8, 8, 200, 290]), (5, [0, 1, 2, 2, 5]), (1, [0, 1]), (1000, [0, 1000]),
           (700, [0, 256, 512, 700]), (300, [300, 300, 300]), (300, [20, 10, 400, -5, 290]), (64, list(range(0, 65))),
           (1500, [0, 3, 1400, 1400, 1500]), (9000, [0, 3000, 3001, 6500, 9000])]


@pytest.mark.parametrize("T,offsets", GROUPED, ids=str)
@pytest.mark.parametrize("N,K", [(1, 1), (128, 512), (300, 700), (513, 1111), (224, 128)])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_grouped_linear_is_exact_where_fp32_is(F, T, offsets, N, K, out):
    """Also rows outside all groups: left as they were."""
    E = len(offsets) - 1
    g = gen(T + N + K)
    x, w = whole(g, (T, K), "e4m3"), whole(g, (E, N, K), "e4m3" if N != 300 else "e5m2")
    ex, ew = exps(g, T, blocks(K)), exps(g, E, blocks(N), blocks(K))
    y = torch.full((T, N), 123.0, dtype=DT[out], device="cuda")
    want = y.clone()
    F.grouped_linear(x, ex, w, ew, torch.tensor(offsets, dtype=torch.int32, device="cuda"), out=out, y=y)
    xv, wv = of_rows(x, ex), of_tiles(w, ew)
    for i, (a, b) in enumerate(counts_of(offsets, T)):
        want[a:b] = rounded(xv[a:b] @ wv[i].T, out)
    assert same(y, want)
    F.check()


@pytest.mark.parametrize("T,offsets", GROUPED, ids=str)
@pytest.mark.parametrize("N,K", [(1, 1), (128, 224), (300, 700), (264, 523)])
@pytest.mark.parametrize("out", ["fp32", "bf16"])
def test_grouped_wgrad_is_exact_where_fp32_is(F, T, offsets, N, K, out):
    E = len(offsets) - 1
    g = gen(T + N + K + 1)
    o = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    dy, x = (torch.randint(-2, 3, (T, n), generator=g, device="cuda").to(torch.bfloat16) for n in (N, K))
    _, _, dyt, edyt = F.quantize(dy, rows=False, columns=True, offsets=o)
    _, _, xt, ext = F.quantize(x, rows=False, columns=True, offsets=o, out="e5m2" if N == 300 else "e4m3")
    dW = F.grouped_wgrad(dyt, edyt, xt, ext, o, out=out)
    want = torch.stack([dy[a:b].double().T @ x[a:b].double() for a, b in counts_of(offsets, T)])
    assert same(dW, rounded(want, out))
    if out == "fp32":
        more = F.grouped_wgrad(dyt, edyt, xt, ext, o, dW=dW, accumulate=True)
        assert more.data_ptr() == dW.data_ptr() and same(dW, rounded(2 * want, out))
    F.check()
