"""The 8-bit layer operators on the GPU against plain implementations in 64 bits (whole
numbers, and whatever the definitions fix to the last bit, exactly)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U32 = 2.0 ** -24                                    # unit roundoffs
UNIT = {"fp32": 2.0 ** -24, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
TOP = {"int8": 127.0, "e4m3": 448.0, "e5m2": 57344.0}
EPS = 1e-5


@pytest.fixture(scope="module")
def O():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_exact_emulation_gb300 import build
    build.build()
    from bit_exact_emulation_gb300 import ops
    return ops


DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def rows(rng, T, H, dt, scale=1.0):
    """Normal rows with a few large channels, on the host."""
    gain = np.exp(0.3 * rng.standard_normal(H))
    gain[rng.random(H) < 0.02] *= 20
    return torch.from_numpy((rng.standard_normal((T, H)) * gain * scale).astype(np.float32)).to(dt)


def strided(t, pad, lead=0):
    """The same matrix on the GPU with `pad` more elements between rows and `lead` in front."""
    T, H = t.shape
    buf = torch.empty(lead + T * (H + pad) + 16, dtype=t.dtype, device="cuda")
    v = buf[lead:lead + T * (H + pad)].view(T, H + pad)[:, :H]
    v.copy_(t)
    return v


def bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]).cpu()


def same(got, want):
    return torch.equal(bits(got), bits(want))


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------
def norm_host(x, w, res, out):
    """h, the 8-bit values (fixed to the last bit by the definition), and rstd, scale and the
    norm itself in 64 bits."""
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    hd = h.double()
    rstd = 1 / torch.sqrt((hd * hd).mean(1) + np.float32(EPS).item())
    y64 = hd * rstd[:, None] * w.double()
    if out == "own":
        return h, None, rstd, None, y64
    v = h.float().numpy() * w.float().numpy()
    A = np.maximum(np.abs(v).max(1), np.float32(2.0 ** -100))
    v = v * (np.float32(TOP[out]) / A)[:, None]
    assert v.dtype == np.float32
    q = torch.from_numpy(np.rint(v)).to(torch.int8) if out == "int8" else torch.from_numpy(v).to(FP8[out])
    return h, q, rstd, torch.from_numpy(A).double() * rstd / TOP[out], y64


def norm_tol(H):
    """Relative error of rstd: half that of the sum of squares, whose longest chain of fp32
    additions is 32 (a thread's elements; H / 1024 in long rows) + 5 (a warp) + 32 (warps), and six
    single roundings."""
    return ((max(32, H / 1024 + 1) + 37) / 2 + 6) * U32


NORM_SHAPES = [(1, 1), (3, 7), (2, 64), (5, 100), (1, 4096), (37, 1000), (700, 128), (650, 1025), (9, 5003),
               (3, 8192), (400, 4104), (2, 16384), (2, 32768), (2, 33001), (700, 2050), (310, 16384), (320, 9001)]


@pytest.mark.parametrize("T,H", NORM_SHAPES)
@pytest.mark.parametrize("fmt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("out", ["int8", "e4m3", "e5m2", "own"])
def test_rmsnorm(O, T, H, fmt, out):
    rng = np.random.default_rng(T * 7919 + H)
    has_res = (T + H) % 2 == 0
    x = rows(rng, T, H, DT[fmt])
    res = rows(rng, T, H, DT[fmt]) if has_res else None
    w = torch.from_numpy((1 + 0.2 * rng.standard_normal(H)).astype(np.float32)).to(DT[fmt] if H % 3 else torch.float32)
    y, scale, rstd, h = O.rmsnorm(x.cuda(), w.cuda(), EPS, residual=None if res is None else res.cuda(), out=out)
    h0, q0, rstd0, scale0, y0 = norm_host(x, w, res, out)
    tol = norm_tol(H)
    assert torch.all((rstd.cpu().double() - rstd0).abs() <= tol * rstd0)
    if has_res:
        assert same(h, h0)
    else:
        assert h is None
    if out == "own":
        assert scale is None and y.dtype == x.dtype
        tiny = 2.0 ** -25 if fmt == "fp16" else 2.0 ** -140
        assert torch.all((y.cpu().double() - y0).abs() <= (UNIT[fmt] + tol + 2 * U32) * y0.abs() * 1.01 + tiny)
    else:
        assert same(y, q0)
        assert torch.all((scale.cpu().double() - scale0).abs() <= (tol + 2 * U32) * scale0)


@pytest.mark.parametrize("H", [3, 201, 500, 1001, 1201, 2001, 2501, 3001, 4001, 4503, 5003, 6001, 8191])
@pytest.mark.parametrize("fmt,out", [("bf16", "int8"), ("fp16", "own"), ("fp32", "e4m3")])
def test_rmsnorm_many_odd_rows(O, H, fmt, out):
    """Many rows that no vector fits, at every number of threads to a row."""
    for T in (305, 700):
        test_rmsnorm(O, T, H, fmt, out)


@pytest.mark.parametrize("H", [201, 1001, 5003])
@pytest.mark.parametrize("pad,lead", [(0, 0), (3, 1), (8, 5)])
def test_rmsnorm_many_odd_rows_strides_and_in_place(O, H, pad, lead):
    rng = np.random.default_rng(H + pad)
    x, r = rows(rng, 500, H, torch.bfloat16), rows(rng, 500, H, torch.bfloat16)
    w = rows(rng, 1, H, torch.bfloat16)[0]
    h, q = norm_host(x, w, r, "int8")[:2]
    for into in (0, 1):
        gx, gr = strided(x, pad, lead), strided(r, pad, lead)
        y, scale, rstd, got = O.rmsnorm(gx, w.cuda(), EPS, residual=gr, h=(gx, gr)[into])
        assert same(got, h) and same(y, q)
    fresh = O.rmsnorm(x.cuda(), w.cuda(), EPS, residual=r.cuda())
    assert same(fresh[0], q) and same(fresh[1], scale) and same(fresh[2], rstd)


@pytest.mark.parametrize("pads", [(8, 8, 16, 16, 0), (1, 3, 5, 7, 1), (8, 8, 8, 3, 0), (0, 0, 0, 0, 1)])
@pytest.mark.parametrize("H", [512, 1001])
def test_rmsnorm_strides(O, pads, H):
    """Rows at any stride and any element offset; what lies between them is not touched."""
    rng = np.random.default_rng(H)
    x, res = rows(rng, 41, H, torch.bfloat16), rows(rng, 41, H, torch.bfloat16)
    w = torch.ones(H, dtype=torch.bfloat16)
    px, pr, ph, py, lead = pads
    h = strided(torch.zeros_like(x), ph, lead)
    y = strided(torch.zeros(41, H, dtype=torch.int8), py, lead)
    back = y.as_strided((41, H + py), (H + py, 1))
    back[:, H:] = 77
    O.rmsnorm(strided(x, px, lead), w.cuda(), EPS, residual=strided(res, pr, lead), out="int8", y=y, h=h)
    h0, q0, *_ = norm_host(x, w, res, "int8")
    assert same(h, h0) and same(y, q0)
    assert torch.all(back[:, H:] == 77)


@pytest.mark.parametrize("H", [300, 2048, 40000])
def test_rmsnorm_in_place(O, H):
    rng = np.random.default_rng(1)
    x, res = rows(rng, 5, H, torch.bfloat16), rows(rng, 5, H, torch.bfloat16)
    w = torch.ones(H, dtype=torch.bfloat16)
    h0, q0, *_ = norm_host(x, w, res, "int8")
    for into in (0, 1):
        gx, gr = x.cuda(), res.cuda()
        y, _, _, h = O.rmsnorm(gx, w.cuda(), EPS, residual=gr, h=(gx, gr)[into])
        assert same(h, h0) and same(y, q0) and h.data_ptr() == (gx, gr)[into].data_ptr()


@pytest.mark.parametrize("out", ["int8", "e4m3", "e5m2"])
@pytest.mark.parametrize("H", [8, 1024, 33000])
def test_rmsnorm_special_rows(O, H, out):
    """Rows of zeros, tiny rows, and rows with an infinity or a NaN, which never read back as
    finite values; their neighbours are not disturbed."""
    x = torch.ones(7, H)
    x[0] = 0
    x[1] = 1e-36
    x[2, H // 2] = float("inf")
    x[3, H - 1] = float("nan")
    x[4] = -2.0 ** -110
    x[5, 0] = 500.0
    w = torch.ones(H)
    y, scale, rstd, _ = O.rmsnorm(x.cuda(), w.cuda(), EPS, out=out)
    got = y.cpu().float() * scale.cpu()[:, None]
    ok = [0, 1, 4, 5, 6]
    _, q0, rstd0, scale0, _ = norm_host(x[ok], w, None, out)
    assert same(y[torch.tensor(ok).cuda()], q0)
    assert torch.all((scale.cpu()[ok].double() - scale0).abs() <= (norm_tol(H) + 2 * U32) * scale0)
    assert torch.all(got[0] == 0)
    assert not torch.isfinite(got[2]).any() and not torch.isfinite(got[3]).any()


def test_rmsnorm_nan_weight_poisons_every_row(O):
    w = torch.ones(256)
    w[100] = float("nan")
    y, scale, _, _ = O.rmsnorm(torch.ones(3, 256).cuda(), w.cuda(), EPS)
    assert torch.isnan(scale).all()


# ---------------------------------------------------------------------------
# checkpoints
# ---------------------------------------------------------------------------
def compress_host(x, fmt):
    T, H = x.shape
    B = -(-H // 128)
    xf = np.zeros((T, B * 128), np.float64)
    xf[:, :H] = x.double().numpy()
    xb = xf.reshape(T, B, 128)
    with np.errstate(invalid="ignore"):
        amax = np.abs(xb).max(-1)
    bad = ~np.isfinite(xb).all(-1)
    amax[bad] = 1.0
    m, e = np.frexp(amax)
    e = e - 7 + (m * 128 > 127)
    e = np.minimum(np.maximum(e, -120), 9 if fmt == "fp16" else 121)
    with np.errstate(invalid="ignore"):
        q = np.clip(np.rint(xb * np.exp2(-e.astype(np.float64))[..., None]), -127, 127)
    e[bad] = -128
    q[np.isnan(q)] = 0
    return q.reshape(T, -1)[:, :H].astype(np.int8), e.astype(np.int8), bad


ACT_SHAPES = [(1, 1), (1, 128), (3, 127), (2, 129), (5, 256), (7, 1000), (33, 4096), (2, 16391), (300, 264), (4, 132)]


@pytest.mark.parametrize("T,H", ACT_SHAPES)
@pytest.mark.parametrize("fmt", ["bf16", "fp16", "fp32"])
def test_act8_roundtrip(O, T, H, fmt):
    rng = np.random.default_rng(H)
    x = rows(rng, T, H, torch.float32) * torch.from_numpy(np.exp2(rng.integers(-10, 4, (T, 1))).astype(np.float32))
    x = x.to(DT[fmt])
    q, e = O.act8_compress(x.cuda())
    q0, e0, _ = compress_host(x, fmt)
    assert np.array_equal(e.cpu().numpy(), e0)
    assert np.array_equal(q.cpu().numpy(), q0)
    want = torch.from_numpy(q0.astype(np.float64) * np.exp2(np.repeat(e0.astype(np.float64), 128, 1)[:, :H]))
    for out in ("bf16", "fp16", "fp32"):
        back = O.act8_expand(q, e, out=out)
        assert same(back, want.to(DT[out]))
    assert torch.equal(want, want.to(torch.bfloat16).double())          # no second rounding in bfloat16
    step = torch.from_numpy(np.exp2(np.repeat(e0.astype(np.float64), 128, 1)[:, :H]))
    assert torch.all((want - x.double()).abs() <= 0.5 * step)


@pytest.mark.parametrize("fmt", ["bf16", "fp16", "fp32"])
def test_act8_special_values(O, fmt):
    big = torch.finfo(DT[fmt]).max
    x = torch.zeros(9, 300)
    x[0, 5], x[1, 130], x[2, 299] = float("inf"), float("nan"), -float("inf")
    x[3] = big
    x[4] = torch.finfo(DT[fmt]).smallest_normal / 4
    x[5, :128] = 127.0
    x[5, 128:] = 127.5 if fmt != "bf16" else 128.0
    x[6] = torch.linspace(-63.5, 63.5, 300)
    x[6, 0] = 127.0
    x[7] = -big
    x = x.to(DT[fmt])
    q, e = O.act8_compress(x.cuda())
    q0, e0, bad = compress_host(x, fmt)
    assert np.array_equal(e.cpu().numpy(), e0) and e0[0, 0] == O.ACT8_NAN
    fine = ~np.repeat(bad, 128, 1)[:, :300]
    assert np.array_equal(q.cpu().numpy()[fine], q0[fine])
    back = O.act8_expand(q, e, out=fmt).cpu().float().numpy()
    assert np.isnan(back[~fine]).all() and np.isfinite(back[fine]).all()


@pytest.mark.parametrize("pad,lead", [(8, 0), (1, 0), (0, 1), (16, 8)])
def test_act8_strides(O, pad, lead):
    rng = np.random.default_rng(5)
    x = rows(rng, 19, 520, torch.bfloat16)
    q = strided(torch.zeros(19, 520, dtype=torch.int8), pad, lead)
    e = strided(torch.zeros(19, 5, dtype=torch.int8), pad, lead)
    O.act8_compress(strided(x, pad, lead), q=q, e=e)
    q0, e0, _ = compress_host(x, "bf16")
    assert np.array_equal(q.cpu().numpy(), q0) and np.array_equal(e.cpu().numpy(), e0)
    out = strided(torch.zeros(19, 520), pad, lead)
    O.act8_expand(q, e, out="fp32", x=out)
    assert np.array_equal(out.cpu().numpy(), q0 * np.exp2(np.repeat(e0.astype(np.float32), 128, 1)[:, :520]))


# ---------------------------------------------------------------------------
# gradients of the norm
# ---------------------------------------------------------------------------
def grad_host(dy, w, rstd, h, dres):
    """dx, dw in 64 bits, with the sums of magnitudes that bound the rounding errors."""
    d, w, r, h = dy.double(), w.double(), rstd.double()[:, None], h.double()
    z, g = h * r, d * w
    mean = (g * z).mean(1, keepdim=True)
    dx = r * (g - z * mean)
    mag = r * (g.abs() + z.abs() * (g * z).abs().mean(1, keepdim=True))
    if dres is not None:
        dx = dx + dres.double()
        mag = mag + dres.double().abs()
    return dx, (d * z).sum(0), mag, (d * z).abs().sum(0)


GRAD_SHAPES = [(1, 1), (2, 7), (3, 64), (1, 4096), (700, 256), (333, 2050), (65, 5003), (40, 8192), (1300, 136),
               (3, 16384), (5, 16390), (7, 20000), (400, 1024), (310, 8200), (160, 16384), (2500, 72)]


@pytest.mark.parametrize("T,H", GRAD_SHAPES)
@pytest.mark.parametrize("fmt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("ckpt", [True, False])
def test_rmsnorm_backward(O, T, H, fmt, ckpt):
    rng = np.random.default_rng(T + H)
    h = rows(rng, T, H, DT[fmt])
    dy = rows(rng, T, H, DT[fmt], 0.1)
    dres = rows(rng, T, H, DT[fmt], 0.1) if (T + H) % 2 else None
    w = torch.from_numpy((1 + 0.2 * rng.standard_normal(H)).astype(np.float32)).to(DT[fmt] if H % 3 else torch.float32)
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    kw = {"dres": None if dres is None else dres.cuda()}
    if ckpt:
        q, e = O.act8_compress(h.cuda())
        h = O.act8_expand(q, e, out="fp32").cpu()
        kw["ckpt"] = (q, e)
    else:
        kw["h"] = h.cuda()
    dx, dw = O.rmsnorm_backward(dy.cuda(), w.cuda(), rstd.cuda(), **kw)
    dx0, dw0, mag, wmag = grad_host(dy, w, rstd, h, dres)
    # dx: the row's mean has at most 32 + 5 + 16 additions in a chain (H / 512 in long rows); ten single roundings
    chain = max(32, H / 512 + 1) + 21 + 10
    assert torch.all((dx.cpu().double() - dx0).abs() <= chain * U32 * mag + UNIT[fmt] * dx0.abs() * 1.01 + 2.0 ** -25)
    # dw: z has two roundings, then T additions in some order
    assert torch.all((dw.cpu().double() - dw0).abs() <= (T + 4) * U32 * wmag + 1e-30)
    again = O.rmsnorm_backward(dy.cuda(), w.cuda(), rstd.cuda(), **kw)
    assert same(dx, again[0]) and same(dw, again[1])


@pytest.mark.parametrize("H", [3, 201, 500, 1001, 1201, 2001, 2501, 3001, 4001, 4503, 5003, 6001, 8191])
@pytest.mark.parametrize("fmt,ckpt", [("bf16", True), ("fp16", False), ("fp32", True), ("fp32", False)])
def test_rmsnorm_backward_odd_rows(O, H, fmt, ckpt):
    """Rows that no vector fits, at every number of threads to a row."""
    test_rmsnorm_backward(O, 330, H, fmt, ckpt)


def test_rmsnorm_backward_against_differences(O):
    """The gradients of sum(c * y) against central differences of the norm in 64 bits."""
    rng = np.random.default_rng(3)
    T, H, d = 4, 96, 1e-5
    h, w, c = rng.standard_normal((T, H)), 1 + 0.2 * rng.standard_normal(H), rng.standard_normal((T, H))
    h, w, c = (torch.from_numpy(v.astype(np.float32)) for v in (h, w, c))

    def f(h, w):
        return (c.double() * h * w / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)).sum().item()

    _, _, rstd, _ = O.rmsnorm(h.cuda(), w.cuda(), EPS, out="own")
    dx, dw = O.rmsnorm_backward(c.cuda(), w.cuda(), rstd, h=h.cuda())
    for t, i in [(0, 0), (1, 50), (3, 95), (2, 17)]:
        e = torch.zeros(T, H, dtype=torch.float64)
        e[t, i] = d
        num = (f(h.double() + e, w.double()) - f(h.double() - e, w.double())) / (2 * d)
        assert abs(num - dx[t, i].item()) <= 1e-5 * (1 + abs(num))
    for i in (0, 33, 95):
        e = torch.zeros(H, dtype=torch.float64)
        e[i] = d
        num = (f(h.double(), w.double() + e) - f(h.double(), w.double() - e)) / (2 * d)
        assert abs(num - dw[i].item()) <= 1e-5 * (1 + abs(num))


@pytest.mark.parametrize("H", [520, 1001])
@pytest.mark.parametrize("pad,lead", [(8, 0), (3, 1)])
def test_rmsnorm_backward_strides_and_in_place(O, H, pad, lead):
    rng = np.random.default_rng(9)
    h, dy, dres = (rows(rng, 21, H, torch.bfloat16) for _ in range(3))
    w = torch.ones(H, dtype=torch.bfloat16)
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    want = O.rmsnorm_backward(dy.cuda(), w.cuda(), rstd.cuda(), h=h.cuda(), dres=dres.cuda())
    for into in (0, 1):
        g, r = strided(dy, pad, lead), strided(dres, pad, lead)
        dx, dw = O.rmsnorm_backward(g, w.cuda(), rstd.cuda(), h=strided(h, pad, lead), dres=r, dx=(g, r)[into])
        tol = 2.0 ** -7                               # one step of bfloat16: sums may associate otherwise
        assert torch.all((dx.float() - want[0].float()).abs() <= tol * want[0].float().abs() + 1e-5)
        assert torch.allclose(dw, want[1], rtol=1e-4, atol=1e-4)


# ---------------------------------------------------------------------------
# product of 8-bit integers
# ---------------------------------------------------------------------------
def linear_host(x, sx, w, sw, bias, out):
    acc = x.numpy().astype(np.float64) @ w.numpy().astype(np.float64).T       # integers below 2^53: exact
    assert np.abs(acc).max(initial=0) < 2 ** 31
    if out == "int32":
        return torch.from_numpy(acc.astype(np.int32))
    v = acc.astype(np.float32) * sx.numpy()[:, None]
    v = v * sw.numpy()[None, :]
    if bias is not None:
        v = v + bias.numpy()[None, :]
    assert v.dtype == np.float32
    return torch.from_numpy(v).to(DT[out])


def int8s(rng, *shape):
    return torch.from_numpy(rng.integers(-128, 128, shape).astype(np.int8))


LINEAR_SHAPES = [(1, 1, 1), (1, 64, 64), (1, 1000, 4096), (1, 5, 16391), (2, 130, 77), (3, 256, 512), (5, 129, 1024),
                 (8, 300, 1040), (9, 64, 128), (16, 4096, 256), (17, 100, 333), (33, 257, 2048), (64, 128, 64),
                 (77, 503, 2049), (128, 128, 1024), (129, 255, 1100), (256, 256, 64), (257, 513, 2111), (300, 40, 4096),
                 (512, 1024, 96), (1000, 264, 520), (31, 1, 100), (2, 3, 0), (700, 700, 15), (40, 130, 20000),
                 (130, 700, 16400), (8000, 264, 256), (1300, 1800, 520), (90, 20000, 256), (100, 3, 0)]


@pytest.mark.parametrize("M,N,K", LINEAR_SHAPES)
def test_int8_linear(O, M, N, K):
    """Exact: the sums as integers, the scaled outputs to the last bit."""
    rng = np.random.default_rng(M * 31 + N * 7 + K)
    x, w = int8s(rng, M, K), int8s(rng, N, K)
    sx = torch.from_numpy(rng.uniform(1e-3, 1e-2, M).astype(np.float32))
    sw = torch.from_numpy(rng.uniform(1e-3, 1e-2, N).astype(np.float32))
    bias = torch.from_numpy(rng.standard_normal(N).astype(np.float32))
    gx, gw = x.cuda(), w.cuda()
    assert same(O.int8_linear(gx, None, gw, None, out="int32"), linear_host(x, sx, w, sw, None, "int32"))
    for out, b in (("bf16", None), ("fp16", bias), ("fp32", bias)):
        got = O.int8_linear(gx, sx.cuda(), gw, sw.cuda(), bias=None if b is None else b.cuda(), out=out)
        assert same(got, linear_host(x, sx, w, sw, b, out)), out


@pytest.mark.parametrize("M", [1, 6, 24, 200])
@pytest.mark.parametrize("K", [1023, 1024, 1025, 4096, 131071])
def test_int8_linear_extreme_sums(O, M, K):
    """The largest sums there are (-128 * -128 throughout) and their neighbours, where an
    accumulator of 24 bits would round."""
    rng = np.random.default_rng(K)
    x = torch.full((M, K), -128, dtype=torch.int8)
    w = torch.full((130, K), -128, dtype=torch.int8)
    w[1] = 127
    w[2, ::2] = 127
    w[3, -1] = -127
    w[4] = int8s(rng, K)
    x[M - 1, 0] = -127
    got = O.int8_linear(x.cuda(), None, w.cuda(), None, out="int32")
    assert same(got, linear_host(x, None, w, None, None, "int32"))


@pytest.mark.parametrize("M", [1, 5, 20, 150])
@pytest.mark.parametrize("pads", [(16, 16, 8, 0), (1, 0, 0, 0), (0, 3, 1, 0), (5, 7, 3, 3), (0, 0, 0, 1)])
def test_int8_linear_strides(O, M, pads):
    rng = np.random.default_rng(M)
    N, K = 203, 528
    x, w = int8s(rng, M, K), int8s(rng, N, K)
    sx, sw = torch.full((M,), 0.5), torch.full((N,), 0.25)
    px, pw, py, lead = pads
    y = strided(torch.zeros(M, N), py, lead)
    back = y.as_strided((M, N + py), (N + py, 1))
    back[:, N:] = 7.0
    O.int8_linear(strided(x, px, lead), sx.cuda(), strided(w, pw, lead), sw.cuda(), out="fp32", y=y)
    assert same(y, linear_host(x, sx, w, sw, None, "fp32"))
    assert torch.all(back[:, N:] == 7.0)


@pytest.mark.parametrize("M,N,K", [(3, 50, 1100), (24, 130, 1100), (40, 300, 1100), (140, 300, 1100), (40, 140, 5)])
def test_int8_linear_every_alignment(O, M, N, K):
    """Rows that start on every byte of sixteen, in either operand."""
    rng = np.random.default_rng(M + N)
    x, w = int8s(rng, M, K), int8s(rng, N, K)
    want = linear_host(x, None, w, None, None, "int32")
    for lead in range(16):
        for px, pw in ((0, 4), (16 - K % 16, 3), (5, 16 - K % 16)):
            got = O.int8_linear(strided(x, px, lead), None, strided(w, pw, (5 * lead + 3) % 16), None, out="int32")
            assert same(got, want), (lead, px, pw)


@pytest.mark.parametrize("M,N,K", [(40, 76 * 128 - 3, 520), (40, 46 * 128 - 5, 900), (100, 36 * 128, 1536),
                                   (40, 28 * 128 - 1, 2000), (77, 23 * 128 - 100, 1999), (128, 15 * 128, 1792), (65, 300, 4096)])
def test_int8_linear_parts_of_k(O, M, N, K):
    """K shared by two to eight blocks, the tokens of a tile dealt out evenly or not."""
    rng = np.random.default_rng(N)
    x, w = int8s(rng, M, K), int8s(rng, N, K)
    assert same(O.int8_linear(x.cuda(), None, w.cuda(), None, out="int32"), linear_host(x, None, w, None, None, "int32"))


def test_int8_linear_matches_the_emulated_unit(O):
    """The sums of the INT8 matrix unit's model, bit for bit."""
    from oracle.presets import block_models
    from bit_exact_emulation_gb300 import binding as L
    rng = np.random.default_rng(12)
    M, N, K = 70, 90, 256
    x, w = int8s(rng, M, K).cuda(), int8s(rng, N, K).cuda()
    model = L.Model(list(block_models("int8", 16).values())[0])
    emu = L.tile_gemm(model, L.tile(0, 32, 32, 16, 8), x, w, torch.zeros(M, N, dtype=torch.int32, device="cuda"))
    assert torch.equal(emu, O.int8_linear(x, None, w, None, out="int32"))


# ---------------------------------------------------------------------------
# weight gradient
# ---------------------------------------------------------------------------
WGRAD_SHAPES = [(1, 1, 1), (1, 128, 128), (5, 7, 130), (64, 64, 64), (63, 200, 129), (256, 128, 256), (257, 130, 300),
                (1000, 520, 136), (2049, 40, 1000), (300, 1030, 514), (4100, 256, 264), (128, 1000, 1), (200, 1300, 1800),
                (2000, 1304, 1800)]


def wgrad_case(rng, T, N, K):
    dy = torch.from_numpy(rng.standard_normal((T, N)).astype(np.float32)).to(torch.bfloat16)
    x = rows(rng, T, K, torch.bfloat16)
    return dy, x


def wgrad_check(got, dy, xq, out, base=None):
    """Each of T products is exact and added with an error of at most 2^-23 of the running sum
    of magnitudes, whatever the order; the matrix unit drops bits in place of rounding."""
    T = dy.shape[0]
    want, mag = dy.double().T @ xq, dy.double().abs().T @ xq.abs()
    if base is not None:
        want, mag = want + base.double(), mag + base.double().abs()
    err = (got.cpu().double() - want).abs()
    assert torch.all(err <= T * 2.0 ** -23 * mag + 2 * UNIT[out] * want.abs() + 1e-37)
    if out == "fp32" and T > 1:                       # and by far less on the whole
        assert err.norm() <= 2e-6 * want.norm()


@pytest.mark.parametrize("T,N,K", WGRAD_SHAPES)
@pytest.mark.parametrize("out", ["fp32", "bf16"])
def test_act8_wgrad(O, T, N, K, out):
    rng = np.random.default_rng(T + N + K)
    dy, x = wgrad_case(rng, T, N, K)
    q, e = O.act8_compress(x.cuda())
    xq = O.act8_expand(q, e, out="fp32").cpu().double()
    got = O.act8_wgrad(dy.cuda(), q, e, out=out)
    wgrad_check(got, dy, xq, out)
    assert same(got, O.act8_wgrad(dy.cuda(), q, e, out=out))
    if out == "fp32":
        base = torch.from_numpy(rng.standard_normal((N, K)).astype(np.float32))
        dW = base.cuda()
        O.act8_wgrad(dy.cuda(), q, e, dW=dW, accumulate=True)
        wgrad_check(dW, dy, xq, out, base)


@pytest.mark.parametrize("pads", [(8, 16, 0, 4, 0), (1, 0, 0, 0, 0), (0, 1, 3, 1, 0), (3, 5, 1, 2, 1), (4, 8, 0, 0, 0)])
def test_act8_wgrad_strides(O, pads):
    rng = np.random.default_rng(2)
    T, N, K = 333, 136, 272
    dy, x = wgrad_case(rng, T, N, K)
    q, e = O.act8_compress(x.cuda())
    xq = O.act8_expand(q, e, out="fp32").cpu().double()
    pd, pq, pe, pw, lead = pads
    dW = strided(torch.zeros(N, K), pw, lead)
    back = dW.as_strided((N, K + pw), (K + pw, 1))
    back[:, K:] = 7.0
    O.act8_wgrad(strided(dy, pd, lead), strided(q.cpu(), pq, lead), strided(e.cpu(), pe, lead), dW=dW)
    wgrad_check(dW, dy, xq, "fp32")
    assert torch.all(back[:, K:] == 7.0)


def test_act8_wgrad_scales_span_the_exponents(O):
    """Blocks of very different exponents meet in one sum; a block that is not finite poisons
    its own columns and no others."""
    rng = np.random.default_rng(4)
    T, N, K = 200, 33, 384
    dy, x = wgrad_case(rng, T, N, K)
    x = x * torch.from_numpy(np.exp2(rng.integers(-60, 30, (T, 1))).astype(np.float32)).to(torch.bfloat16)
    q, e = O.act8_compress(x.cuda())
    xq = O.act8_expand(q, e, out="fp32").cpu().double()
    wgrad_check(O.act8_wgrad(dy.cuda(), q, e), dy, xq, "fp32")
    x[77, 200] = float("inf")
    q, e = O.act8_compress(x.cuda())
    got = O.act8_wgrad(dy.cuda(), q, e).cpu()
    assert torch.isnan(got[:, 128:256]).all()
    assert torch.isfinite(got[:, :128]).all() and torch.isfinite(got[:, 256:]).all()


def test_act8_wgrad_is_a_gradient(O):
    """dW against differences of sum(dy * (X W^T)) in W, in 64 bits (linear in W: one step)."""
    rng = np.random.default_rng(6)
    T, N, K = 96, 20, 150
    dy, x = wgrad_case(rng, T, N, K)
    q, e = O.act8_compress(x.cuda())
    xq = O.act8_expand(q, e, out="fp32").cpu().double()
    got = O.act8_wgrad(dy.cuda(), q, e).cpu().double()
    W = torch.from_numpy(rng.standard_normal((N, K)))
    f = lambda W: (dy.double() * (xq @ W.T)).sum()
    for n, k in [(0, 0), (19, 149), (7, 128)]:
        d = torch.zeros_like(W)
        d[n, k] = 0.5
        mag = (dy.double()[:, n].abs() * xq[:, k].abs()).sum()
        assert abs((f(W + d) - f(W - d)) - got[n, k]) <= T * 2.0 ** -23 * mag + 1e-9 * abs(f(W))


# ---------------------------------------------------------------------------
# empty calls, streams, refusals
# ---------------------------------------------------------------------------
def test_empty_calls(O):
    z = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device="cuda")
    y, scale, rstd, h = O.rmsnorm(z(0, 64), z(64), EPS, residual=z(0, 64))
    assert y.shape == (0, 64) and scale.shape == (0,)
    dx, dw = O.rmsnorm_backward(z(0, 64), z(64), z(0, dt=torch.float32), h=z(0, 64))
    assert dx.shape == (0, 64) and torch.all(dw == 0)
    q, e = O.act8_compress(z(0, 64))
    assert q.shape == (0, 64) and e.shape == (0, 1)
    i8, f = torch.int8, torch.float32
    assert O.int8_linear(z(0, 8, dt=i8), z(0, dt=f), z(4, 8, dt=i8), z(4, dt=f)).shape == (0, 4)
    y = O.int8_linear(z(3, 0, dt=i8), torch.ones(3, device="cuda"), z(4, 0, dt=i8), torch.ones(4, device="cuda"),
                      bias=torch.arange(4.0, device="cuda"), out="fp32")
    assert torch.equal(y.cpu(), torch.arange(4.0).expand(3, 4))
    dW = O.act8_wgrad(z(0, 5), z(0, 9, dt=i8), z(0, 1, dt=i8))
    assert torch.all(dW == 0) and dW.shape == (5, 9)
    keep = torch.ones(5, 9, device="cuda")
    O.act8_wgrad(z(0, 5), z(0, 9, dt=i8), z(0, 1, dt=i8), dW=keep, accumulate=True)
    assert torch.all(keep == 1)


def test_calls_run_on_the_current_stream(O):
    rng = np.random.default_rng(8)
    x = rows(rng, 600, 1024, torch.bfloat16)
    w8 = int8s(rng, 512, 1024)
    w = torch.ones(1024, dtype=torch.bfloat16)
    gw, gw8, sw = w.cuda(), w8.cuda(), torch.full((512,), 0.01, device="cuda")
    src = x.cuda()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        late = torch.zeros_like(src)
        late.copy_(src)                               # the operators must wait for this
        y, scale, rstd, _ = O.rmsnorm(late, gw, EPS)
        out = O.int8_linear(y, scale, gw8, sw, out="fp32")
        q, e = O.act8_compress(late)
        dW = O.act8_wgrad(late[:, :64], q, e)
        dx, dw = O.rmsnorm_backward(late, gw, rstd, ckpt=(q, e))
    s.synchronize()
    y2, scale2, rstd2, _ = O.rmsnorm(src, gw, EPS)
    assert same(y, y2) and same(scale, scale2)
    assert same(out, O.int8_linear(y2, scale2, gw8, sw, out="fp32"))
    q2, e2 = O.act8_compress(src)
    assert same(dW, O.act8_wgrad(src[:, :64], q2, e2))
    dx2, dw2 = O.rmsnorm_backward(src, gw, rstd2, ckpt=(q2, e2))
    assert same(dx, dx2) and same(dw, dw2)


def test_capture_in_a_graph(O):
    """Every operator can be captured once its workspaces exist."""
    rng = np.random.default_rng(21)
    x = rows(rng, 300, 512, torch.bfloat16).cuda()
    w, w8 = torch.ones(512, dtype=torch.bfloat16, device="cuda"), int8s(rng, 256, 512).cuda()
    sw = torch.full((256,), 0.01, device="cuda")

    def step():
        y, scale, rstd, _ = O.rmsnorm(x, w, EPS)
        q, e = O.act8_compress(x)
        return (O.int8_linear(y, scale, w8, sw), O.int8_linear(y[:4], scale[:4], w8, sw), O.act8_wgrad(x, q, e),
                *O.rmsnorm_backward(x, w, rstd, ckpt=(q, e)))

    want = step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(2):
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("H", [135_000_008, 68_000_001])
def test_act8_very_long_rows(O, H):
    """A row of more blocks than a grid's second axis has: the same codes as its parts."""
    g = torch.Generator("cuda").manual_seed(H)
    x = torch.randn(1, H, device="cuda", generator=g).bfloat16()
    q, e = O.act8_compress(x)
    for a, b in ((0, 1 << 20), (64 << 20, 67_500_000), ((H - 100_000) // 128 * 128, H)):
        qa, ea = O.act8_compress(x[:, a:b].contiguous())
        assert same(q[:, a:b], qa) and same(e[:, a // 128:-(-b // 128)], ea)


def test_rmsnorm_backward_very_long_rows(O):
    """Against 64 bits, with the bounds of shorter rows."""
    T, H = 2, 17_000_001
    rng = np.random.default_rng(1)
    h, dy, w = (rows(rng, n, H, torch.bfloat16) for n in (T, T, 1))
    rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
    dx, dw = O.rmsnorm_backward(dy.cuda(), w[0].cuda(), rstd.cuda(), h=h.cuda())
    dx0, dw0, mag, wmag = grad_host(dy, w[0], rstd, h, None)
    chain = H / 512 + 1 + 21 + 10
    assert torch.all((dx.cpu().double() - dx0).abs() <= chain * U32 * mag + UNIT["bf16"] * dx0.abs() * 1.01 + 2.0 ** -25)
    assert torch.all((dw.cpu().double() - dw0).abs() <= (T + 4) * U32 * wmag + 1e-30)


def inside(need):
    """`need` bytes on a 16-byte boundary that is no 32-byte one, and what lies around them."""
    buf = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    assert buf.data_ptr() % 32 == 0
    return buf[16:16 + need], (buf[:16], buf[16 + need:])


@pytest.mark.parametrize("M,N,K", [(1300, 1800, 520), (1100, 1030, 1024)])
def test_workspace_of_the_product(O, M, N, K):
    """Any 16-byte boundary will do, and nothing outside the workspace is written."""
    rng = np.random.default_rng(K)
    x, w = int8s(rng, M, K), int8s(rng, N, K)
    need = O.lib().mcemu_int8_linear_workspace(M, N, K, K % 16 == 0)
    assert need > 0
    ws, around = inside(need)
    got = O.int8_linear(x.cuda(), None, w.cuda(), None, out="int32", workspace=ws)
    assert same(got, linear_host(x, None, w, None, None, "int32"))
    assert all(torch.all(b == 0xA5) for b in around)


@pytest.mark.parametrize("T,N,K", [(300, 264, 200), (700, 257, 130), (5000, 520, 1000)])
def test_workspace_of_the_weight_gradient(O, T, N, K):
    g = torch.Generator("cuda").manual_seed(T)
    dy = torch.randn(T, N, device="cuda", generator=g).bfloat16()
    q, e = O.act8_compress(torch.randn(T, K, device="cuda", generator=g))
    ws, around = inside(O.lib().mcemu_act8_wgrad_workspace(T, N, K, int(N % 8 == 0)))
    assert same(O.act8_wgrad(dy, q, e, workspace=ws), O.act8_wgrad(dy, q, e))
    assert all(torch.all(b == 0xA5) for b in around)


def test_python_refusals(O):
    E = O.McemuError
    bf, f, i8 = torch.bfloat16, torch.float32, torch.int8
    z = lambda *s, dt=bf: torch.zeros(*s, dtype=dt, device="cuda")
    for bad in (lambda: O.rmsnorm(z(4, 8).cpu(), z(8), EPS), lambda: O.rmsnorm(z(4, 8), z(7), EPS),
                lambda: O.rmsnorm(z(4, 8), z(8), EPS, out="fp4"), lambda: O.rmsnorm(z(8, 4).t(), z(8), EPS),
                lambda: O.rmsnorm(z(4, 8), z(8), EPS, residual=z(4, 9)), lambda: O.rmsnorm(z(4, 8), z(8), -1.0),
                lambda: O.rmsnorm(z(4, 8), z(8), float("nan")), lambda: O.rmsnorm(z(4, 8), z(8), EPS, h=z(4, 8)),
                lambda: O.rmsnorm(z(4, 8, dt=torch.float64), z(8), EPS), lambda: O.rmsnorm(z(1, 8).expand(4, 8), z(8), EPS),
                lambda: O.rmsnorm_backward(z(4, 8), z(8), z(4, dt=f)),
                lambda: O.rmsnorm_backward(z(4, 8), z(8), z(4, dt=f), h=z(4, 8), ckpt=(z(4, 8, dt=i8), z(4, 1, dt=i8))),
                lambda: O.rmsnorm_backward(z(4, 8), z(8), z(4, dt=f), ckpt=(z(4, 8, dt=i8), z(4, 2, dt=i8))),
                lambda: O.rmsnorm_backward(z(4, 8), z(8), z(4, dt=f), h=z(4, 8), workspace=z(1, dt=torch.uint8)),
                lambda: O.int8_linear(z(4, 8, dt=i8), z(4, dt=f), z(5, 9, dt=i8), z(5, dt=f)),
                lambda: O.int8_linear(z(4, 8, dt=i8), None, z(5, 8, dt=i8), z(5, dt=f)),
                lambda: O.int8_linear(z(4, 8, dt=i8), z(4, dt=f), z(5, 8, dt=i8), z(5, dt=f), out="int32"),
                lambda: O.int8_linear(z(4, 8), z(4, dt=f), z(5, 8, dt=i8), z(5, dt=f)),
                lambda: O.int8_linear(z(1, 131072, dt=i8), z(1, dt=f), z(1, 131072, dt=i8), z(1, dt=f)),
                lambda: O.act8_compress(z(4, 8, dt=i8)), lambda: O.act8_expand(z(4, 200, dt=i8), z(4, 1, dt=i8)),
                lambda: O.act8_wgrad(z(4, 8, dt=f), z(4, 8, dt=i8), z(4, 1, dt=i8)),
                lambda: O.act8_wgrad(z(4, 8), z(5, 8, dt=i8), z(5, 1, dt=i8)),
                lambda: O.act8_wgrad(z(4, 8), z(4, 8, dt=i8), z(4, 1, dt=i8), out="bf16", accumulate=True),
                lambda: O.act8_wgrad(z(4, 8), z(4, 8, dt=i8), z(4, 1, dt=i8), dW=z(8, 9, dt=f))):
        with pytest.raises(E):
            bad()
    torch.cuda.synchronize()


def test_no_wait_gave_up(O):
    x, w = torch.ones(200, 2048, dtype=torch.int8, device="cuda"), torch.ones(300, 2048, dtype=torch.int8, device="cuda")
    assert torch.all(O.int8_linear(x, None, w, None, out="int32") == 2048)
    O.check()


def test_eight_bit_layer_example(O):
    """The example's layer: int8 rounding costs about a step of 1/127 of a row's largest value in each
    operand (a few thousandths of the output for normal data: at most 2 %); the emulated unit
    has the same integers; of the two FP8 units the one with fewer fraction bits is worse; 8-bit
    checkpoints move gradients by at most half a step of their blocks (at most 2 %)."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "eight_bit_layer.py")
    spec = importlib.util.spec_from_file_location("eight_bit_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    got = example.main(tokens=200, width=512, channels=264)
    assert got["same_integers_as_the_emulated_unit"] and got["one_token_agrees"]
    assert got["int8_layer_error"] < 0.02 and got["output_error"] < 0.01
    assert got["b200_fp8_error"] < got["h100_fp8_error"] < 0.01
    for k in ("weight_gradient_error", "input_gradient_error", "norm_weight_gradient_error"):
        assert got[k] < 0.02, k
