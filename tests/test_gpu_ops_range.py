"""The norm and its gradients over the whole range of their types, against 64 bits."""
import numpy as np
import pytest

from test_gpu_ops import DT, FP8, O, TOP, U32, UNIT, grad_host, norm_tol, rows, same  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DENORMAL = 2.0 ** -149
# every kernel of the norm: rows in vectors, one and several to a block; odd rows, few and many; long rows
SHAPES = [(6, 512), (700, 2048), (6, 501), (700, 501), (6, 40000), (6, 33001)]


def spread(T, H, dt, scales, seed):
    """Rows of the given sizes in turn, each after an ordinary one."""
    rng = np.random.default_rng(seed)
    x = rows(rng, T, H, torch.float32).clamp(-8, 8)
    s = torch.ones(T)
    s[1::2] = torch.tensor(scales)[torch.arange(T // 2) % len(scales)]
    return (x * s[:, None]).to(dt)


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("fmt", ["bf16", "fp32"])
@pytest.mark.parametrize("out", ["own", "int8", "e4m3"])
@pytest.mark.parametrize("scales,eps", [((1e19, 1e25, 1e37), 1e-5), ((1e-20, 1e-25, 1e-28), 0.0), ((1e-20, 1e-21, 1e-22), 1e-42)])
def test_rmsnorm_of_rows_whose_squares_leave_fp32(O, T, H, fmt, out, scales, eps):
    """Squares or their sum beyond fp32, or below its normal numbers where eps does not hide it."""
    x = spread(T, H, DT[fmt], scales, H)
    res = torch.zeros_like(x) if H % 2 else None
    rng = np.random.default_rng(T)
    w = torch.from_numpy((1 + 0.2 * rng.standard_normal(H)).astype(np.float32)).to(DT[fmt])
    y, scale, rstd, h = O.rmsnorm(x.cuda(), w.cuda(), eps, residual=None if res is None else res.cuda(), out=out)
    hd = x.double()
    rstd0 = 1 / torch.sqrt((hd * hd).mean(1) + float(np.float32(eps)))
    tol = norm_tol(H)
    assert torch.all((rstd.cpu().double() - rstd0).abs() <= tol * rstd0)
    if res is not None:
        assert same(h, x)
    if out == "own":
        y0 = hd * rstd0[:, None] * w.double()
        assert torch.all((y.cpu().double() - y0).abs() <= (UNIT[fmt] + tol + 2 * U32) * y0.abs() * 1.01 + DENORMAL * rstd0[:, None])
        return
    v = x.float().numpy() * w.float().numpy()
    A = np.maximum(np.abs(v).max(1), np.float32(2.0 ** -100))
    v = v * (np.float32(TOP[out]) / A)[:, None]
    assert same(y, torch.from_numpy(np.rint(v)).to(torch.int8) if out == "int8" else torch.from_numpy(v).to(FP8[out]))
    scale0 = torch.from_numpy(A).double() * rstd0 / TOP[out]
    assert torch.all((scale.cpu().double() - scale0).abs() <= (tol + 2 * U32) * scale0)


@pytest.mark.parametrize("H", [512, 501, 40000, 33001])
def test_rmsnorm_rows_beyond_repair(O, H):
    """Infinities and NaN among rows whose squares overflow do not read back as finite, and rows of zeros
    without eps have an infinite factor; the other rows stand."""
    x = torch.full((8, H), 1e25)
    x[1, 3], x[3, H - 1], x[5] = float("inf"), float("nan"), 0
    y, scale, rstd, _ = O.rmsnorm(x.cuda(), torch.ones(H).cuda(), 0.0)
    back = (y.cpu().float() * scale.cpu()[:, None])
    assert not torch.isfinite(back[[1, 3, 5]]).any() and torch.isinf(rstd[5]).item()
    assert torch.all((back[[0, 2, 4, 6, 7]] - 1).abs() <= 1e-5)


@pytest.mark.parametrize("H", [512, 501, 9001])
@pytest.mark.parametrize("fmt", ["bf16", "fp32"])
@pytest.mark.parametrize("ckpt", [True, False])
@pytest.mark.parametrize("scales", [(1e19, 1e25, 1e30), (1e-20, 1e-25, 1e-28)])
def test_rmsnorm_backward_of_very_large_and_small_rows(O, H, fmt, ckpt, scales):
    """No intermediate of dx leaves the range that rstd and dx themselves keep to."""
    T = 330
    h = spread(T, H, DT[fmt], scales, H)
    dy = rows(np.random.default_rng(H), T, H, DT[fmt], 0.1)
    w = torch.from_numpy((1 + 0.2 * np.random.default_rng(1).standard_normal(H)).astype(np.float32)).to(DT[fmt])
    if ckpt:
        q, e = O.act8_compress(h.cuda())
        h = O.act8_expand(q, e, out="fp32").cpu()
        kw = {"ckpt": (q, e)}
    else:
        kw = {"h": h.cuda()}
    rstd = (1 / torch.sqrt(h.double().square().mean(1))).float()
    dx, dw = O.rmsnorm_backward(dy.cuda(), w.cuda(), rstd.cuda(), **kw)
    dx0, dw0, mag, wmag = grad_host(dy, w, rstd, h, None)
    chain = max(32, H / 512 + 1) + 21 + 10
    assert torch.all((dx.cpu().double() - dx0).abs() <= chain * U32 * mag + UNIT[fmt] * dx0.abs() * 1.01 + DENORMAL)
    assert torch.all((dw.cpu().double() - dw0).abs() <= (T + 4) * U32 * wmag + 1e-30)
