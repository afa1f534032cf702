"""The C ABI of the 8-bit layer operators without a GPU: every declared function is exported and
bound, and arguments that do not fit are refused before anything is launched."""
import ctypes
import os
import re
import subprocess

import pytest

from bit_exact_emulation_gb300 import build as B

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mcemu_ops.h")
FP16, BF16, XF32, FP32, E4M3, E5M2, INT8, UINT8, INT32 = range(9)
OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 4, 7


@pytest.fixture(scope="module")
def L():
    B.build()
    from bit_exact_emulation_gb300 import ops
    return ops.lib()


def test_library_exports_every_declared_symbol(L):
    from bit_exact_emulation_gb300 import ops
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(mcemu_[a-z0-9_]+)\s*\(", text))
    out = subprocess.run(["nm", "-D", "--defined-only", B.LIB_PATH], capture_output=True, text=True).stdout
    assert names <= set(re.findall(r"\bT (mcemu_\w+)", out))
    assert set(ops.SYMBOLS) == names
    assert int(re.search(r"MCEMU_ACT8_BLOCK (\d+)", text).group(1)) == ops.ACT8_BLOCK
    assert int(re.search(r"MCEMU_ACT8_NAN \((-\d+)\)", text).group(1)) == ops.ACT8_NAN
    assert int(re.search(r"MCEMU_INT32 = (\d+)", text).group(1)) == ops.INT32


# Pointers that are never followed: every call below is refused (or empty) before a launch.
P, ODD = 0x10000, 0x10001


def norm(L, fmt=BF16, wfmt=BF16, out=INT8, T=4, H=64, x=P, ldx=64, res=0, ldr=64, w=P, eps=1e-5, h=0, ldh=64, y=P, ldy=64,
         scale=P, rstd=P):
    return L.mcemu_rmsnorm(fmt, wfmt, out, T, H, x, ldx, res, ldr, w, eps, h, ldh, y, ldy, scale, rstd, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), OK), (dict(T=0, x=0, y=0), OK), (dict(fmt=9), INVALID), (dict(fmt=-1), INVALID), (dict(fmt=INT8), UNSUPPORTED),
    (dict(fmt=XF32), UNSUPPORTED), (dict(wfmt=FP16), UNSUPPORTED), (dict(out=FP32), UNSUPPORTED), (dict(out=UINT8), UNSUPPORTED),
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(x=0), INVALID), (dict(w=0), INVALID), (dict(y=0), INVALID), (dict(scale=0), INVALID),
    (dict(res=P), INVALID), (dict(h=P), INVALID), (dict(ldx=63), INVALID), (dict(ldy=63), INVALID),
    (dict(res=P, h=P, ldr=63), INVALID), (dict(res=P, h=P, ldh=63), INVALID), (dict(x=ODD), ALIGNMENT), (dict(w=ODD), ALIGNMENT),
    (dict(wfmt=FP32, w=P + 2), ALIGNMENT), (dict(out=BF16, y=ODD), ALIGNMENT), (dict(scale=P + 2), ALIGNMENT),
    (dict(rstd=P + 2), ALIGNMENT), (dict(res=ODD, h=P), ALIGNMENT)])
def test_rmsnorm_refusals(L, kw, status):
    assert norm(L, **kw) == status


def grad(L, fmt=BF16, wfmt=BF16, T=4, H=200, dy=P, lddy=200, dres=0, lddr=200, h=P, ldh=200, q=0, ldq=200, e=0, lde=2, rstd=P,
         w=P, dx=P, lddx=200, dw=P, ws=P, nws=1 << 30):
    return L.mcemu_rmsnorm_backward(fmt, wfmt, T, H, dy, lddy, dres, lddr, h, ldh, q, ldq, e, lde, rstd, w, dx, lddx, dw, ws,
                                    nws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=INT8), UNSUPPORTED), (dict(fmt=99), INVALID), (dict(wfmt=FP16), UNSUPPORTED), (dict(T=-1), INVALID),
    (dict(H=0), INVALID), (dict(dw=0), INVALID), (dict(dw=P + 2), ALIGNMENT), (dict(dy=0), INVALID), (dict(w=0), INVALID),
    (dict(dx=0), INVALID), (dict(rstd=0), INVALID), (dict(h=0), INVALID), (dict(q=P, e=P), INVALID), (dict(h=0, q=P), INVALID),
    (dict(h=0, e=P), INVALID), (dict(h=0, q=P, e=P, ldq=199), INVALID), (dict(h=0, q=P, e=P, lde=1), INVALID),
    (dict(lddy=199), INVALID), (dict(lddx=199), INVALID), (dict(ldh=199), INVALID), (dict(dres=P, lddr=199), INVALID),
    (dict(dy=ODD), ALIGNMENT), (dict(h=ODD), ALIGNMENT), (dict(dres=ODD), ALIGNMENT), (dict(dx=ODD), ALIGNMENT),
    (dict(rstd=ODD), ALIGNMENT), (dict(nws=0), WORKSPACE), (dict(nws=-1), WORKSPACE), (dict(ws=0), INVALID),
    (dict(ws=P + 8), ALIGNMENT)])
def test_rmsnorm_backward_refusals(L, kw, status):
    if kw.get("nws") == -1:                         # one byte short
        kw = dict(nws=L.mcemu_rmsnorm_backward_workspace(4, 200) - 1)
    assert grad(L, **kw) == status


def linear(L, M=4, N=8, K=32, x=P, ldx=32, sx=P, w=P, ldw=32, sw=P, bias=0, out=BF16, y=P, ldy=8, ws=P, nws=1 << 40):
    return L.mcemu_int8_linear(M, N, K, x, ldx, sx, w, ldw, sw, bias, out, y, ldy, ws, nws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), OK), (dict(N=0), OK), (dict(M=0, x=0, y=0), OK), (dict(M=-1), INVALID), (dict(N=-1), INVALID),
    (dict(K=-1), INVALID), (dict(K=131072, ldx=131072, ldw=131072), UNSUPPORTED), (dict(out=INT8), UNSUPPORTED),
    (dict(out=XF32), UNSUPPORTED), (dict(out=9), INVALID), (dict(x=0), INVALID), (dict(w=0), INVALID), (dict(y=0), INVALID),
    (dict(sx=0), INVALID), (dict(sw=0), INVALID), (dict(out=INT32), INVALID), (dict(out=INT32, sx=0, sw=0, bias=P), INVALID),
    (dict(ldx=31), INVALID), (dict(ldw=31), INVALID), (dict(ldy=7), INVALID), (dict(y=ODD), ALIGNMENT),
    (dict(out=INT32, sx=0, sw=0, y=P + 2), ALIGNMENT), (dict(sx=P + 2), ALIGNMENT), (dict(sw=P + 2), ALIGNMENT),
    (dict(bias=P + 2), ALIGNMENT)])
def test_int8_linear_refusals(L, kw, status):
    assert linear(L, **kw) == status


def act(L, f="mcemu_act8_compress", fmt=BF16, T=4, H=200, x=P, ldx=200, q=P, ldq=200, e=P, lde=2):
    a = (x, ldx, q, ldq, e, lde) if f == "mcemu_act8_compress" else (q, ldq, e, lde, x, ldx)
    return getattr(L, f)(fmt, T, H, *a, None)


@pytest.mark.parametrize("f", ["mcemu_act8_compress", "mcemu_act8_expand"])
@pytest.mark.parametrize("kw,status", [
    (dict(T=0), OK), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(fmt=INT8), UNSUPPORTED), (dict(fmt=77), INVALID),
    (dict(x=0), INVALID), (dict(q=0), INVALID), (dict(e=0), INVALID), (dict(ldx=199), INVALID), (dict(ldq=199), INVALID),
    (dict(lde=1), INVALID), (dict(x=ODD), ALIGNMENT), (dict(fmt=FP32, x=P + 2), ALIGNMENT)])
def test_act8_refusals(L, f, kw, status):
    assert act(L, f, **kw) == status


def wgrad(L, T=4, N=8, K=200, dy=P, lddy=8, q=P, ldq=200, e=P, lde=2, out=FP32, acc=0, dW=P, lddw=200, ws=P, nws=1 << 40):
    return L.mcemu_act8_wgrad(T, N, K, dy, lddy, q, ldq, e, lde, out, acc, dW, lddw, ws, nws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(N=0), OK), (dict(K=0), OK), (dict(T=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID),
    (dict(out=FP16), UNSUPPORTED), (dict(out=BF16, acc=1), UNSUPPORTED), (dict(acc=2), INVALID), (dict(out=42), INVALID),
    (dict(dy=0), INVALID), (dict(q=0), INVALID), (dict(e=0), INVALID), (dict(dW=0), INVALID), (dict(lddy=7), INVALID),
    (dict(ldq=199), INVALID), (dict(lde=1), INVALID), (dict(lddw=199), INVALID), (dict(dy=ODD), ALIGNMENT),
    (dict(dW=P + 2), ALIGNMENT)])
def test_act8_wgrad_refusals(L, kw, status):
    assert wgrad(L, **kw) == status


def test_sizes_beyond_32_bits_are_refused(L):
    """Sizes so near 2^31 that what they are rounded up to would not fit."""
    n = 2 ** 31 - 65535
    big = dict(ldx=n, ldy=n, lddy=n, lddx=n, ldh=n, ldq=n, lde=n, lddw=n)
    some = lambda *names: {k: big[k] for k in names}
    assert norm(L, H=n, **some("ldx", "ldy")) == UNSUPPORTED and norm(L, T=n) == UNSUPPORTED
    assert grad(L, H=n, **some("lddy", "lddx", "ldh")) == UNSUPPORTED and grad(L, T=n) == UNSUPPORTED
    assert linear(L, M=n) == UNSUPPORTED and linear(L, N=n, ldy=n) == UNSUPPORTED
    for f in ("mcemu_act8_compress", "mcemu_act8_expand"):
        assert act(L, f, H=n, **some("ldx", "ldq", "lde")) == UNSUPPORTED and act(L, f, T=n) == UNSUPPORTED
    assert wgrad(L, T=n) == UNSUPPORTED and wgrad(L, N=n, lddy=n) == UNSUPPORTED
    assert wgrad(L, K=n, **some("ldq", "lde", "lddw")) == UNSUPPORTED
    for need in (L.mcemu_rmsnorm_backward_workspace(n, 5), L.mcemu_int8_linear_workspace(n, 5, 5, 1),
                 L.mcemu_act8_wgrad_workspace(5, n, 5, 1)):
        assert need == 0


def test_workspaces(L):
    """Sizes come without a device, are 0 for empty problems and do not wrap for large ones."""
    assert L.mcemu_rmsnorm_backward_workspace(0, 10) == 0
    assert L.mcemu_rmsnorm_backward_workspace(1 << 20, 16384) >= 16384 * 4
    assert L.mcemu_int8_linear_workspace(0, 5, 5, 1) == 0 and L.mcemu_act8_wgrad_workspace(5, 0, 5, 1) == 0
    for M, N, K in ((1 << 20, 1 << 20, 131071), (1, 1 << 30, 4096), (1 << 30, 1, 4096)):
        assert L.mcemu_int8_linear_workspace(M, N, K, 0) < 1 << 62


def test_cpu_tensors_are_refused(L):
    from bit_exact_emulation_gb300 import ops
    with pytest.raises(ops.McemuError) as e:
        ops.rmsnorm(torch.zeros(2, 8), torch.zeros(8), 1e-5)
    assert e.value.status == INVALID and "rmsnorm" in str(e.value)
