"""The C ABI and the binding of the FP8 layer operators without a GPU: every declared function is exported
and bound, and what does not fit is refused before anything is launched."""
import os
import re
import subprocess

import pytest

from bit_exact_emulation_gb300 import build as B

torch = pytest.importorskip("torch")
from bit_exact_emulation_gb300 import fp8, ops  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mcemu_fp8.h")
FP16, BF16, XF32, FP32, E4M3, E5M2, INT8, UINT8, INT32 = range(9)
OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 4, 7
P, ODD = 0x10000, 0x10001                          # pointers that are never followed
BIG = 2 ** 31 - 65535


@pytest.fixture(scope="module")
def L():
    B.build()
    return fp8.lib()


def test_library_exports_every_declared_symbol(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(mcemu_[a-z0-9_]+)\s*\(", text))
    out = subprocess.run(["nm", "-D", "--defined-only", B.LIB_PATH], capture_output=True, text=True).stdout
    assert names <= set(re.findall(r"\bT (mcemu_\w+)", out))
    assert set(fp8.SYMBOLS) == names
    assert int(re.search(r"MCEMU_FP8_BLOCK (\d+)", text).group(1)) == fp8.BLOCK
    assert int(re.search(r"MCEMU_FP8_NAN \((-\d+)\)", text).group(1)) == fp8.NAN
    assert int(re.search(r"MCEMU_FP8_MAX_GROUPS (\d+)", text).group(1)) == fp8.MAX_GROUPS


def quantize(L, fmt=BF16, out=E4M3, T=4, H=200, x=P, ldx=200, q=P, ldq=200, e=P, lde=2, qt=0, ldqt=128, et=0, ldet=1, E=0, o=0):
    return L.mcemu_fp8_quantize(fmt, out, T, H, x, ldx, q, ldq, e, lde, qt, ldqt, et, ldet, E, o, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), OK), (dict(T=0, x=0), OK), (dict(T=0, qt=P, et=P), OK), (dict(fmt=9), INVALID), (dict(fmt=-1), INVALID),
    (dict(fmt=INT8), UNSUPPORTED), (dict(fmt=XF32), UNSUPPORTED), (dict(out=INT8), UNSUPPORTED), (dict(out=BF16), UNSUPPORTED),
    (dict(out=77), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(x=0), INVALID), (dict(q=0), INVALID), (dict(e=0), INVALID),
    (dict(q=0, e=0), INVALID), (dict(qt=P), INVALID), (dict(et=P), INVALID), (dict(ldx=199), INVALID), (dict(ldq=199), INVALID),
    (dict(lde=1), INVALID), (dict(qt=P, et=P, ldqt=127), INVALID), (dict(qt=P, et=P, ldet=0), INVALID), (dict(E=1), INVALID),
    (dict(E=0, o=P), INVALID), (dict(E=1025, o=P), INVALID), (dict(E=-1, o=P), INVALID), (dict(E=3, o=P, qt=P, et=P, ldqt=255, ldet=3), INVALID),
    (dict(E=3, o=P + 2, qt=P, et=P, ldqt=384, ldet=3), ALIGNMENT), (dict(x=ODD), ALIGNMENT), (dict(fmt=FP32, x=P + 2), ALIGNMENT),
    (dict(T=BIG), UNSUPPORTED), (dict(H=BIG, ldx=BIG, ldq=BIG, lde=BIG), UNSUPPORTED),
    (dict(T=BIG - 1, q=0, e=0, qt=P, et=P, E=1024, o=P, ldqt=2 ** 40, ldet=2 ** 40), UNSUPPORTED)])
def test_quantize_refusals(L, kw, status):
    assert quantize(L, **kw) == status


def test_columns(L):
    for T, E, want in ((0, 0, 0), (1, 0, 128), (128, 0, 128), (129, 1, 256), (0, 3, 256), (300, 5, 896), (10 ** 9, 1024, 1000130048)):
        assert L.mcemu_fp8_columns(T, E) == want == fp8.columns(T, E)
        if E > 1 and T < 10 ** 6:                  # enough for any division: one row in all groups but one
            most = sum(-(-n // 128) for n in [1] * min(E - 1, T) + [max(T - (E - 1), 0)])
            assert most * 128 <= want
    assert L.mcemu_fp8_columns(-1, 0) == 0 and L.mcemu_fp8_columns(5, 1025) == 0


def weight(L, fmt=BF16, out=E4M3, E=2, N=100, K=200, w=P, ldw=200, sw=20000, q=P, ldq=200, sq=20000, e=P, qt=P, ldqt=100, sqt=20000, et=P):
    return L.mcemu_fp8_quantize_weight(fmt, out, E, N, K, w, ldw, sw, q, ldq, sq, e, qt, ldqt, sqt, et, None)


@pytest.mark.parametrize("kw,status", [
    (dict(N=0), OK), (dict(K=0), OK), (dict(fmt=E4M3), UNSUPPORTED), (dict(out=INT8), UNSUPPORTED), (dict(fmt=12), INVALID),
    (dict(E=0), INVALID), (dict(E=1025), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID), (dict(w=0), INVALID), (dict(q=0), INVALID),
    (dict(e=0), INVALID), (dict(qt=0), INVALID), (dict(et=0), INVALID), (dict(ldw=199), INVALID), (dict(ldq=199), INVALID),
    (dict(ldqt=99), INVALID), (dict(sw=19999), INVALID), (dict(sq=19999), INVALID), (dict(sqt=19999), INVALID), (dict(w=ODD), ALIGNMENT),
    (dict(N=BIG), UNSUPPORTED), (dict(K=BIG), UNSUPPORTED)])
def test_quantize_weight_refusals(L, kw, status):
    assert weight(L, **kw) == status


def linear(L, M=4, N=8, K=32, xf=E4M3, x=P, ldx=32, ex=P, ldex=1, wf=E4M3, w=P, ldw=32, ew=P, ldew=1, tiles=1, bias=0, out=BF16, acc=0,
           y=P, ldy=8, ws=P, nws=1 << 40):
    return L.mcemu_fp8_linear(M, N, K, xf, x, ldx, ex, ldex, wf, w, ldw, ew, ldew, tiles, bias, out, acc, y, ldy, ws, nws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), OK), (dict(N=0), OK), (dict(M=0, x=0, y=0), OK), (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID),
    (dict(xf=INT8), UNSUPPORTED), (dict(wf=BF16), UNSUPPORTED), (dict(out=INT8), UNSUPPORTED), (dict(out=XF32), UNSUPPORTED),
    (dict(xf=9), INVALID), (dict(out=9), INVALID), (dict(tiles=2), INVALID), (dict(acc=2), INVALID), (dict(acc=1), UNSUPPORTED),
    (dict(acc=1, out=FP32, bias=P), INVALID), (dict(x=0), INVALID), (dict(w=0), INVALID), (dict(ex=0), INVALID), (dict(ew=0), INVALID),
    (dict(y=0), INVALID), (dict(ldx=31), INVALID), (dict(ldw=31), INVALID), (dict(ldy=7), INVALID), (dict(ldex=0), INVALID),
    (dict(ldew=0), INVALID), (dict(y=ODD), ALIGNMENT), (dict(out=FP32, y=P + 2), ALIGNMENT), (dict(bias=P + 2), ALIGNMENT),
    (dict(x=ODD, nws=0), WORKSPACE), (dict(x=ODD, ws=0), INVALID), (dict(x=ODD, ws=P + 8), ALIGNMENT), (dict(ldw=33, nws=255), WORKSPACE),
    (dict(M=BIG), UNSUPPORTED), (dict(N=BIG, ldy=BIG), UNSUPPORTED), (dict(K=BIG, ldx=BIG, ldw=BIG, ldex=BIG, ldew=BIG), UNSUPPORTED)])
def test_linear_refusals(L, kw, status):
    assert linear(L, **kw) == status


def grouped(L, T=4, E=3, N=8, K=32, xf=E4M3, x=P, ldx=32, ex=P, ldex=1, wf=E4M3, w=P, ldw=32, sw=256, ew=P, o=P, out=BF16, y=P, ldy=8, ws=P,
            nws=1 << 40):
    return L.mcemu_fp8_grouped_linear(T, E, N, K, xf, x, ldx, ex, ldex, wf, w, ldw, sw, ew, o, out, y, ldy, ws, nws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), OK), (dict(N=0), OK), (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(E=1025), INVALID), (dict(o=0), INVALID),
    (dict(x=0), INVALID), (dict(w=0), INVALID), (dict(ex=0), INVALID), (dict(ew=0), INVALID), (dict(y=0), INVALID), (dict(sw=255), INVALID),
    (dict(ldx=31), INVALID), (dict(ldw=31), INVALID), (dict(ldy=7), INVALID), (dict(ldex=0), INVALID), (dict(xf=FP16), UNSUPPORTED),
    (dict(wf=INT8), UNSUPPORTED), (dict(out=E4M3), UNSUPPORTED), (dict(out=-1), INVALID), (dict(o=P + 2), ALIGNMENT), (dict(y=ODD), ALIGNMENT),
    (dict(sw=257, nws=0), WORKSPACE), (dict(w=ODD, ws=0), INVALID), (dict(T=BIG), UNSUPPORTED)])
def test_grouped_linear_refusals(L, kw, status):
    assert grouped(L, **kw) == status


def wgrad(L, Pc=256, E=3, N=8, K=32, df=E4M3, d=P, ldd=256, ed=P, lded=2, xf=E4M3, x=P, ldx=256, ex=P, ldex=2, o=P, out=FP32, acc=0, dW=P,
          lddw=32, sdw=256, ws=P, nws=1 << 40):
    return L.mcemu_fp8_grouped_wgrad(Pc, E, N, K, df, d, ldd, ed, lded, xf, x, ldx, ex, ldex, o, out, acc, dW, lddw, sdw, ws, nws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(N=0), OK), (dict(K=0), OK), (dict(Pc=0, d=0, x=0, acc=1), OK), (dict(Pc=-128), INVALID), (dict(Pc=255), INVALID), (dict(E=0), INVALID),
    (dict(E=1025), INVALID), (dict(o=0), INVALID), (dict(d=0), INVALID), (dict(x=0), INVALID), (dict(ed=0), INVALID), (dict(ex=0), INVALID),
    (dict(dW=0), INVALID), (dict(ldd=255), INVALID), (dict(ldx=255), INVALID), (dict(lded=1), INVALID), (dict(ldex=1), INVALID),
    (dict(lddw=31), INVALID), (dict(sdw=255), INVALID), (dict(out=INT32), UNSUPPORTED), (dict(acc=1, out=BF16), UNSUPPORTED),
    (dict(acc=3), INVALID), (dict(df=FP32), UNSUPPORTED), (dict(xf=33), INVALID), (dict(dW=P + 2), ALIGNMENT), (dict(o=ODD), ALIGNMENT),
    (dict(d=ODD, nws=0), WORKSPACE), (dict(x=ODD, nws=32 * 256 - 1), WORKSPACE), (dict(N=BIG), UNSUPPORTED)])
def test_grouped_wgrad_refusals(L, kw, status):
    assert wgrad(L, **kw) == status


def test_workspaces(L):
    """Sizes come without a device, are 0 where nothing is copied and do not wrap for large operands."""
    assert L.mcemu_fp8_linear_workspace(5, 6, 7, 1, 1) == 0 and L.mcemu_fp8_linear_workspace(0, 6, 7, 0, 0) == 0
    assert L.mcemu_fp8_linear_workspace(5, 6, 7, 0, 1) == 5 * 16 and L.mcemu_fp8_linear_workspace(5, 6, 17, 0, 0) == 11 * 32
    assert L.mcemu_fp8_grouped_linear_workspace(5, 3, 6, 7, 1, 0) == 3 * 6 * 16
    assert L.mcemu_fp8_grouped_wgrad_workspace(128, 3, 6, 7, 0, 0) == 13 * 128
    big = 2 ** 30
    assert L.mcemu_fp8_grouped_linear_workspace(big, 1024, big, 16, 0, 0) == (1 + 1024) * big * 16
    assert L.mcemu_fp8_linear_workspace(BIG, 6, 7, 0, 0) == 0


# ---------------------------------------------------------------------------
# the binding, on tensors that hold no memory
# ---------------------------------------------------------------------------
C8, BF, F32, I8, I32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int8, torch.int32


@pytest.fixture
def F(monkeypatch):
    """A call that would reach a kernel fails the test."""
    class Library:
        def __getattr__(self, name):
            return (lambda *a: 0) if name.endswith("workspace") else lambda *a: pytest.fail(f"{name} was called")

    monkeypatch.setattr(fp8, "_lib", Library())
    monkeypatch.setattr(ops, "_device", lambda where, t: -1)
    monkeypatch.setattr(ops, "_stream", lambda dev: 0)
    monkeypatch.setattr(ops, "_empty", lambda *s, dtype, device: z(*s, dt=dtype))
    monkeypatch.setattr(fp8, "_strided", lambda s, st, dtype, device: torch.empty_strided(s, st, dtype=dtype, device="meta"))
    return fp8


def z(*size, dt=BF):
    return torch.empty(*size, dtype=dt, device="meta")


@pytest.mark.parametrize("n", [2 ** 31 - 65535, 2 ** 31, 2 ** 32, 2 ** 32 + 4])
def test_sizes_beyond_32_bits_raise(F, n):
    """Not taken modulo 2^32."""
    o = z(4, dt=I32)
    calls = (lambda: F.quantize(z(n, 1)), lambda: F.quantize(z(1, n)), lambda: F.quantize_weight(z(n, 1)), lambda: F.quantize_weight(z(2, 1, n)),
             lambda: F.linear(z(n, 1, dt=C8), z(n, 1, dt=I8), z(4, 1, dt=C8), z(1, 1, dt=I8)),
             lambda: F.linear(z(4, 1, dt=C8), z(4, 1, dt=I8), z(n, 1, dt=C8), z(n, 1, dt=I8)),
             lambda: F.grouped_linear(z(n, 1, dt=C8), z(n, 1, dt=I8), z(3, 4, 1, dt=C8), z(3, 1, 1, dt=I8), o),
             lambda: F.grouped_linear(z(4, 1, dt=C8), z(4, 1, dt=I8), z(3, n, 1, dt=C8), z(3, -(-n // 128), 1, dt=I8), o),
             lambda: F.grouped_wgrad(z(n, 128, dt=C8), z(n, 1, dt=I8), z(4, 128, dt=C8), z(4, 1, dt=I8), o))
    for i, call in enumerate(calls):
        with pytest.raises(F.McemuError) as e:
            call()
        assert e.value.status == UNSUPPORTED, i


def test_a_gradient_is_not_dropped_silently(F):
    """Refused where torch records, taken where it does not."""
    g = lambda *s, dt=BF: z(*s, dt=dt).requires_grad_()
    q, e, w, ew = z(4, 8, dt=C8), z(4, 1, dt=I8), z(5, 8, dt=C8), z(1, 1, dt=I8)
    calls = (lambda: F.quantize(g(4, 8)), lambda: F.quantize_weight(g(4, 8)), lambda: F.quantize_weight(g(2, 4, 8)),
             lambda: F.linear(q, e, w, ew, bias=g(5, dt=F32)), lambda: F.linear(q, e, w, ew, out="fp32", y=g(4, 5, dt=F32)))
    for call in calls:
        with pytest.raises(F.McemuError, match="gradient"):
            call()
        with torch.no_grad(), pytest.raises(pytest.fail.Exception, match="was called"):
            call()


def test_cpu_tensors_are_refused(L):
    with pytest.raises(fp8.McemuError) as e:
        fp8.quantize(torch.zeros(2, 8))
    assert e.value.status == INVALID and "quantize" in str(e.value)
