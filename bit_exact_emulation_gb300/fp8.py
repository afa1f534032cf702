"""The FP8 layer operators of libmcemu.so (C ABI in include/mcemu_fp8.h), on torch CUDA tensors:
argument checks and marshalling only.

Operands are 8-bit floating-point codes (``torch.float8_e4m3fn`` or ``torch.float8_e5m2``) with
an exponent (int8) for each block of 128: a number is code * 2^e.  ``quantize`` makes
them from activations and gradients (blocks of 128 along a row; blocks of 128 rows of a column,
transposed), ``quantize_weight`` from weights (blocks of 128 x 128).  ``linear`` multiplies two
operands; ``grouped_linear`` rows grouped by expert, a weight for each group;
``grouped_wgrad`` gives the groups' weight gradients:

    forward             y  = linear(x, ex, w, ew)                   x, ex = quantize(x);  w, ew, wt, ewt = quantize_weight(W)
    input's gradient    dx = linear(dy, edy, wt, ewt)
    weight's gradient   dW = linear(dyt, edyt, xt, ext, out="fp32")   the columns of quantize(..., columns=True)

Groups are given as offsets [E + 1], int32 on the device: group g has the rows offsets[g] to
offsets[g + 1] - 1.  They are read by the kernels alone, so that no call waits for the device.

Conventions are those of ``ops``: matrices with contiguous rows (any row stride) on the current device,
calls on torch's current stream, ``McemuError`` for an argument that does not fit, results
and workspaces allocated by torch where they are not passed in, nothing recorded for autograd.
Codes that are allocated here have rows on 16-byte boundaries, which the products read in
place; operands with other rows are copied at every call.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding, ops
from .binding import FMT, McemuError
from .ops import _FLOATS, _F32, _FMT_OF, _MOST, _bad, _matrix, _recorded, _vector, _workspace

BLOCK = 128                      # MCEMU_FP8_BLOCK
NAN = -128                       # MCEMU_FP8_NAN: exponent of a block that is not finite
MAX_GROUPS = 1024                # MCEMU_FP8_MAX_GROUPS

_V, _I, _L, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
SYMBOLS = {
    # name: (restype, argtypes)
    "mcemu_fp8_quantize": (_I, [_I] * 4 + [_V, _L] * 5 + [_I, _V, _V]),
    "mcemu_fp8_columns": (_L, [_I] * 2),
    "mcemu_fp8_quantize_weight": (_I, [_I] * 5 + [_V, _L, _L] * 2 + [_V, _V, _L, _L, _V, _V]),
    "mcemu_fp8_linear": (_I, [_I] * 4 + [_V, _L] * 2 + [_I] + [_V, _L] * 2 + [_I, _V, _I, _I, _V, _L, _V, _Z, _V]),
    "mcemu_fp8_linear_workspace": (_Z, [_I] * 5),
    "mcemu_fp8_grouped_linear": (_I, [_I] * 5 + [_V, _L] * 2 + [_I, _V, _L, _L, _V, _V, _I, _V, _L, _V, _Z, _V]),
    "mcemu_fp8_grouped_linear_workspace": (_Z, [_I] * 6),
    "mcemu_fp8_grouped_wgrad": (_I, [_I] * 5 + [_V, _L] * 2 + [_I] + [_V, _L] * 2 + [_V, _I, _I, _V, _L, _L, _V, _Z, _V]),
    "mcemu_fp8_grouped_wgrad_workspace": (_Z, [_I] * 6),
    "mcemu_fp8_check": (_I, [_V]),
}
_CODE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_CODE_FMT = {torch.float8_e4m3fn: FMT["e4m3"], torch.float8_e5m2: FMT["e5m2"]}
_CODES = tuple(_CODE_FMT)
_OUT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
_I8 = (torch.int8,)
_I32 = (torch.int32,)
_lib = None


def lib():
    """The loaded library with these operators' signatures; raises when it has not been built."""
    global _lib
    if _lib is None:
        L = binding.lib()
        for name, (res, args) in SYMBOLS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


_strided = torch.empty_strided


def _codes(shape, dtype, dev):
    """(new codes whose rows start on 16-byte boundaries, their pointer and row stride)."""
    cols = shape[-1]
    if cols % 16 == 0:
        t = ops._empty(shape, dtype=dtype, device=dev)
        return t, t.data_ptr(), cols
    ld = (cols + 15) // 16 * 16
    t = _strided(shape, (ld, 1) if len(shape) == 2 else (shape[1] * ld, ld, 1), dtype=dtype, device=dev)
    return t, t.data_ptr(), ld


def _matrices(where, name, t, dtypes, dev, shape=None):
    """Data pointer, row stride and stride between matrices of a 3-D tensor on the current device."""
    size = t.shape
    if len(size) != 3 or t.dtype not in dtypes or t.get_device() != dev:
        _bad(where, f"{name} must be a 3-D tensor of {' or '.join(map(str, dtypes))} on the current device (cuda:{dev})")
    if shape is not None and size != shape:
        _bad(where, f"{name} must have the shape {tuple(shape)}")
    if t.requires_grad:
        _recorded(where, name)
    E, rows, cols = size
    if rows > _MOST or cols > _MOST:
        raise McemuError(2, f"{where}: {name} has more than {_MOST} rows or columns")
    if E < 1 or E > MAX_GROUPS:
        _bad(where, f"{name} must have 1 to {MAX_GROUPS} matrices")
    stride, ld, one = t.stride()
    if rows <= 1:
        ld = cols
    if E == 1:
        stride = rows * ld
    if (one != 1 and cols > 1) or ld < cols or stride < (rows - 1) * ld + cols:
        _bad(where, f"{name} must have contiguous rows that do not overlap")
    return t.data_ptr(), ld, stride


def _dense(where, name, t, shape, dev):
    """Data pointer of contiguous exponents."""
    if t.shape != shape or t.dtype != torch.int8 or t.get_device() != dev or not t.is_contiguous():
        _bad(where, f"{name} must be a contiguous torch.int8 tensor of shape {tuple(shape)} on the current device (cuda:{dev})")
    return t.data_ptr()


def _offsets(where, offsets, dev, groups=None):
    """(pointer, groups) of the groups' offsets."""
    if offsets.dim() != 1 or not 2 <= offsets.shape[0] <= MAX_GROUPS + 1 or (groups is not None and offsets.shape[0] != groups + 1):
        _bad(where, f"offsets must have {'2 to ' + str(MAX_GROUPS + 1) if groups is None else groups + 1} entries, one more than groups")
    return _vector(where, "offsets", offsets, _I32, dev, offsets.shape[0]), offsets.shape[0] - 1


def columns(T: int, groups: int = 1) -> int:
    """Columns of the transposed codes of T rows in that many groups: a multiple of 128."""
    return (T + 127 * max(groups, 1)) // BLOCK * BLOCK


def quantize(x, out: str = "e4m3", rows: bool = True, columns: bool = False, offsets=None, q=None, e=None, qt=None, et=None):
    """(q, e, qt, et) of x [T, H], H at least 1; what is not asked for is None.

    ``rows``: q [T, H] and e [T, ceil(H / 128)], blocks of 128 along each row.
    ``columns``: the transposed codes qt [H, P] and et [H, P / 128], blocks of 128 rows of each
    column, P = ``columns(T, groups)``.  With ``offsets`` each group of rows begins a block; places
    that no row fills are zeros, and rows outside all groups are left out.
    ``out`` is "e4m3" or "e5m2" (OCP).  A block with a NaN or an infinity reads back as NaN."""
    w = "quantize"
    dev = ops._device(w, x)
    px, ldx = _matrix(w, "x", x, _FLOATS, dev)
    T, H = x.shape
    if out not in _CODE:
        _bad(w, "out must be 'e4m3' or 'e5m2'")
    if not rows and not columns:
        _bad(w, "rows, columns or both must be asked for")
    code = _CODE[out]
    pq = ldq = pe = lde = pqt = ldqt = pet = ldet = po = E = 0
    if offsets is not None:
        po, E = _offsets(w, offsets, dev)
    if rows:
        if q is None:
            q, pq, ldq = _codes((T, H), code, dev)
        else:
            pq, ldq = _matrix(w, "q", q, (code,), dev, (T, H))
        if e is None:
            lde = _blocks(H)
            e = ops._empty((T, lde), dtype=torch.int8, device=dev)
            pe = e.data_ptr()
        else:
            pe, lde = _matrix(w, "e", e, _I8, dev, (T, _blocks(H)))
    elif q is not None or e is not None:
        _bad(w, "q and e are written only with rows")
    if columns:
        P = (T + 127 * max(E, 1)) // BLOCK * BLOCK
        if qt is None:
            qt = ops._empty((H, P), dtype=code, device=dev)
            pqt, ldqt = qt.data_ptr(), P
        else:
            pqt, ldqt = _matrix(w, "qt", qt, (code,), dev, (H, P))
        if et is None:
            et = ops._empty((H, P // BLOCK), dtype=torch.int8, device=dev)
            pet, ldet = et.data_ptr(), P // BLOCK
        else:
            pet, ldet = _matrix(w, "et", et, _I8, dev, (H, P // BLOCK))
        if P == 0:
            pqt = pet = 0
    elif qt is not None or et is not None:
        _bad(w, "qt and et are written only with columns")
    if T == 0 and not pqt:
        return q, e, qt, et
    st = (_lib or lib()).mcemu_fp8_quantize(_FMT_OF[x.dtype], FMT[out], T, H, px, ldx, pq if T else 0, ldq, pe if T else 0, lde, pqt, ldqt,
                                            pet, ldet, E, po, ops._stream(dev))
    if st:
        raise McemuError(st, w)
    return q, e, qt, et


def quantize_weight(weight, out: str = "e4m3", transposed: bool = False, q=None, e=None, qt=None, et=None):
    """(q, e, qt, et) of a weight [N, K], or [E, N, K] for E experts, in blocks of 128 x 128: q like the
    weight and e [.., ceil(N / 128), ceil(K / 128)]; with ``transposed`` the same numbers as qt
    [.., K, N] and et [.., ceil(K / 128), ceil(N / 128)] (None otherwise)."""
    w = "quantize_weight"
    dev = ops._device(w, weight)
    if weight.dim() == 2:
        one = lambda t: None if t is None else t.unsqueeze(0)
        got = quantize_weight(weight.unsqueeze(0), out, transposed, one(q), one(e), one(qt), one(et))
        return tuple(None if t is None else t[0] for t in got)
    pw, ldw, sw = _matrices(w, "weight", weight, _FLOATS, dev)
    E, N, K = weight.shape
    if out not in _CODE:
        _bad(w, "out must be 'e4m3' or 'e5m2'")
    code = _CODE[out]
    if q is None:
        q, pq, ldq = _codes((E, N, K), code, dev)
        sq = N * ldq
    else:
        pq, ldq, sq = _matrices(w, "q", q, (code,), dev, (E, N, K))
    shape = E, _blocks(N), _blocks(K)
    if e is None:
        e = ops._empty(shape, dtype=torch.int8, device=dev)
        pe = e.data_ptr()
    else:
        pe = _dense(w, "e", e, shape, dev)
    pqt = ldqt = sqt = pet = 0
    if transposed:
        if qt is None:
            qt, pqt, ldqt = _codes((E, K, N), code, dev)
            sqt = K * ldqt
        else:
            pqt, ldqt, sqt = _matrices(w, "qt", qt, (code,), dev, (E, K, N))
        shape = E, _blocks(K), _blocks(N)
        if et is None:
            et = ops._empty(shape, dtype=torch.int8, device=dev)
            pet = et.data_ptr()
        else:
            pet = _dense(w, "et", et, shape, dev)
    elif qt is not None or et is not None:
        _bad(w, "qt and et are written only when transposed")
    if N == 0 or K == 0:
        return q, e, qt, et
    st = (_lib or lib()).mcemu_fp8_quantize_weight(_FMT_OF[weight.dtype], FMT[out], E, N, K, pw, ldw, sw, pq, ldq, sq, pe, pqt, ldqt, sqt, pet,
                                                   ops._stream(dev))
    if st:
        raise McemuError(st, w)
    return q, e, qt, et


def linear(x, ex, weight, ew, bias=None, out: str = "bf16", y=None, accumulate: bool = False, workspace=None):
    """y [M, N] = (x * 2^ex) @ (weight * 2^ew).T + bias: x [M, K] with ex [M, ceil(K / 128)]; weight
    [N, K] with ew [ceil(N / 128), ceil(K / 128)] (``quantize_weight``) or [N, ceil(K / 128)]
    (``quantize``).  Sums are held in fp32.  ``out`` is "bf16", "fp16" or "fp32"; with
    ``accumulate`` the product is added to y (fp32, no bias)."""
    w = "linear"
    dev = ops._device(w, x)
    px, ldx = _matrix(w, "x", x, _CODES, dev)
    pw, ldw = _matrix(w, "weight", weight, _CODES, dev)
    M, K = x.shape
    N, k = weight.shape
    if k != K:
        _bad(w, f"weight must have {K} columns")
    blocks = (K + BLOCK - 1) // BLOCK
    pex, ldex = _matrix(w, "ex", ex, _I8, dev, (M, blocks))
    tiles = ew.shape != (N, blocks)
    pew, ldew = _matrix(w, "ew", ew, _I8, dev, ((N + BLOCK - 1) // BLOCK if tiles else N, blocks))
    pb = None if bias is None else _vector(w, "bias", bias, _F32, dev, N)
    if out not in _OUT or (accumulate and (out != "fp32" or y is None or bias is not None)):
        _bad(w, "out must be 'bf16', 'fp16' or 'fp32'; accumulate adds to an fp32 y that is passed in, without a bias")
    if y is None:
        y = ops._empty((M, N), dtype=_OUT[out], device=dev)
        py, ldy = y.data_ptr(), N
    else:
        py, ldy = _matrix(w, "y", y, (_OUT[out],), dev, (M, N))
    L = _lib or lib()
    xr, wr = (px | (ldx if M != 1 else 0)) % 16 == 0, (pw | (ldw if N != 1 else 0)) % 16 == 0
    ws, pws, nws = (None, None, 0) if xr and wr else _workspace(w, L.mcemu_fp8_linear_workspace(M, N, K, xr, wr), dev, workspace)
    st = L.mcemu_fp8_linear(M, N, K, _CODE_FMT[x.dtype], px, ldx, pex, ldex, _CODE_FMT[weight.dtype], pw, ldw, pew, ldew, tiles, pb,
                            FMT[out], accumulate, py, ldy, pws, nws, ops._stream(dev))
    if st:
        raise McemuError(st, w)
    return y


def grouped_linear(x, ex, weight, ew, offsets, out: str = "bf16", y=None, workspace=None):
    """y [T, N]: for the rows t of each group g, y[t] = (x[t] * 2^ex[t]) @ (weight[g] * 2^ew[g]).T.
    x [T, K] with ex [T, ceil(K / 128)]; weight [E, N, K] with ew [E, ceil(N / 128),
    ceil(K / 128)]; offsets [E + 1].  Rows outside all groups are left as they are (in a y that
    is allocated here: not initialised)."""
    w = "grouped_linear"
    dev = ops._device(w, x)
    px, ldx = _matrix(w, "x", x, _CODES, dev)
    pw, ldw, sw = _matrices(w, "weight", weight, _CODES, dev)
    T, K = x.shape
    E, N, k = weight.shape
    if k != K:
        _bad(w, f"weight must have {K} columns")
    blocks = (K + BLOCK - 1) // BLOCK
    pex, ldex = _matrix(w, "ex", ex, _I8, dev, (T, blocks))
    pew = _dense(w, "ew", ew, (E, (N + BLOCK - 1) // BLOCK, blocks), dev)
    po, _ = _offsets(w, offsets, dev, E)
    if out not in _OUT:
        _bad(w, "out must be 'bf16', 'fp16' or 'fp32'")
    if y is None:
        y = ops._empty((T, N), dtype=_OUT[out], device=dev)
        py, ldy = y.data_ptr(), N
    else:
        py, ldy = _matrix(w, "y", y, (_OUT[out],), dev, (T, N))
    L = _lib or lib()
    xr, wr = (px | (ldx if T != 1 else 0)) % 16 == 0, (pw | (ldw if N != 1 else 0) | (sw if E > 1 else 0)) % 16 == 0
    ws, pws, nws = (None, None, 0) if xr and wr else _workspace(w, L.mcemu_fp8_grouped_linear_workspace(T, E, N, K, xr, wr), dev, workspace)
    st = L.mcemu_fp8_grouped_linear(T, E, N, K, _CODE_FMT[x.dtype], px, ldx, pex, ldex, _CODE_FMT[weight.dtype], pw, ldw, sw, pew, po,
                                    FMT[out], py, ldy, pws, nws, ops._stream(dev))
    if st:
        raise McemuError(st, w)
    return y


def grouped_wgrad(dyt, edyt, xt, ext, offsets, out: str = "fp32", dW=None, accumulate: bool = False, workspace=None):
    """dW [E, N, K]: for each group g the sum over its rows t of dy[t][n] * x[t][k].  dyt [N, P], edyt and
    xt [K, P], ext are what ``quantize`` gives with columns=True and the same offsets.  A group
    without rows gets zeros.  ``out`` is "fp32", "bf16" or "fp16"; with ``accumulate`` it is added to
    dW (fp32)."""
    w = "grouped_wgrad"
    dev = ops._device(w, dyt)
    pd, ldd = _matrix(w, "dyt", dyt, _CODES, dev)
    px, ldx = _matrix(w, "xt", xt, _CODES, dev)
    N, P = dyt.shape
    K, p = xt.shape
    if p != P or P % BLOCK:
        _bad(w, f"dyt and xt must have the same columns, a multiple of {BLOCK}")
    ped, lded = _matrix(w, "edyt", edyt, _I8, dev, (N, P // BLOCK))
    pex, ldex = _matrix(w, "ext", ext, _I8, dev, (K, P // BLOCK))
    po, E = _offsets(w, offsets, dev)
    if out not in _OUT or (accumulate and (out != "fp32" or dW is None)):
        _bad(w, "out must be 'bf16', 'fp16' or 'fp32'; accumulate adds to an fp32 dW that is passed in")
    if dW is None:
        dW = ops._empty((E, N, K), dtype=_OUT[out], device=dev)
        pw, ldw, sw = dW.data_ptr(), K, N * K
    else:
        pw, ldw, sw = _matrices(w, "dW", dW, (_OUT[out],), dev, (E, N, K))
    L = _lib or lib()
    dr, xr = (pd | ldd) % 16 == 0, (px | ldx) % 16 == 0
    ws, pws, nws = (None, None, 0) if xr and dr else _workspace(w, L.mcemu_fp8_grouped_wgrad_workspace(P, E, N, K, dr, xr), dev, workspace)
    st = L.mcemu_fp8_grouped_wgrad(P, E, N, K, _CODE_FMT[dyt.dtype], pd, ldd, ped, lded, _CODE_FMT[xt.dtype], px, ldx, pex, ldex, po,
                                   FMT[out], accumulate, pw, ldw, sw, pws, nws, ops._stream(dev))
    if st:
        raise McemuError(st, w)
    return dW


def check():
    """Waits for the current stream; raises (status 6) when a bounded wait inside one of these
    products' kernels gave up since the last call, which leaves that launch's results invalid."""
    st = (_lib or lib()).mcemu_fp8_check(ops._stream(torch.cuda.current_device()))
    if st:
        raise McemuError(st, "check")
