"""The 8-bit layer operators of libmcemu.so (C ABI in include/mcemu_ops.h), on torch CUDA
tensors: argument checks and marshalling only.

``rmsnorm`` turns a residual stream into 8-bit operands with a scale for each token;
``int8_linear`` multiplies such operands by 8-bit weights with a scale for each channel;
``act8_compress`` keeps an activation for the backward pass in 8 bits, and ``act8_wgrad`` and
``rmsnorm_backward`` compute gradients from it.  Matrices are two-dimensional with contiguous
rows (any row stride).  Calls run on torch's current CUDA stream and return before the work
finishes.  An argument that does not fit raises ``McemuError`` and nothing runs.  Results and
workspaces that are not passed in are allocated by torch.  There is no fallback when the
library is missing.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding
from .binding import FMT, McemuError

ACT8_BLOCK = 128                 # MCEMU_ACT8_BLOCK: elements of a row that share an exponent
ACT8_NAN = -128                  # MCEMU_ACT8_NAN: exponent of a block that is not finite
INT32 = 8                        # MCEMU_INT32

_V, _I, _L, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
SYMBOLS = {
    # name: (restype, argtypes)
    "mcemu_rmsnorm": (_I, [_I] * 5 + [_V, _L, _V, _L, _V, ctypes.c_float, _V, _L, _V, _L, _V, _V, _V]),
    "mcemu_rmsnorm_backward": (_I, [_I] * 4 + [_V, _L] * 5 + [_V, _V, _V, _L, _V, _V, _Z, _V]),
    "mcemu_rmsnorm_backward_workspace": (_Z, [_I] * 2),
    "mcemu_int8_linear": (_I, [_I] * 3 + [_V, _L, _V, _V, _L, _V, _V, _I, _V, _L, _V, _Z, _V]),
    "mcemu_int8_linear_workspace": (_Z, [_I] * 3),
    "mcemu_act8_compress": (_I, [_I] * 3 + [_V, _L] * 3 + [_V]),
    "mcemu_act8_expand": (_I, [_I] * 3 + [_V, _L] * 3 + [_V]),
    "mcemu_act8_wgrad": (_I, [_I] * 3 + [_V, _L] * 3 + [_I, _I, _V, _L, _V, _Z, _V]),
    "mcemu_act8_wgrad_workspace": (_Z, [_I] * 4),
    "mcemu_ops_check": (_I, [_V]),
}
_FMT_OF = {torch.float16: FMT["fp16"], torch.bfloat16: FMT["bf16"], torch.float32: FMT["fp32"]}
_OUT = {"int8": (FMT["int8"], torch.int8), "e4m3": (FMT["e4m3"], torch.float8_e4m3fn),
        "e5m2": (FMT["e5m2"], torch.float8_e5m2)}
_DTYPE = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32, "int32": torch.int32}
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


def _bad(where: str, why: str):
    raise McemuError(1, f"{where}: {why}")


def _matrix(where, name, t, dtypes, shape=None):
    """Data pointer and row stride of a matrix whose rows are contiguous."""
    if t.dim() != 2 or t.dtype not in dtypes or not t.is_cuda:
        _bad(where, f"{name} must be a 2-D CUDA tensor of {' or '.join(str(d) for d in dtypes)}")
    if shape is not None and tuple(t.shape) != shape:
        _bad(where, f"{name} must have the shape {shape}")
    rows, cols = t.shape
    ld = t.stride(0) if rows > 1 else cols
    if (cols > 1 and t.stride(1) != 1) or ld < cols:
        _bad(where, f"{name} must have contiguous rows that do not overlap")
    return t.data_ptr(), ld


def _vector(where, name, t, dtypes, n):
    if t.dim() != 1 or t.shape[0] != n or t.dtype not in dtypes or not t.is_cuda or (n > 1 and t.stride(0) != 1):
        _bad(where, f"{name} must be a contiguous CUDA vector of {n} {' or '.join(str(d) for d in dtypes)}")
    return t.data_ptr()


def _same_device(where, *tensors):
    """The current stream, once every tensor is known to lie on its device."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.device.index != dev:
            _bad(where, f"tensors must be on the current device (cuda:{dev})")
    return torch.cuda.current_stream().cuda_stream


def _run(where, name, *args):
    st = getattr(lib(), name)(*args)
    if st:
        raise McemuError(st, where)


def _workspace(need, like, workspace):
    if need == 0:
        return None, None, 0
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=like.device)
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


_FLOATS = tuple(_FMT_OF)
_F32 = (torch.float32,)
_I8 = (torch.int8,)


def rmsnorm(x, weight, eps: float, residual=None, out: str = "int8", y=None, scale=None, rstd=None, h=None):
    """(y, scale, rstd, h): the root-mean-square norm of h = x + residual (or x) along its rows.

    ``out`` is "int8", "e4m3" or "e5m2" (OCP): y holds 8-bit values and y * scale[:, None] is the
    norm; or "own": y has x's type and scale is None.  h is None without a residual; it may
    be passed as x or residual to add in place.  rstd [T] is what ``rmsnorm_backward`` takes."""
    w = "rmsnorm"
    px, ldx = _matrix(w, "x", x, _FLOATS)
    T, H = x.shape
    if out != "own" and out not in _OUT:
        _bad(w, "out must be 'int8', 'e4m3', 'e5m2' or 'own'")
    fmt = _FMT_OF[x.dtype]
    out_fmt, out_dtype = _OUT.get(out, (fmt, x.dtype))
    dev = x.device
    pw = _vector(w, "weight", weight, (x.dtype, torch.float32), H)
    pr = ldr = ph = ldh = ps = 0
    if residual is not None:
        pr, ldr = _matrix(w, "residual", residual, (x.dtype,), (T, H))
        if h is None:
            h = torch.empty((T, H), dtype=x.dtype, device=dev)
        ph, ldh = _matrix(w, "h", h, (x.dtype,), (T, H))
    elif h is not None:
        _bad(w, "h is written only with a residual")
    if y is None:
        y = torch.empty((T, H), dtype=out_dtype, device=dev)
    py, ldy = _matrix(w, "y", y, (out_dtype,), (T, H))
    if out == "own":
        if scale is not None:
            _bad(w, "scale is written only for 8-bit outputs")
    else:
        if scale is None:
            scale = torch.empty(T, dtype=torch.float32, device=dev)
        ps = _vector(w, "scale", scale, _F32, T)
    if rstd is None:
        rstd = torch.empty(T, dtype=torch.float32, device=dev)
    pd = _vector(w, "rstd", rstd, _F32, T)
    st = _same_device(w, x, weight, residual, h, y, scale, rstd)
    _run(w, "mcemu_rmsnorm", fmt, _FMT_OF[weight.dtype], out_fmt, T, H, px, ldx, pr, ldr, pw, eps, ph, ldh, py, ldy,
         ps, pd, st)
    return y, scale, rstd, h


def rmsnorm_backward(dy, weight, rstd, h=None, ckpt=None, dres=None, dx=None, dw=None, workspace=None):
    """(dx, dw): gradients of the norm's input (dres, the residual path's gradient, added) and
    of its weight (fp32).  The input is given as h or as a checkpoint ckpt = (q, e)."""
    w = "rmsnorm_backward"
    pdy, lddy = _matrix(w, "dy", dy, _FLOATS)
    T, H = dy.shape
    if (h is None) == (ckpt is None):
        _bad(w, "the norm's input is given as h or as ckpt")
    pw = _vector(w, "weight", weight, (dy.dtype, torch.float32), H)
    prs = _vector(w, "rstd", rstd, _F32, T)
    ph = ldh = pq = ldq = pe = lde = pr = ldr = 0
    q = e = None
    if h is not None:
        ph, ldh = _matrix(w, "h", h, (dy.dtype,), (T, H))
    else:
        q, e = ckpt
        pq, ldq, pe, lde = _ckpt(w, q, e, T, H)
    if dres is not None:
        pr, ldr = _matrix(w, "dres", dres, (dy.dtype,), (T, H))
    if dx is None:
        dx = torch.empty((T, H), dtype=dy.dtype, device=dy.device)
    pdx, lddx = _matrix(w, "dx", dx, (dy.dtype,), (T, H))
    if dw is None:
        dw = torch.empty(H, dtype=torch.float32, device=dy.device)
    pdw = _vector(w, "dw", dw, _F32, H)
    ws, pws, nws = _workspace(lib().mcemu_rmsnorm_backward_workspace(T, H), dy, workspace)
    st = _same_device(w, dy, weight, rstd, h, q, e, dres, dx, dw, ws)
    _run(w, "mcemu_rmsnorm_backward", _FMT_OF[dy.dtype], _FMT_OF[weight.dtype], T, H, pdy, lddy, pr, ldr, ph, ldh, pq,
         ldq, pe, lde, prs, pw, pdx, lddx, pdw, pws, nws, st)
    return dx, dw


def int8_linear(x, sx, weight, sw, bias=None, out: str = "bf16", y=None, workspace=None):
    """y = (x @ weight.T) * sx[:, None] * sw + bias, x [M, K] and weight [N, K] int8, the sums
    exact.  ``out`` is "bf16", "fp16" or "fp32"; "int32" gives the sums themselves (sx, sw and
    bias None)."""
    w = "int8_linear"
    px, ldx = _matrix(w, "x", x, _I8)
    M, K = x.shape
    pw, ldw = _matrix(w, "weight", weight, _I8)
    N = weight.shape[0]
    if weight.shape[1] != K:
        _bad(w, f"weight must have {K} columns")
    if out not in _DTYPE:
        _bad(w, "out must be 'bf16', 'fp16', 'fp32' or 'int32'")
    psx = psw = pb = None
    if out == "int32":
        if sx is not None or sw is not None or bias is not None:
            _bad(w, "sums in int32 take neither scales nor a bias")
    else:
        if sx is None or sw is None:
            _bad(w, "scales are missing")
        psx, psw = _vector(w, "sx", sx, _F32, M), _vector(w, "sw", sw, _F32, N)
        if bias is not None:
            pb = _vector(w, "bias", bias, _F32, N)
    dt = _DTYPE[out]
    if y is None:
        y = torch.empty((M, N), dtype=dt, device=x.device)
    py, ldy = _matrix(w, "y", y, (dt,), (M, N))
    ws, pws, nws = _workspace(lib().mcemu_int8_linear_workspace(M, N, K), x, workspace)
    st = _same_device(w, x, weight, sx, sw, bias, y, ws)
    _run(w, "mcemu_int8_linear", M, N, K, px, ldx, psx, pw, ldw, psw, pb, INT32 if out == "int32" else FMT[out], py, ldy,
         pws, nws, st)
    return y


def _ckpt(where, q, e, T, H):
    pq, ldq = _matrix(where, "q", q, _I8, (T, H))
    pe, lde = _matrix(where, "e", e, _I8, (T, -(-H // ACT8_BLOCK)))
    return pq, ldq, pe, lde


def act8_compress(x, q=None, e=None):
    """(q, e): int8 codes [T, H] and exponents [T, ceil(H / 128)] with x ~ q * 2^e."""
    w = "act8_compress"
    px, ldx = _matrix(w, "x", x, _FLOATS)
    T, H = x.shape
    if q is None:
        q = torch.empty((T, H), dtype=torch.int8, device=x.device)
    if e is None:
        e = torch.empty((T, -(-H // ACT8_BLOCK)), dtype=torch.int8, device=x.device)
    pq, ldq, pe, lde = _ckpt(w, q, e, T, H)
    st = _same_device(w, x, q, e)
    _run(w, "mcemu_act8_compress", _FMT_OF[x.dtype], T, H, px, ldx, pq, ldq, pe, lde, st)
    return q, e


def act8_expand(q, e, out: str = "bf16", x=None):
    """q * 2^e in "bf16", "fp16" or "fp32"."""
    w = "act8_expand"
    if q.dim() != 2 or out not in ("bf16", "fp16", "fp32"):
        _bad(w, "q must be a matrix and out 'bf16', 'fp16' or 'fp32'")
    T, H = q.shape
    pq, ldq, pe, lde = _ckpt(w, q, e, T, H)
    if x is None:
        x = torch.empty((T, H), dtype=_DTYPE[out], device=q.device)
    px, ldx = _matrix(w, "x", x, (_DTYPE[out],), (T, H))
    st = _same_device(w, q, e, x)
    _run(w, "mcemu_act8_expand", FMT[out], T, H, pq, ldq, pe, lde, px, ldx, st)
    return x


def act8_wgrad(dy, q, e, out: str = "fp32", dW=None, accumulate: bool = False, workspace=None):
    """dW [N, K] = dy.T @ (q * 2^e): the gradient of a linear layer's weight from dy [T, N]
    (bfloat16) and the checkpoint of its input [T, K].  With ``accumulate`` it is added to
    dW (fp32)."""
    w = "act8_wgrad"
    pdy, lddy = _matrix(w, "dy", dy, (torch.bfloat16,))
    T, N = dy.shape
    if q.dim() != 2 or q.shape[0] != T:
        _bad(w, f"q must be a matrix of {T} rows")
    K = q.shape[1]
    pq, ldq, pe, lde = _ckpt(w, q, e, T, K)
    if out not in ("bf16", "fp32") or (accumulate and (out != "fp32" or dW is None)):
        _bad(w, "out must be 'bf16' or 'fp32'; accumulate adds to an fp32 dW that is passed in")
    if dW is None:
        dW = torch.empty((N, K), dtype=_DTYPE[out], device=dy.device)
    pd, ldd = _matrix(w, "dW", dW, (_DTYPE[out],), (N, K))
    ws, pws, nws = _workspace(lib().mcemu_act8_wgrad_workspace(T, N, K, int(pdy % 16 == 0 and lddy % 8 == 0)), dy,
                             workspace)
    st = _same_device(w, dy, q, e, dW, ws)
    _run(w, "mcemu_act8_wgrad", T, N, K, pdy, lddy, pq, ldq, pe, lde, FMT[out], int(bool(accumulate)), pd, ldd, pws,
         nws, st)
    return dW


def check():
    """Waits for the current stream; raises (status 6) when a bounded wait inside one of the
    product kernels gave up since the last call, which leaves that launch's results invalid."""
    _run("check", "mcemu_ops_check", torch.cuda.current_stream().cuda_stream)
