"""The 8-bit layer operators of libmcemu.so (C ABI in include/mcemu_ops.h), on torch CUDA
tensors: argument checks and marshalling only.

``rmsnorm`` turns a residual stream into 8-bit operands with a scale for each token;
``int8_linear`` multiplies such operands by 8-bit weights with a scale for each channel;
``act8_compress`` keeps an activation for the backward pass in 8 bits, and ``act8_wgrad`` and
``rmsnorm_backward`` compute gradients from it.  Matrices are two-dimensional with contiguous
rows (any row stride).  Calls run on torch's current CUDA stream and return before the work
finishes.  An argument that does not fit raises ``McemuError`` and nothing runs.  Results and
workspaces that are not passed in are allocated by torch.  Nothing is recorded for autograd:
gradients are calls of their own, and a tensor that requires one is refused while torch
records.  There is no fallback when the library is missing.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding
from .binding import FMT, McemuError

ACT8_BLOCK = 128                 # MCEMU_ACT8_BLOCK: elements of a row that share an exponent
ACT8_NAN = -128                  # MCEMU_ACT8_NAN: exponent of a block that is not finite
INT32 = 8                        # MCEMU_INT32
_MOST = 2 ** 31 - 65536          # of any size; ctypes would take a larger one modulo 2^32

_V, _I, _L, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
SYMBOLS = {
    # name: (restype, argtypes)
    "mcemu_rmsnorm": (_I, [_I] * 5 + [_V, _L, _V, _L, _V, ctypes.c_float, _V, _L, _V, _L, _V, _V, _V]),
    "mcemu_rmsnorm_backward": (_I, [_I] * 4 + [_V, _L] * 5 + [_V, _V, _V, _L, _V, _V, _Z, _V]),
    "mcemu_rmsnorm_backward_workspace": (_Z, [_I] * 2),
    "mcemu_int8_linear": (_I, [_I] * 3 + [_V, _L, _V, _V, _L, _V, _V, _I, _V, _L, _V, _Z, _V]),
    "mcemu_int8_linear_workspace": (_Z, [_I] * 4),
    "mcemu_act8_compress": (_I, [_I] * 3 + [_V, _L] * 3 + [_V]),
    "mcemu_act8_expand": (_I, [_I] * 3 + [_V, _L] * 3 + [_V]),
    "mcemu_act8_wgrad": (_I, [_I] * 3 + [_V, _L] * 3 + [_I, _I, _V, _L, _V, _Z, _V]),
    "mcemu_act8_wgrad_workspace": (_Z, [_I] * 4),
    "mcemu_ops_check": (_I, [_V]),
}
_FMT_OF = {torch.float16: FMT["fp16"], torch.bfloat16: FMT["bf16"], torch.float32: FMT["fp32"]}
_OUT = {"int8": (FMT["int8"], torch.int8), "e4m3": (FMT["e4m3"], torch.float8_e4m3fn),
        "e5m2": (FMT["e5m2"], torch.float8_e5m2)}
_LINEAR_OUT = {"fp16": FMT["fp16"], "bf16": FMT["bf16"], "fp32": FMT["fp32"], "int32": INT32}
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


_empty = torch.empty


def _bad(where: str, why: str):
    raise McemuError(1, f"{where}: {why}")


def _device(where, t):
    """The current device, on which `t` must be."""
    dev = t.get_device()
    if dev < 0 or dev != _current():
        _bad(where, "tensors must be on the current CUDA device")
    return dev


_current = torch.cuda.current_device
if hasattr(torch._C, "_cuda_getDevice"):                # the same number, 1 us sooner
    _current = torch._C._cuda_getDevice


def _stream(dev):
    """Torch's current stream on its current device, as the C ABI takes it."""
    return torch.cuda.current_stream(dev).cuda_stream


if hasattr(torch._C, "_cuda_getCurrentRawStream"):       # the same number, 3 us sooner
    _stream = torch._C._cuda_getCurrentRawStream


def _recorded(where, name):
    """What autograd would lose: called for a tensor that requires a gradient."""
    if torch.is_grad_enabled():
        _bad(where, f"{name} requires a gradient, which this call does not record: detach it, or call under torch.no_grad() "
                    f"or from an autograd.Function")


def _matrix(where, name, t, dtypes, dev, shape=None):
    """Data pointer and row stride of a matrix on the current device whose rows are contiguous."""
    size = t.shape
    if len(size) != 2 or t.dtype not in dtypes or t.get_device() != dev:
        _bad(where, f"{name} must be a 2-D tensor of {' or '.join(map(str, dtypes))} on the current device (cuda:{dev})")
    if shape is not None and size != shape:
        _bad(where, f"{name} must have the shape {tuple(shape)}")
    if t.requires_grad:
        _recorded(where, name)
    rows, cols = size
    if rows > _MOST or cols > _MOST:
        raise McemuError(2, f"{where}: {name} has more than {_MOST} rows or columns")
    ld, one = t.stride()
    if rows <= 1:
        ld = cols
    if (one != 1 and cols > 1) or ld < cols:
        _bad(where, f"{name} must have contiguous rows that do not overlap")
    return t.data_ptr(), ld


def _vector(where, name, t, dtypes, dev, n):
    if t.shape != (n,) or t.dtype not in dtypes or t.get_device() != dev or (n > 1 and t.stride(0) != 1):
        _bad(where, f"{name} must be a contiguous vector of {n} {' or '.join(map(str, dtypes))} on the current device "
                    f"(cuda:{dev})")
    if t.requires_grad:
        _recorded(where, name)
    return t.data_ptr()


def _workspace(where, need, dev, workspace):
    """(tensor to keep until the launch, pointer, bytes) of the caller's workspace or a new one."""
    if need == 0:
        return None, None, 0
    if workspace is None:
        workspace = _empty(need, dtype=torch.uint8, device=dev)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        _bad(where, f"workspace must be contiguous and on the current device (cuda:{dev})")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _ckpt(where, q, e, dev, T, H):
    pq, ldq = _matrix(where, "q", q, _I8, dev, (T, H))
    pe, lde = _matrix(where, "e", e, _I8, dev, (T, (H + ACT8_BLOCK - 1) // ACT8_BLOCK))
    return pq, ldq, pe, lde


_FLOATS = tuple(_FMT_OF)
_F32 = (torch.float32,)
_I8 = (torch.int8,)
_BF16 = (torch.bfloat16,)


def rmsnorm(x, weight, eps: float, residual=None, out: str = "int8", y=None, scale=None, rstd=None, h=None):
    """(y, scale, rstd, h): the root-mean-square norm of h = x + residual (or x) along its rows.

    ``out`` is "int8", "e4m3" or "e5m2" (OCP): y holds 8-bit values and y * scale[:, None] is the
    norm; or "own": y has x's type and scale is None.  h is None without a residual; it may
    be passed as x or residual to add in place.  rstd [T] is what ``rmsnorm_backward`` takes."""
    w = "rmsnorm"
    dev = _device(w, x)
    dtype = x.dtype
    px, ldx = _matrix(w, "x", x, _FLOATS, dev)
    size = T, H = x.shape
    fmt = _FMT_OF[dtype]
    if out == "own":
        out_fmt, out_dtype = fmt, dtype
    elif out in _OUT:
        out_fmt, out_dtype = _OUT[out]
    else:
        _bad(w, "out must be 'int8', 'e4m3', 'e5m2' or 'own'")
    pw = _vector(w, "weight", weight, (dtype, torch.float32), dev, H)
    pr = ldr = ph = ldh = ps = 0
    if residual is not None:
        pr, ldr = _matrix(w, "residual", residual, (dtype,), dev, size)
        if h is None:
            h = _empty(size, dtype=dtype, device=dev)
            ph, ldh = h.data_ptr(), H
        else:
            ph, ldh = _matrix(w, "h", h, (dtype,), dev, size)
    elif h is not None:
        _bad(w, "h is written only with a residual")
    if y is None:
        y = _empty(size, dtype=out_dtype, device=dev)
        py, ldy = y.data_ptr(), H
    else:
        py, ldy = _matrix(w, "y", y, (out_dtype,), dev, size)
    if out == "own":
        if scale is not None:
            _bad(w, "scale is written only for 8-bit outputs")
    elif scale is None:
        scale = _empty(T, dtype=torch.float32, device=dev)
        ps = scale.data_ptr()
    else:
        ps = _vector(w, "scale", scale, _F32, dev, T)
    if rstd is None:
        rstd = _empty(T, dtype=torch.float32, device=dev)
        pd = rstd.data_ptr()
    else:
        pd = _vector(w, "rstd", rstd, _F32, dev, T)
    st = (_lib or lib()).mcemu_rmsnorm(fmt, _FMT_OF[weight.dtype], out_fmt, T, H, px, ldx, pr, ldr, pw, eps, ph, ldh, py,
                                       ldy, ps, pd, _stream(dev))
    if st:
        raise McemuError(st, w)
    return y, scale, rstd, h


def rmsnorm_backward(dy, weight, rstd, h=None, ckpt=None, dres=None, dx=None, dw=None, workspace=None):
    """(dx, dw): gradients of the norm's input (dres, the residual path's gradient, added) and
    of its weight (fp32).  The input is given as h or as a checkpoint ckpt = (q, e)."""
    w = "rmsnorm_backward"
    dev = _device(w, dy)
    dtype = dy.dtype
    pdy, lddy = _matrix(w, "dy", dy, _FLOATS, dev)
    size = T, H = dy.shape
    if (h is None) == (ckpt is None):
        _bad(w, "the norm's input is given as h or as ckpt")
    pw = _vector(w, "weight", weight, (dtype, torch.float32), dev, H)
    prs = _vector(w, "rstd", rstd, _F32, dev, T)
    ph = ldh = pq = ldq = pe = lde = pr = ldr = 0
    if h is not None:
        ph, ldh = _matrix(w, "h", h, (dtype,), dev, size)
    else:
        pq, ldq, pe, lde = _ckpt(w, *ckpt, dev, T, H)
    if dres is not None:
        pr, ldr = _matrix(w, "dres", dres, (dtype,), dev, size)
    if dx is None:
        dx = _empty(size, dtype=dtype, device=dev)
        pdx, lddx = dx.data_ptr(), H
    else:
        pdx, lddx = _matrix(w, "dx", dx, (dtype,), dev, size)
    if dw is None:
        dw = _empty(H, dtype=torch.float32, device=dev)
        pdw = dw.data_ptr()
    else:
        pdw = _vector(w, "dw", dw, _F32, dev, H)
    L = _lib or lib()
    ws, pws, nws = _workspace(w, L.mcemu_rmsnorm_backward_workspace(T, H), dev, workspace)
    st = L.mcemu_rmsnorm_backward(_FMT_OF[dtype], _FMT_OF[weight.dtype], T, H, pdy, lddy, pr, ldr, ph, ldh, pq, ldq, pe,
                                  lde, prs, pw, pdx, lddx, pdw, pws, nws, _stream(dev))
    if st:
        raise McemuError(st, w)
    return dx, dw


def int8_linear(x, sx, weight, sw, bias=None, out: str = "bf16", y=None, workspace=None):
    """y = (x @ weight.T) * sx[:, None] * sw + bias, x [M, K] and weight [N, K] int8, the sums
    exact.  ``out`` is "bf16", "fp16" or "fp32"; "int32" gives the sums themselves (sx, sw and
    bias None)."""
    w = "int8_linear"
    dev = _device(w, x)
    px, ldx = _matrix(w, "x", x, _I8, dev)
    pw, ldw = _matrix(w, "weight", weight, _I8, dev)
    M, K = x.shape
    N, k = weight.shape
    if k != K:
        _bad(w, f"weight must have {K} columns")
    if out not in _DTYPE:
        _bad(w, "out must be 'bf16', 'fp16', 'fp32' or 'int32'")
    psx = psw = pb = None
    if out == "int32":
        if sx is not None or sw is not None or bias is not None:
            _bad(w, "sums in int32 take neither scales nor a bias")
    elif sx is None or sw is None:
        _bad(w, "scales are missing")
    else:
        psx, psw = _vector(w, "sx", sx, _F32, dev, M), _vector(w, "sw", sw, _F32, dev, N)
        if bias is not None:
            pb = _vector(w, "bias", bias, _F32, dev, N)
    if y is None:
        y = _empty((M, N), dtype=_DTYPE[out], device=dev)
        py, ldy = y.data_ptr(), N
    else:
        py, ldy = _matrix(w, "y", y, (_DTYPE[out],), dev, (M, N))
    L = _lib or lib()
    ws, pws, nws = _workspace(w, L.mcemu_int8_linear_workspace(M, N, K, (px | ldx | pw | ldw) % 16 == 0), dev,
                             workspace)
    st = L.mcemu_int8_linear(M, N, K, px, ldx, psx, pw, ldw, psw, pb, _LINEAR_OUT[out], py, ldy, pws, nws, _stream(dev))
    if st:
        raise McemuError(st, w)
    return y


def act8_compress(x, q=None, e=None):
    """(q, e): int8 codes [T, H] and exponents [T, ceil(H / 128)] with x ~ q * 2^e."""
    w = "act8_compress"
    dev = _device(w, x)
    px, ldx = _matrix(w, "x", x, _FLOATS, dev)
    size = T, H = x.shape
    blocks = (H + ACT8_BLOCK - 1) // ACT8_BLOCK
    if q is None:
        q = _empty(size, dtype=torch.int8, device=dev)
        pq, ldq = q.data_ptr(), H
    else:
        pq, ldq = _matrix(w, "q", q, _I8, dev, size)
    if e is None:
        e = _empty((T, blocks), dtype=torch.int8, device=dev)
        pe, lde = e.data_ptr(), blocks
    else:
        pe, lde = _matrix(w, "e", e, _I8, dev, (T, blocks))
    st = (_lib or lib()).mcemu_act8_compress(_FMT_OF[x.dtype], T, H, px, ldx, pq, ldq, pe, lde, _stream(dev))
    if st:
        raise McemuError(st, w)
    return q, e


def act8_expand(q, e, out: str = "bf16", x=None):
    """q * 2^e in "bf16", "fp16" or "fp32"."""
    w = "act8_expand"
    dev = _device(w, q)
    if q.dim() != 2 or out not in ("bf16", "fp16", "fp32"):
        _bad(w, "q must be a matrix and out 'bf16', 'fp16' or 'fp32'")
    T, H = q.shape
    pq, ldq, pe, lde = _ckpt(w, q, e, dev, T, H)
    if x is None:
        x = _empty((T, H), dtype=_DTYPE[out], device=dev)
    px, ldx = _matrix(w, "x", x, (_DTYPE[out],), dev, (T, H))
    st = (_lib or lib()).mcemu_act8_expand(FMT[out], T, H, pq, ldq, pe, lde, px, ldx, _stream(dev))
    if st:
        raise McemuError(st, w)
    return x


def act8_wgrad(dy, q, e, out: str = "fp32", dW=None, accumulate: bool = False, workspace=None):
    """dW [N, K] = dy.T @ (q * 2^e): the gradient of a linear layer's weight from dy [T, N]
    (bfloat16) and the checkpoint of its input [T, K].  With ``accumulate`` it is added to
    dW (fp32)."""
    w = "act8_wgrad"
    dev = _device(w, dy)
    pdy, lddy = _matrix(w, "dy", dy, _BF16, dev)
    T, N = dy.shape
    if q.dim() != 2 or q.shape[0] != T:
        _bad(w, f"q must be a matrix of {T} rows")
    K = q.shape[1]
    pq, ldq, pe, lde = _ckpt(w, q, e, dev, T, K)
    if out not in ("bf16", "fp32") or (accumulate and (out != "fp32" or dW is None)):
        _bad(w, "out must be 'bf16' or 'fp32'; accumulate adds to an fp32 dW that is passed in")
    if dW is None:
        dW = _empty((N, K), dtype=_DTYPE[out], device=dev)
        pd, ldd = dW.data_ptr(), K
    else:
        pd, ldd = _matrix(w, "dW", dW, (_DTYPE[out],), dev, (N, K))
    L = _lib or lib()
    ws, pws, nws = _workspace(w, L.mcemu_act8_wgrad_workspace(T, N, K, int(pdy % 16 == 0 and lddy % 8 == 0)), dev, workspace)
    st = L.mcemu_act8_wgrad(T, N, K, pdy, lddy, pq, ldq, pe, lde, FMT[out], int(bool(accumulate)), pd, ldd, pws, nws,
                            _stream(dev))
    if st:
        raise McemuError(st, w)
    return dW


def check():
    """Waits for the current stream; raises (status 6) when a bounded wait inside one of the
    product kernels gave up since the last call, which leaves that launch's results invalid."""
    st = (_lib or lib()).mcemu_ops_check(_stream(torch.cuda.current_device()))
    if st:
        raise McemuError(st, "check")
