"""Measured cases of the 8-bit layer operators (``bit_exact_emulation_gb300.ops``).

Five calls that a user makes one after another around the matrix products of a layer
whose operands are held in 8 bits:

  rmsnorm            residual addition, root-mean-square norm, output in 8 bits with a scale for each token
  int8_linear        product of 8-bit integers with a scale for each token and each channel
  act8_compress      activation checkpoint: 8 bits an element, a power-of-two scale for each 128 of a row
  act8_wgrad         a linear layer's weight gradient, from the checkpoint of its input
  rmsnorm_backward   the norm's gradients, from the checkpoint of its input

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits; with
``own`` true it makes the library's calls.
"""
import math

import torch

own = False

BLOCK = 128                       # elements of a row that share a checkpoint's scale
DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "int8": 1, "e4m3": 1, "e5m2": 1}
TOP = {"int8": 127.0, "e4m3": 448.0, "e5m2": 57344.0}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
AMAX_FLOOR = 2.0 ** -100          # a row's largest |h w| counts as at least this
EPS = 1e-5


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token of a serving step: latency
        {"name": "norm_one_token", "op": "norm", "T": 1, "H": 4096, "fmt": "bf16", "out": "int8", "res": True},
        # a prompt (or a training batch) through the norm in front of an 8-bit product
        {"name": "norm_prompt", "op": "norm", "T": 8192, "H": 8192, "fmt": "bf16", "out": "int8", "res": True},
        # ragged batch of an odd width, FP8 output for the emulated FP8 units
        {"name": "norm_ragged_e4m3", "op": "norm", "T": 1021, "H": 5005, "fmt": "fp16", "out": "e4m3", "res": False},
        # one token through a linear layer: the weights' bytes are all there is
        {"name": "linear_one_token", "op": "linear", "M": 1, "N": 4096, "K": 4096, "out": "bf16", "bias": False},
        # a small ragged batch with sizes that no vector width divides
        {"name": "linear_ragged", "op": "linear", "M": 77, "N": 5003, "K": 2049, "out": "fp32", "bias": True},
        # a prompt through a linear layer: matrix-unit bound
        {"name": "linear_prompt", "op": "linear", "M": 8192, "N": 8192, "K": 4096, "out": "bf16", "bias": True},
        # saving a large activation
        {"name": "compress_large", "op": "compress", "T": 16384, "H": 8192, "fmt": "bf16"},
        # saving a small one of an odd width, from 32-bit activations
        {"name": "compress_ragged", "op": "compress", "T": 509, "H": 2047, "fmt": "fp32"},
        # the weight gradient of a square layer over a batch of tokens, kept in 32 bits
        {"name": "wgrad_batch", "op": "wgrad", "T": 8192, "N": 4096, "K": 4096, "out": "fp32"},
        # the same for a narrow layer and a token count that no tile divides: few tiles, a long sum
        {"name": "wgrad_narrow", "op": "wgrad", "T": 5001, "N": 520, "K": 1000, "out": "bf16"},
        # the norm's gradients for a batch of tokens
        {"name": "norm_grad_batch", "op": "norm_grad", "T": 8192, "H": 4096, "fmt": "bf16", "res": True},
        # and for a short odd one
        {"name": "norm_grad_ragged", "op": "norm_grad", "T": 333, "H": 2050, "fmt": "fp32", "res": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """Spread over the logarithm; multiples of 64, of 8 and odd sizes among them."""
    v, kind = _log(rng, lo, hi), rng.randrange(3)
    step = (64, 8, 1)[kind]
    v = max(lo, min(hi, (v + step - 1) // step * step)) if v >= step else v
    return v + 64 if v == 3072 and v < hi else v


def draw(rng):
    op = rng.choice(["norm", "linear", "compress", "wgrad", "norm_grad"])
    if op == "norm":
        H, fmt = _size(rng, 64, 16384), rng.choice(["bf16", "bf16", "fp16", "fp32"])
        return {"op": op, "T": _size(rng, 1, min(16384, 8192 * 8192 * 2 // (H * SIZE[fmt]))), "H": H, "fmt": fmt,
                "out": rng.choice(["int8", "e4m3", "e5m2", "own"]), "res": rng.random() < 0.6}
    if op == "norm_grad":
        H, fmt = _size(rng, 64, 16384), rng.choice(["bf16", "bf16", "fp16", "fp32"])
        return {"op": op, "T": _size(rng, 1, min(16384, 8192 * 8192 * 2 // (H * SIZE[fmt]))), "H": H, "fmt": fmt,
                "res": rng.random() < 0.6}
    if op == "compress":
        H, fmt = _size(rng, 64, 16384), rng.choice(["bf16", "bf16", "fp16", "fp32"])
        return {"op": op, "T": _size(rng, 1, min(16384, 16384 * 8192 * 2 // (H * SIZE[fmt]))), "H": H, "fmt": fmt}
    if op == "linear":
        N, K = _size(rng, 64, 16384), _size(rng, 64, 16384)
        return {"op": op, "M": _size(rng, 1, max(1, min(8192, 8192 * 8192 * 4096 // (N * K)))), "N": N, "K": K,
                "out": rng.choice(["bf16", "fp16", "fp32"]), "bias": rng.random() < 0.5}
    N, K = _size(rng, 64, 8192), _size(rng, 64, 8192)
    return {"op": op, "T": _size(rng, 64, max(64, min(16384, 8192 * 4096 * 4096 // (N * K)))), "N": N, "K": K,
            "out": rng.choice(["bf16", "fp32"])}


def work(case):
    op = case["op"]
    if op == "norm":
        T, H, s = case["T"], case["H"], SIZE[case["fmt"]]
        out = s if case["out"] == "own" else 1
        return {"bytes": T * H * (s + out + (2 * s if case["res"] else 0)) + H * s + T * (4 if case["out"] == "own" else 8),
                "flops": 6 * T * H}
    if op == "norm_grad":
        T, H, s = case["T"], case["H"], SIZE[case["fmt"]]
        return {"bytes": T * H * (2 * s + 1 + (s if case["res"] else 0)) + T * _blocks(H) + 4 * T + H * (s + 4),
                "flops": 10 * T * H}
    if op == "compress":
        T, H = case["T"], case["H"]
        return {"bytes": T * H * (SIZE[case["fmt"]] + 1) + T * _blocks(H), "flops": 3 * T * H}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + M * N * SIZE[case["out"]] + 4 * (M + N + (N if case["bias"] else 0)),
                "flops": 2 * M * N * K}
    T, N, K = case["T"], case["N"], case["K"]
    return {"bytes": 2 * T * N + T * K + T * _blocks(K) + N * K * SIZE[case["out"]], "flops": 2 * T * N * K}


def _blocks(n):
    return -(-n // BLOCK)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, T, H, dtype):
    """Normal values whose channels differ in size, a few of them large, as between the
    layers of a language model; the last row of a batch is padding (zeros)."""
    gain = torch.exp(0.3 * _normal(g, H))
    gain[torch.rand(H, generator=g, device="cuda") < 0.005] *= 20.0
    x = _normal(g, T, H).mul_(gain)
    if T > 8:
        x[-1] = 0
    return x.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, s = case["op"], {"case": dict(case)}
    if op == "norm":
        T, H, dt = case["T"], case["H"], DTYPE[case["fmt"]]
        s["x"] = _activations(g, T, H, dt)
        s["res"] = _normal(g, T, H).to(dt) if case["res"] else None
        s["w"] = (1 + 0.1 * _normal(g, H)).to(dt)
    elif op == "norm_grad":
        T, H, dt = case["T"], case["H"], DTYPE[case["fmt"]]
        h = _activations(g, T, H, dt)
        s["q"], s["e"] = _compress(h)
        s["rstd"] = torch.rsqrt(h.float().square().mean(-1) + EPS)
        del h
        s["w"] = (1 + 0.1 * _normal(g, H)).to(dt)
        s["dy"] = _normal(g, T, H).mul_(1e-3).to(dt)
        s["dres"] = _normal(g, T, H).mul_(1e-3).to(dt) if case["res"] else None
    elif op == "compress":
        s["x"] = _activations(g, case["T"], case["H"], DTYPE[case["fmt"]])
    elif op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = _normal(g, M, K).mul_(32).round_().clamp_(-127, 127).to(torch.int8)
        s["sx"] = torch.rand(M, generator=g, device="cuda") * 0.03 + 0.005
        s["w"] = _normal(g, N, K).mul_(40).round_().clamp_(-127, 127).to(torch.int8)
        s["sw"] = torch.rand(N, generator=g, device="cuda") * 1e-3 + 1e-4
        s["bias"] = _normal(g, N) if case["bias"] else None
    else:
        T, N, K = case["T"], case["N"], case["K"]
        s["dy"] = _normal(g, T, N).mul_(1e-3).to(torch.bfloat16)
        s["q"], s["e"] = _compress(_activations(g, T, K, torch.bfloat16))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from bit_exact_emulation_gb300 import ops
    c = s["case"]
    if c["op"] == "norm":
        y, scale, rstd, h = ops.rmsnorm(s["x"], s["w"], EPS, residual=s["res"], out=c["out"])
        return {"y": y, "scale": scale, "rstd": rstd, "h": h}
    if c["op"] == "norm_grad":
        dx, dw = ops.rmsnorm_backward(s["dy"], s["w"], s["rstd"], ckpt=(s["q"], s["e"]), dres=s["dres"])
        return {"dx": dx, "dw": dw}
    if c["op"] == "compress":
        q, e = ops.act8_compress(s["x"])
        return {"q": q, "e": e}
    if c["op"] == "linear":
        return {"y": ops.int8_linear(s["x"], s["sx"], s["w"], s["sw"], bias=s["bias"], out=c["out"])}
    return {"dw": ops.act8_wgrad(s["dy"], s["q"], s["e"], out=c["out"])}


def _run_plain(s):
    c = s["case"]
    if c["op"] == "norm":
        return _norm(s["x"], s["w"], s["res"], c["out"])
    if c["op"] == "norm_grad":
        h, w, dy, r = _expand(s["q"], s["e"]), s["w"].float(), s["dy"].float(), s["rstd"][:, None]
        xhat = h * r
        gw = dy * w
        dx = (gw - xhat * (gw * xhat).mean(-1, keepdim=True)) * r
        if s["dres"] is not None:
            dx = dx + s["dres"].float()
        return {"dx": dx.to(s["dy"].dtype), "dw": (dy * xhat).sum(0)}
    if c["op"] == "compress":
        q, e = _compress(s["x"])
        return {"q": q, "e": e}
    if c["op"] == "linear":
        y = (s["x"].float() @ s["w"].float().t()) * s["sx"][:, None] * s["sw"]
        if s["bias"] is not None:
            y = y + s["bias"]
        return {"y": y.to(DTYPE[c["out"]])}
    return {"dw": (s["dy"].float().t() @ _expand(s["q"], s["e"])).to(DTYPE[c["out"]])}


def _norm(x, w, res, out):
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    hf, wf = h.float(), w.float()
    rstd = torch.rsqrt(hf.square().mean(-1) + EPS)
    got = {"rstd": rstd, "h": None if res is None else h, "scale": None}
    if out == "own":
        got["y"] = (hf * rstd[:, None] * wf).to(x.dtype)
        return got
    v = hf * wf
    amax = v.abs().amax(-1).clamp_min(AMAX_FLOOR)
    v = v * torch.div(torch.full_like(amax, TOP[out]), amax)[:, None]
    got["y"] = v.round().to(torch.int8) if out == "int8" else v.to(FP8[out])
    got["scale"] = amax * rstd / TOP[out]
    return got


def _compress(x):
    """(codes int8 [T, H], exponents int8 [T, ceil(H / 128)]): the least exponent e >= -120
    with 127 * 2^e >= the block's largest magnitude, codes rounded to nearest, ties to even."""
    T, H = x.shape
    B = _blocks(H)
    xf = torch.nn.functional.pad(x.float(), (0, B * BLOCK - H)).view(T, B, BLOCK)
    m, e = torch.frexp(xf.abs().amax(-1))         # amax = m * 2^e, m in [1/2, 1)
    e = (e - 7 + (m * 128 > 127).int()).clamp_min(-120)
    q = torch.ldexp(xf, -e[..., None]).round().to(torch.int8)
    return q.view(T, B * BLOCK)[:, :H].contiguous(), e.to(torch.int8)


def _expand(q, e):
    T, H = q.shape
    s = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e.int())
    return q.float() * s.repeat_interleave(BLOCK, 1)[:, :H]


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    d = torch.float64
    if op == "compress":
        return None                                # whole numbers only
    if op == "linear":
        y = torch.mm(s["x"].to(d), s["w"].to(d).T)
        y *= s["sx"].to(d).unsqueeze(1) * s["sw"].to(d).unsqueeze(0)
        return {"y": y if s["bias"] is None else y + s["bias"].to(d)}
    if op == "wgrad":
        return {"dw": torch.mm(s["dy"].to(d).T, _expand64(s["q"], s["e"]))}
    w = s["w"].to(d)
    if op == "norm_grad":
        z = _expand64(s["q"], s["e"]) * s["rstd"].to(d).unsqueeze(1)
        dy = s["dy"].to(d)
        g = dy * w
        proj = torch.einsum("th,th->t", g, z) / case["H"]
        dx = s["rstd"].to(d).unsqueeze(1) * (g - proj.unsqueeze(1) * z)
        if case["res"]:
            dx += s["dres"].to(d)
        return {"dx": dx, "dw": torch.einsum("th,th->h", dy, z)}
    total = s["x"].to(d)
    if case["res"]:
        total = total + s["res"].to(d)
    h = total.to(DTYPE[case["fmt"]]).to(d)         # the norm acts on the residual as it is stored
    rstd = (torch.linalg.vector_norm(h, dim=1) ** 2 / case["H"] + EPS) ** -0.5
    y = h * rstd.unsqueeze(1) * w
    got = {"rstd": rstd, "h": total if case["res"] else None, "scale": None, "y": y}
    if case["out"] != "own":
        peak = torch.clamp((h * w).abs().max(dim=1).values, min=AMAX_FLOOR)
        got["scale"] = peak * rstd / TOP[case["out"]]
        got["y"] = None if case["out"] == "int8" else h * w * (TOP[case["out"]] / peak).unsqueeze(1)
    return got


def _expand64(q, e):
    H = q.shape[1]
    at = torch.arange(H, device=q.device) // BLOCK
    return q.to(torch.float64) * torch.pow(2.0, e.to(torch.float64))[:, at]
