"""Measured cases of the FP8 layer operators (``bit_exact_emulation_gb300.fp8``).

Matrix products of 8-bit floating-point numbers with a scale, a power of two, for each block of
128, what makes their operands, and the same grouped by expert:

  quantize          rows in blocks of 128 columns; columns in blocks of 128 rows, transposed
  quantize_weight   blocks of 128 x 128, as they lie and transposed
  linear            product of two such operands (a forward pass, both gradients of a linear layer)
  grouped_linear    the same with a weight for each of a ragged set of row groups
  grouped_wgrad     the groups' weight gradients

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits; with
``own`` true it makes the library's calls.
"""
import math
import random

import torch

own = False

BLOCK = 128
DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP_EXP = {"e4m3": 9, "e5m2": 16}          # the largest number is 0.875 * 2^this: 448 and 57344
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
LEAST = -120                               # of a block's exponent


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token of a serving step in front of a product: latency
        {"name": "quant_one_token", "op": "quant", "T": 1, "H": 4096, "fmt": "bf16", "out": "e4m3", "cols": False, "E": 0},
        # a training batch's activation sorted by expert: rows for the product, columns for the weight gradient
        {"name": "quant_batch", "op": "quant", "T": 8192, "H": 8192, "fmt": "bf16", "out": "e4m3", "cols": True, "E": 8},
        # a layer's weight after an optimizer step, for the forward product and the input's gradient
        {"name": "weight_layer", "op": "weight", "E": 1, "N": 8192, "K": 8192, "fmt": "bf16", "out": "e4m3", "cols": True},
        # a few small experts of odd sizes, from 32-bit weights
        {"name": "weight_odd_experts", "op": "weight", "E": 5, "N": 1001, "K": 523, "fmt": "fp32", "out": "e4m3", "cols": True},
        # one token through a linear layer: the weight's bytes are all there is
        {"name": "linear_one_token", "op": "linear", "M": 1, "N": 4096, "K": 4096, "fx": "e4m3", "tiles": True, "out": "bf16", "bias": False},
        # a prompt through a linear layer: bound by the matrix unit
        {"name": "linear_prompt", "op": "linear", "M": 8192, "N": 8192, "K": 4096, "fx": "e4m3", "tiles": True, "out": "bf16", "bias": True},
        # a small weight gradient of odd sizes: both operands scaled along the sum, gradients in E5M2
        {"name": "linear_odd_gradient", "op": "linear", "M": 77, "N": 5003, "K": 2049, "fx": "e5m2", "tiles": False, "out": "fp32", "bias": False},
        # a serving step of a few requests through many experts: a few rows each, some with none
        {"name": "experts_decode", "op": "experts", "T": 128, "E": 32, "N": 2048, "K": 4096, "out": "bf16"},
        # a training batch through experts of ragged loads
        {"name": "experts_batch", "op": "experts", "T": 16384, "E": 16, "N": 4096, "K": 2048, "out": "bf16"},
        # a few rows through small experts of odd sizes
        {"name": "experts_odd", "op": "experts", "T": 1003, "E": 7, "N": 1000, "K": 1111, "out": "fp32"},
        # the weight gradients of a training batch, kept in 32 bits
        {"name": "wgrad_batch", "op": "wgrad", "T": 16384, "E": 8, "N": 4096, "K": 2048, "out": "fp32"},
        # and of a small one of odd sizes
        {"name": "wgrad_odd", "op": "wgrad", "T": 1003, "E": 5, "N": 264, "K": 523, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def _size(rng, lo, hi):
    """Spread over the logarithm; multiples of 128, of 8 and odd sizes among them."""
    v, step = _log(rng, lo, hi), (128, 8, 1)[rng.randrange(3)]
    return max(lo, min(hi, -(-v // step) * step)) if v >= step else v


def draw(rng):
    op = rng.choice(["quant", "weight", "linear", "experts", "wgrad"])
    if op == "quant":
        H, fmt, cols = _size(rng, 64, 16384), rng.choice(["bf16", "bf16", "fp16", "fp32"]), rng.random() < 0.5
        return {"op": op, "T": _size(rng, 1, min(16384, 8192 * 8192 * 2 // (H * SIZE[fmt]))), "H": H, "fmt": fmt,
                "out": rng.choice(["e4m3", "e4m3", "e5m2"]), "cols": cols, "E": rng.randint(1, 32) if cols and rng.random() < 0.6 else 0}
    if op == "weight":
        E, fmt = rng.choice([1, 1, 2, 3, 8, 16]), rng.choice(["bf16", "bf16", "fp16", "fp32"])
        N = _size(rng, 64, 8192)
        return {"op": op, "E": E, "N": N, "K": _size(rng, 64, min(16384, 8192 * 8192 * 2 // (E * N * SIZE[fmt]))), "fmt": fmt,
                "out": rng.choice(["e4m3", "e4m3", "e5m2"]), "cols": rng.random() < 0.5}
    if op == "linear":
        N, K = _size(rng, 64, 16384), _size(rng, 64, 16384)
        return {"op": op, "M": _size(rng, 1, max(1, min(8192, 8192 * 8192 * 4096 // (N * K)))), "N": N, "K": K,
                "fx": rng.choice(["e4m3", "e4m3", "e5m2"]), "tiles": rng.random() < 0.6,
                "out": rng.choice(["bf16", "fp16", "fp32"]), "bias": rng.random() < 0.4}
    E = _log(rng, 1, 64)
    N = _size(rng, 64, 8192)
    K = _size(rng, 64, min(8192, max(64, (1 << 28) // (E * N))))
    blocks = min(128, 1200_000_000 // (N * K) - E)         # what the plain form holds in 32 bits
    return {"op": op, "T": _size(rng, 1, max(1, min(16384, 128 * blocks))), "E": E, "N": N, "K": K,
            "out": rng.choice(["bf16", "fp32"])}


def _blocks(n):
    return -(-n // BLOCK)


def _room(T, E):
    """Blocks of 128 rows that T rows in E groups, each beginning a block, may need."""
    return (T + 127 * max(1, E)) // BLOCK


def work(case):
    op = case["op"]
    if op == "quant":
        T, H, s = case["T"], case["H"], SIZE[case["fmt"]]
        cols = T * H + H * _blocks(T) if case["cols"] else 0
        return {"bytes": T * H * (s + 1) + T * _blocks(H) + cols, "flops": 3 * T * H}
    if op == "weight":
        E, N, K = case["E"], case["N"], case["K"]
        sides = 2 if case["cols"] else 1
        return {"bytes": E * (N * K * (SIZE[case["fmt"]] + sides) + sides * _blocks(N) * _blocks(K)), "flops": 3 * E * N * K}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        scales = _blocks(K) * (M + (_blocks(N) if case["tiles"] else N))
        return {"bytes": M * K + N * K + scales + M * N * SIZE[case["out"]] + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    T, E, N, K = case["T"], case["E"], case["N"], case["K"]
    if op == "experts":
        active = E * (1 - (1 - 1 / E) ** T)                # experts that any row goes to, on average
        return {"bytes": T * K + T * _blocks(K) + active * (N * K + _blocks(N) * _blocks(K)) + T * N * SIZE[case["out"]] + 4 * E,
                "flops": 2 * T * N * K}
    return {"bytes": T * (N + K) + _blocks(T) * (N + K) + E * N * K * SIZE[case["out"]] + 4 * E, "flops": 2 * T * N * K}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, T, H, dtype):
    """Normal values whose channels differ in size, a few of them large; the last rows of a batch
    are padding (zeros)."""
    gain = torch.exp(0.3 * _normal(g, H))
    gain[torch.rand(H, generator=g, device="cuda") < 0.005] *= 20.0
    x = _normal(g, T, H).mul_(gain)
    if T > 200:
        x[-150:] = 0
    return x.to(dtype)


def _offsets(seed, T, E):
    """Where each group's rows begin, and where the last ends: T rows sent to E experts, some of
    them liked better than others."""
    r = random.Random(seed)
    likes = [math.exp(0.5 * r.gauss(0, 1)) for _ in range(E)]
    counts = [0] * E
    for e in r.choices(range(E), likes, k=T):
        counts[e] += 1
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, s = case["op"], {"case": dict(case)}
    if op == "quant":
        s["x"] = _activations(g, case["T"], case["H"], DTYPE[case["fmt"]])
        s["offsets"] = _offsets(seed, case["T"], case["E"]) if case["E"] else None
        return s
    if op == "weight":
        s["w"] = _normal(g, case["E"], case["N"], case["K"]).mul_(case["K"] ** -0.5).to(DTYPE[case["fmt"]])
        return s
    N, K = case["N"], case["K"]
    if op == "linear":
        s["x"], s["ex"] = _rows(_activations(g, case["M"], K, torch.bfloat16), case["fx"])
        w = _normal(g, N, K).mul_(K ** -0.5)
        s["w"], s["ew"] = [t[0] for t in _tiles(w[None], "e4m3")] if case["tiles"] else _rows(w, "e4m3")
        s["bias"] = _normal(g, N) if case["bias"] else None
        return s
    T, E = case["T"], case["E"]
    s["offsets"] = _offsets(seed, T, E)
    if op == "experts":
        s["x"], s["ex"] = _rows(_activations(g, T, K, torch.bfloat16), "e4m3")
        s["w"], s["ew"] = _tiles(_normal(g, E, N, K).mul_(K ** -0.5), "e4m3")
    else:
        s["dyt"], s["edyt"] = _columns(_normal(g, T, N).mul_(1e-3), "e4m3", s["offsets"])
        s["xt"], s["ext"] = _columns(_activations(g, T, K, torch.bfloat16), "e4m3", s["offsets"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from bit_exact_emulation_gb300 import fp8
    c = s["case"]
    if c["op"] == "quant":
        q, e, qt, et = fp8.quantize(s["x"], out=c["out"], columns=c["cols"], offsets=s["offsets"])
        return {"q": q, "e": e, "qt": qt, "et": et}
    if c["op"] == "weight":
        q, e, qt, et = fp8.quantize_weight(s["w"], out=c["out"], transposed=c["cols"])
        return {"q": q, "e": e, "qt": qt, "et": et}
    if c["op"] == "linear":
        return {"y": fp8.linear(s["x"], s["ex"], s["w"], s["ew"], bias=s["bias"], out=c["out"])}
    if c["op"] == "experts":
        return {"y": fp8.grouped_linear(s["x"], s["ex"], s["w"], s["ew"], s["offsets"], out=c["out"])}
    return {"dw": fp8.grouped_wgrad(s["dyt"], s["edyt"], s["xt"], s["ext"], s["offsets"], out=c["out"])}


def _run_plain(s):
    c = s["case"]
    if c["op"] == "quant":
        q, e = _rows(s["x"], c["out"])
        qt, et = _columns(s["x"], c["out"], s["offsets"]) if c["cols"] else (None, None)
        return {"q": q, "e": e, "qt": qt, "et": et}
    if c["op"] == "weight":
        q, e = _tiles(s["w"], c["out"])
        if not c["cols"]:
            return {"q": q, "e": e, "qt": None, "et": None}
        return {"q": q, "e": e, "qt": q.transpose(1, 2).contiguous(), "et": e.transpose(1, 2).contiguous()}
    if c["op"] == "linear":
        w = _of_tiles(s["w"][None], s["ew"][None])[0] if c["tiles"] else _of_rows(s["w"], s["ew"])
        y = _of_rows(s["x"], s["ex"]) @ w.t()
        if s["bias"] is not None:
            y = y + s["bias"]
        return {"y": y.to(DTYPE[c["out"]])}
    if c["op"] == "experts":
        # each group's rows in blocks of 128 of its own, each block by its group's weight
        row, real, group = _padded(s["offsets"], c["T"])
        x = _of_rows(s["x"], s["ex"])[row.clamp_max(c["T"] - 1)].view(-1, BLOCK, c["K"])
        w = _of_tiles(s["w"], s["ew"])[group.clamp_max(c["E"] - 1)]
        y = torch.bmm(x, w.transpose(1, 2)).view(-1, c["N"]).to(DTYPE[c["out"]])
        out = torch.empty(c["T"] + 1, c["N"], dtype=y.dtype, device=y.device)
        out[torch.where(real, row, c["T"])] = y             # blocks' empty places go to a row of their own
        return {"y": out[:c["T"]]}
    # a product for each block of 128 rows, then each group's sum
    group = _padded(s["offsets"], c["T"])[2]
    dy = _of_rows(s["dyt"], s["edyt"]).view(c["N"], -1, BLOCK).permute(1, 0, 2)
    x = _of_rows(s["xt"], s["ext"]).view(c["K"], -1, BLOCK).permute(1, 2, 0)
    mine = (group == torch.arange(c["E"], device=group.device)[:, None]).float()
    return {"dw": (mine @ torch.bmm(dy, x).view(len(group), -1)).view(c["E"], c["N"], c["K"]).to(DTYPE[c["out"]])}


def _exponents(amax, out):
    """The least exponent >= LEAST with amax <= TOP * 2^e, int32."""
    m, e = torch.frexp(amax)                   # amax = m * 2^e, m in [1/2, 1)
    e = (e - TOP_EXP[out] + (m > 0.875).int()).clamp_min(LEAST)
    return torch.where(amax == 0, LEAST, e)


def _rows(x, out):
    """(codes [T, H], exponents int8 [T, blocks]): blocks of 128 along each row."""
    T, H = x.shape
    B = _blocks(H)
    xf = torch.nn.functional.pad(x.float(), (0, B * BLOCK - H)).view(T, B, BLOCK)
    e = _exponents(xf.abs().amax(-1), out)
    q = torch.ldexp(xf, -e[..., None]).view(T, B * BLOCK)[:, :H].contiguous()
    return q.to(FP8[out]), e.to(torch.int8)


def _padded(offsets, T):
    """Rows in blocks of 128, each group beginning a block: for each place its row, whether it
    holds one, and for each block its group (the number of groups behind the last)."""
    n = (offsets[1:] - offsets[:-1]).long()
    ends = ((n + BLOCK - 1) // BLOCK).cumsum(0)
    blocks = torch.arange(_room(T, len(n)), device=n.device)
    group = torch.searchsorted(ends, blocks, right=True)
    g = group.clamp_max(len(n) - 1)
    first = (blocks - ends[g] + (n[g] + BLOCK - 1) // BLOCK) * BLOCK           # of the block's places, in its group
    at = (first[:, None] + torch.arange(BLOCK, device=n.device))
    real = (at < n[g][:, None]) & (group < len(n))[:, None]
    return (at + offsets[g][:, None]).view(-1), real.view(-1), group


def _columns(x, out, offsets):
    """(codes [H, P], exponents int8 [H, P / 128]): blocks of 128 rows of each column, transposed;
    each group of rows begins a block, and what no row fills is zero."""
    T, H = x.shape
    if offsets is None:
        offsets = torch.arange(2, device=x.device, dtype=torch.int32) * T
    row, real, _ = _padded(offsets, T)
    xt = torch.where(real[:, None], x.float()[row.clamp_max(T - 1)], 0.0).t()
    return _rows(xt, out)


def _tiles(w, out):
    """(codes [E, N, K], exponents int8 [E, ceil(N / 128), ceil(K / 128)])."""
    E, N, K = w.shape
    n, k = _blocks(N), _blocks(K)
    wf = torch.nn.functional.pad(w.float(), (0, k * BLOCK - K, 0, n * BLOCK - N)).view(E, n, BLOCK, k, BLOCK)
    e = _exponents(wf.abs().amax((2, 4)), out)
    q = torch.ldexp(wf, -e[:, :, None, :, None]).view(E, n * BLOCK, k * BLOCK)[:, :N, :K].contiguous()
    return q.to(FP8[out]), e.to(torch.int8)


def _of_rows(q, e):
    s = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e.int())
    return q.float() * s.repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _of_tiles(q, e):
    s = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e.int())
    return q.float() * s.repeat_interleave(BLOCK, 1)[:, :q.shape[1]].repeat_interleave(BLOCK, 2)[:, :, :q.shape[2]]


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "quant":
        got = {"q": _scaled64(s["x"].double(), case["out"]), "e": None, "qt": None, "et": None}
        if case["cols"]:
            at = [0, case["T"]] if s["offsets"] is None else s["offsets"].tolist()
            qt = torch.zeros(case["H"], BLOCK * _room(case["T"], len(at) - 1), dtype=torch.float64, device="cuda")
            first = 0
            for a, b in zip(at, at[1:]):
                qt[:, first:first + b - a] = _scaled64(s["x"][a:b].double().T, case["out"])
                first += BLOCK * _blocks(b - a)
            got["qt"] = qt
        return got
    if op == "weight":
        q = s["w"].double()
        for i in range(0, case["N"], BLOCK):
            peak = q[:, i:i + BLOCK].abs().amax(1, keepdim=True)
            q[:, i:i + BLOCK] = _nearest64(q[:, i:i + BLOCK] / _steps64(peak, case["out"]), case["out"])
        return {"q": q, "e": None, "qt": q.mT if case["cols"] else None, "et": None}
    if op == "linear":
        w = _value64(s["w"], s["ew"].repeat_interleave(BLOCK, 0)[:case["N"]] if case["tiles"] else s["ew"])
        y = torch.mm(_value64(s["x"], s["ex"]), w.T)
        return {"y": y if s["bias"] is None else y + s["bias"].double()}
    at, N, K = s["offsets"].tolist(), case["N"], case["K"]
    if op == "experts":
        x, y = _value64(s["x"], s["ex"]), torch.zeros(case["T"], N, dtype=torch.float64, device="cuda")
        for i, (a, b) in enumerate(zip(at, at[1:])):
            y[a:b] = x[a:b] @ _value64(s["w"][i], s["ew"][i].repeat_interleave(BLOCK, 0)[:N]).T
        return {"y": y}
    dy, x, first = _value64(s["dyt"], s["edyt"]), _value64(s["xt"], s["ext"]), 0
    dw = torch.zeros(case["E"], N, K, dtype=torch.float64, device="cuda")
    for i, (a, b) in enumerate(zip(at, at[1:])):
        dw[i] = dy[:, first:first + b - a] @ x[:, first:first + b - a].T
        first += BLOCK * _blocks(b - a)
    return {"dw": dw}


def _steps64(peak, out):
    """2^e for the largest magnitudes [..., H] of columns, the columns in blocks of 128."""
    H = peak.shape[-1]
    p = torch.stack([b.amax(-1) for b in peak.split(BLOCK, -1)], -1)
    e = torch.ceil(torch.log2(p / TOP[out])).clamp(min=LEAST)
    return torch.exp2(e)[..., torch.arange(H, device=peak.device) // BLOCK]


def _scaled64(x, out):
    return _nearest64(x / _steps64(x.abs(), out), out) if x.numel() else x


def _nearest64(x, out):
    """The nearest numbers of the format, ties to even: 3 (2) bits behind the first, exponents from -6 (-14) on."""
    digits, least = (3, -6) if out == "e4m3" else (2, -14)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** least))) - digits)
    return torch.round(x / step) * step


def _value64(q, e):
    at = torch.arange(q.shape[-1], device=q.device) // BLOCK
    return q.double() * torch.pow(2.0, e.double())[:, at]
