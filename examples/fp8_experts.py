"""A layer of experts in FP8, forward and backward, and a linear layer served in FP8.

  1. Tokens sorted by expert go through each expert's weight: operands with a power-of-two scale for
     each block of 128, products of ragged groups, gradients of the input and of the weights from the
     same codes.  Errors against the unquantised layer, and against the quantised operands themselves
     in 64 bits: what is left there is the GPU's arithmetic.
  2. The same operands through the emulated FP8 unit: the product's sums within a block are those of
     the emulated B200 unit, bit for bit.

Run on a GPU: python examples/fp8_experts.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_exact_emulation_gb300 import binding, fp8  # noqa: E402


def rel(got, want):
    """Norm-wise relative error."""
    return float((got.detach().double() - want.detach().double()).norm() / want.detach().double().norm())


def value(q, e):
    """What codes and their exponents stand for, in 64 bits."""
    rows = e.double().exp2()
    if e.shape[-2] != q.shape[-2]:
        rows = rows.repeat_interleave(fp8.BLOCK, -2)[..., :q.shape[-2], :]
    return q.double() * rows.repeat_interleave(fp8.BLOCK, -1)[..., :q.shape[-1]]


class Experts(torch.autograd.Function):
    """y[t] = x[t] @ W[g].T for the tokens t of each group g, W [E, N, K]; products in FP8."""

    @staticmethod
    def forward(ctx, x, W, offsets):
        q, e, qt, et = fp8.quantize(x, columns=True, offsets=offsets)      # rows for now, columns for dW
        w, ew, wt, ewt = fp8.quantize_weight(W, transposed=True)
        ctx.save_for_backward(qt, et, wt, ewt, offsets)
        return fp8.grouped_linear(q, e, w, ew, offsets)

    @staticmethod
    def backward(ctx, dy):
        qt, et, wt, ewt, offsets = ctx.saved_tensors
        d, ed, dt, edt = fp8.quantize(dy.contiguous(), out="e5m2", columns=True, offsets=offsets)
        dx = fp8.grouped_linear(d, ed, wt, ewt, offsets)
        dW = fp8.grouped_wgrad(dt, edt, qt, et, offsets, out="bf16")
        return dx, dW, None


def train(x, W, dy, offsets):
    """One step, and its errors."""
    at = offsets.tolist()
    x, W = x.detach().requires_grad_(), W.detach().requires_grad_()
    y = Experts.apply(x, W, offsets)
    y.backward(dy)
    full = torch.cat([x[a:b].double() @ W[g].double().T for g, (a, b) in enumerate(zip(at, at[1:]))])
    dx = torch.cat([dy[a:b].double() @ W[g].double() for g, (a, b) in enumerate(zip(at, at[1:]))])
    dW = torch.stack([dy[a:b].double().T @ x[a:b].double() for a, b in zip(at, at[1:])])
    with torch.no_grad():
        (q, e, _, _), (w, ew, _, _) = fp8.quantize(x), fp8.quantize_weight(W)
        xv, wv = value(q, e), value(w, ew)
        same = torch.cat([xv[a:b] @ wv[g].T for g, (a, b) in enumerate(zip(at, at[1:]))])
        got = fp8.grouped_linear(q, e, w, ew, offsets, out="fp32")
    return {"output_error": rel(y, full), "input_gradient_error": rel(x.grad, dx), "weight_gradient_error": rel(W.grad, dW),
            "error_of_the_arithmetic": rel(got, same)}


def serve(x, W):
    """One token and a batch through a linear layer; and the emulated unit's sums."""
    w, ew, _, _ = fp8.quantize_weight(W)
    q, e, _, _ = fp8.quantize(x)
    y, one = fp8.linear(q, e, w, ew), fp8.linear(q[:1], e[:1], w, ew)
    M, N, K = min(64, len(x)), min(64, len(W)), fp8.BLOCK
    zero = lambda rows: torch.zeros(rows, 1, dtype=torch.int8, device=x.device)
    sums = fp8.linear(q[:M, :K], zero(M), w[:N, :K], zero(N), out="fp32")
    unit = binding.Model(binding.preset_desc("b200_fp8"))
    emulated = binding.tile_gemm(unit, binding.tile(0, 16, 16, 32, 8), q[:M, :K], w[:N, :K],
                                 torch.zeros(M, N, dtype=torch.int32, device=x.device))
    return {"served_error": rel(y, x.double() @ W.double().T), "one_token_error": rel(one, x[:1].double() @ W.double().T),
            "same_bits_as_the_emulated_unit": bool(torch.equal(sums.view(torch.int32), emulated))}


def main(tokens=600, experts=5, width=1024, channels=768, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, dy = normal(tokens, width).to(torch.bfloat16), (1e-3 * normal(tokens, channels)).to(torch.bfloat16)
    W = (normal(experts, channels, width) / width ** 0.5).to(torch.bfloat16)
    ends = torch.randint(0, tokens + 1, (experts - 1,), generator=g, device="cuda").sort().values
    offsets = torch.cat([ends.new_zeros(1), ends, ends.new_full((1,), tokens)]).to(torch.int32)
    result = {**train(x, W, dy, offsets), **serve(x, W[0])}
    fp8.check()
    return result


if __name__ == "__main__":
    for name, number in main().items():
        print(f"{name:40s} {number if isinstance(number, bool) else format(number, '.3g')}")
