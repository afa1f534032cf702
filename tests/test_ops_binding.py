"""The binding of the 8-bit layer operators without a GPU: what it refuses before the library is called."""
import pytest

torch = pytest.importorskip("torch")
from bit_exact_emulation_gb300 import ops  # noqa: E402

UNSUPPORTED = 2
BF16, F32, I8 = torch.bfloat16, torch.float32, torch.int8


@pytest.fixture
def O(monkeypatch):
    """The binding with tensors that hold no memory in place of a device's; a call that would reach
    the library fails the test."""
    class Library:
        def __getattr__(self, name):
            return lambda *a: pytest.fail(f"{name} was called")

    monkeypatch.setattr(ops, "_lib", Library())
    monkeypatch.setattr(ops, "_device", lambda where, t: -1)
    monkeypatch.setattr(ops, "_stream", lambda dev: 0)
    monkeypatch.setattr(ops, "_empty", lambda *s, dtype, device: z(*s, dt=dtype))
    return ops


def z(*size, dt=BF16):
    return torch.empty(*size, dtype=dt, device="meta")


@pytest.mark.parametrize("n", [2 ** 31 - 65535, 2 ** 31, 2 ** 32, 2 ** 32 + 4])
def test_sizes_beyond_32_bits_raise(O, n):
    """Not taken modulo 2^32: nothing would be computed for 2^32 rows, four for 2^32 + 4."""
    calls = (lambda: O.rmsnorm(z(n, 1), z(1), 1e-5), lambda: O.rmsnorm(z(1, n), z(n), 1e-5),
             lambda: O.rmsnorm_backward(z(n, 1), z(1), z(n, dt=F32), h=z(n, 1)),
             lambda: O.rmsnorm_backward(z(1, n), z(n), z(1, dt=F32), h=z(1, n)),
             lambda: O.int8_linear(z(n, 1, dt=I8), z(n, dt=F32), z(4, 1, dt=I8), z(4, dt=F32)),
             lambda: O.int8_linear(z(4, 1, dt=I8), z(4, dt=F32), z(n, 1, dt=I8), z(n, dt=F32)),
             lambda: O.int8_linear(z(1, n, dt=I8), None, z(1, n, dt=I8), None, out="int32"),
             lambda: O.act8_compress(z(n, 1)), lambda: O.act8_compress(z(1, n)),
             lambda: O.act8_expand(z(n, 1, dt=I8), z(n, 1, dt=I8)),
             lambda: O.act8_wgrad(z(n, 1), z(n, 1, dt=I8), z(n, 1, dt=I8)),
             lambda: O.act8_wgrad(z(1, n), z(1, 1, dt=I8), z(1, 1, dt=I8)),
             lambda: O.act8_wgrad(z(1, 1), z(1, n, dt=I8), z(1, -(-n // 128), dt=I8)))
    for i, call in enumerate(calls):
        with pytest.raises(ops.McemuError) as e:
            call()
        assert e.value.status == UNSUPPORTED, i


def test_a_gradient_is_not_dropped_silently(O):
    """The operators record nothing for autograd: a tensor that requires a gradient is refused where one
    would be recorded, and taken where it would not."""
    def g(*size, dt=BF16):
        return z(*size, dt=dt).requires_grad_()

    f = lambda *s: z(*s, dt=F32)
    i = lambda *s: z(*s, dt=I8)
    calls = (lambda: O.rmsnorm(g(4, 8), z(8), 1e-5), lambda: O.rmsnorm(z(4, 8), g(8), 1e-5),
             lambda: O.rmsnorm(z(4, 8), z(8), 1e-5, residual=g(4, 8)), lambda: O.rmsnorm(z(4, 8), z(8), 1e-5, out="own", y=g(4, 8)),
             lambda: O.rmsnorm_backward(g(4, 8), z(8), f(4), h=z(4, 8)), lambda: O.rmsnorm_backward(z(4, 8), g(8), f(4), h=z(4, 8)),
             lambda: O.rmsnorm_backward(z(4, 8), z(8), g(4, dt=F32), h=z(4, 8)), lambda: O.rmsnorm_backward(z(4, 8), z(8), f(4), h=g(4, 8)),
             lambda: O.rmsnorm_backward(z(4, 8), z(8), f(4), h=z(4, 8), dres=g(4, 8)),
             lambda: O.int8_linear(i(4, 8), g(4, dt=F32), i(5, 8), f(5)), lambda: O.int8_linear(i(4, 8), f(4), i(5, 8), g(5, dt=F32)),
             lambda: O.int8_linear(i(4, 8), f(4), i(5, 8), f(5), bias=g(5, dt=F32)), lambda: O.act8_compress(g(4, 8)),
             lambda: O.act8_wgrad(g(4, 8), i(4, 9), i(4, 1)))
    for n, call in enumerate(calls):
        with pytest.raises(ops.McemuError, match="gradient"):
            call()
        with torch.no_grad(), pytest.raises(pytest.fail.Exception, match="was called"):
            call()
