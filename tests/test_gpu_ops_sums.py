"""The order in which the 8-bit layer operators add."""
import pytest

from test_gpu_ops import O, U32, norm_tol  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("H", [99_999, 100_000])
def test_rmsnorm_long_rows_add_in_short_chains(O, H):
    """A row whose squares are 1 and many that a running sum of 1 drops: the error stays within the bound
    of H / 1024 additions a thread."""
    x = torch.zeros(1, H)
    x[0, ::512] = (0.99 * U32) ** 0.5
    x[0, 0] = 1
    _, _, rstd, _ = O.rmsnorm(x.cuda(), torch.ones(H).cuda(), 0.0)
    want = 1 / (x.double() ** 2).mean().sqrt().item()
    assert abs(rstd.item() - want) <= norm_tol(H) * want
