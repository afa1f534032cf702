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


@pytest.mark.parametrize("H", [8, 7, 9001])
def test_rmsnorm_backward_joins_in_a_tree(O, H):
    """dw from one row of 1 and 31 others that a running sum of 1 drops: each of 32 rows is a block's, and
    their join costs five roundings, beside four of a product and of a row's part."""
    dy = torch.full((32, H), 0.99 * U32)
    dy[0] = 1
    one = torch.ones(32, H, device="cuda")
    _, dw = O.rmsnorm_backward(dy.cuda(), torch.ones(H).cuda(), torch.ones(32).cuda(), h=one)
    want = dy.double().sum(0)
    assert torch.all((dw.cpu().double() - want).abs() <= 9 * U32 * want)
