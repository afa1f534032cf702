"""The order in which the 8-bit layer operators add, and products whose sums take several steps."""
import numpy as np
import pytest

from test_gpu_ops import O, U32, int8s, linear_host, norm_tol, same, wgrad_case, wgrad_check  # noqa: F401

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


@pytest.mark.parametrize("M,N,K", [(1300, 1800, 2100), (1100, 1030, 3080), (2048, 1024, 1040), (1500, 2300, 4097)])
def test_int8_linear_panels_of_long_sums(O, M, N, K):
    """Panels whose accumulators are taken out more than once."""
    rng = np.random.default_rng(K)
    assert O.lib().mcemu_int8_linear_workspace(M, N, K, K % 16 == 0) > 0
    x, w = int8s(rng, M, K), int8s(rng, N, K)
    sx = torch.from_numpy(rng.uniform(1e-3, 1e-2, M).astype(np.float32))
    sw = torch.from_numpy(rng.uniform(1e-3, 1e-2, N).astype(np.float32))
    bias = torch.from_numpy(rng.standard_normal(N).astype(np.float32))
    gx, gw = x.cuda(), w.cuda()
    assert same(O.int8_linear(gx, None, gw, None, out="int32"), linear_host(x, sx, w, sw, None, "int32"))
    for out in ("bf16", "fp16", "fp32"):
        got = O.int8_linear(gx, sx.cuda(), gw, sw.cuda(), bias=bias.cuda(), out=out)
        assert same(got, linear_host(x, sx, w, sw, bias, out)), out


@pytest.mark.parametrize("K", [1024, 1025, 4096, 20000])
def test_int8_linear_panels_of_extreme_sums(O, K):
    """-128 * -128 throughout and its neighbours through the panels, where 1024 products reach 2^24."""
    rng = np.random.default_rng(K)
    M, N = 1300, 1300
    assert O.lib().mcemu_int8_linear_workspace(M, N, K, K % 16 == 0) > 0
    x = torch.full((M, K), -128, dtype=torch.int8)
    w = torch.full((N, K), -128, dtype=torch.int8)
    w[1] = 127
    w[2, ::2] = 127
    w[3, -1] = -127
    w[4:] = int8s(rng, N - 4, K)
    w[1000:] = -128
    x[5:9] = int8s(rng, 4, K)
    x[M - 1, 0] = -127
    got = O.int8_linear(x.cuda(), None, w.cuda(), None, out="int32")
    assert same(got, linear_host(x, None, w, None, None, "int32"))


@pytest.mark.parametrize("T,N,K", [(2000, 2304, 2304), (3001, 2301, 2300), (4100, 2600, 2304)])
@pytest.mark.parametrize("out", ["fp32", "bf16"])
def test_act8_wgrad_of_whole_and_shared_tiles(O, T, N, K, out):
    """More tiles than pairs of multiprocessors: most are one pair's, those of the last round are shared."""
    rng = np.random.default_rng(T)
    dy, x = wgrad_case(rng, T, N, K)
    q, e = O.act8_compress(x.cuda())
    xq = O.act8_expand(q, e, out="fp32").cpu().double()
    ttiles, blocks = -(-T // 64), lambda n: -(-n // 256) * 2
    panels = (blocks(K) + (blocks(N) if N % 8 else 0)) * ttiles * 16384
    assert O.lib().mcemu_act8_wgrad_workspace(T, N, K, int(N % 8 == 0)) > panels + 64       # parts of shared tiles
    assert blocks(K) // 2 * (blocks(N) // 2) > 76
    got = O.act8_wgrad(dy.cuda(), q, e, out=out)
    wgrad_check(got, dy, xq, out)
    if out == "fp32":
        base = torch.from_numpy(rng.standard_normal((N, K)).astype(np.float32))
        dW = base.cuda()
        O.act8_wgrad(dy.cuda(), q, e, dW=dW, accumulate=True)
        wgrad_check(dW, dy, xq, out, base)


def test_rmsnorm_backward_joins_many_blocks(O):
    """dw from 2432 rows, a block's each: what a strand of 76 blocks would drop from 1 is kept by four
    shorter ones.  19 additions in a row, two and five joins, four roundings of a row's part."""
    T, H = 2432, 263
    dy = torch.zeros(T, H)
    dy[::32] = 0.99 * U32
    dy[0] = 1
    _, dw = O.rmsnorm_backward(dy.cuda(), torch.ones(H).cuda(), torch.ones(T).cuda(), h=torch.ones(T, H, device="cuda"))
    want = dy.double().sum(0)
    assert torch.all((dw.cpu().double() - want).abs() <= 30 * U32 * want)


@pytest.mark.parametrize("N,K", [(64, 128), (300, 200)])
def test_act8_wgrad_takes_the_accumulators_out(O, N, K):
    """One product of 2^24 and 1023 of 1/16, sixteen of which the matrix unit's accumulators drop beside it:
    at most the other 511 tokens' of its 512 are lost, and a step of the result."""
    T = 1024
    dy, x = torch.full((T, N), 1 / 16), torch.ones(T, K)
    dy[0], x[0] = 4096, 4096
    got = O.act8_wgrad(dy.bfloat16().cuda(), *O.act8_compress(x.cuda()))
    assert torch.all((got.cpu().double() - (2.0 ** 24 + 1023 / 16)).abs() <= 511 / 16 + 2)
