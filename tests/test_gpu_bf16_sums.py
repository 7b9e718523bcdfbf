"""What the bf16 products lose in their sums, which a bf16 output alone does not show: every row of x is the same, and an
fp32 bias takes the exact sums away again, so that y is what is lost."""
import pytest
import torch

from bf16_helpers import BF, F32, align, err_flag, experts, gen, operand, routes
from lora_moe_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _loss(K, run):
    """Products of one sign, in runs of `run` columns that the tensor cores add up: a run's run / 16 additions of 16 products
    each lose less than 2^-23 of its sum, the additions of the runs and of up to eight shares of K half of that."""
    return (run / 16 + (K / run + 8) / 2) * 2.0 ** -23


def _rows(M, N, K, E=1):
    """Equal rows x, weights, and -(their sums) in fp32 with the exact sums."""
    g = gen(K)
    row = (torch.rand(K, generator=g, device="cuda") + 0.5).to(BF)
    w = (torch.rand((E * N, K), generator=g, device="cuda") + 0.5).to(BF)
    s = torch.cat([p.double() @ row.double() for p in w.split(16)]).view(E, N)
    x = operand(row.expand(M, K))
    return x, experts(w.view(E, N, K)), s, -s.float()


def _check(y, s, bias, K, run):
    """sum + bias is exact (the two are within a factor of two), so that y is one rounding away."""
    off = (y.double() - (s + bias.double())).abs()
    bound = _loss(K, run) * s
    worst = (off / s).max().item()
    assert (off <= bound * (1 + 2.0 ** -8) + 2.0 ** -8 * (s + bias.double()).abs()).all(), "%g of the sum, bound %g" % (
        worst, _loss(K, run))


@pytest.mark.parametrize("M,N,K", [(3, 200, 7168), (40, 200, 7168), (65, 300, 7168), (300, 700, 7168), (300, 3000, 7168),
                                   (6000, 1100, 4096), (3000, 4096, 2048), (128, 256, 1 << 20), (5000, 1000, 30000)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_dense(M, N, K, dtype):
    x, w, s, bias = _rows(M, N, K)
    y, err = torch.empty((M, N), dtype=dtype, device="cuda"), err_flag()
    B.moe_bf16_matmul(x, w[0], y, bias=bias[0], err_flag=err)
    assert err.item() == 0
    _check(y, s, bias, K, 256 if dtype == F32 or M <= 64 else 1024)


@pytest.mark.parametrize("M,topk,E,N,K,block", [(6, 2, 4, 200, 4096, 0), (20, 2, 4, 200, 4096, 16), (1500, 2, 4, 300, 4096, 64),
                                                (4000, 2, 3, 1000, 7168, 128), (600, 2, 4, 520, 70000, 16)])
def test_grouped(M, topk, E, N, K, block):
    x, w, s, bias = _rows(M, N, K, E)
    ids = routes(M, topk, E, gen(M))
    y, err = torch.empty((M, topk, N), dtype=BF, device="cuda"), err_flag()
    if block:
        B.moe_bf16_grouped_matmul(x, w, y, *align(ids, E, block), block, bias=bias, err_flag=err)
    else:
        B.moe_bf16_grouped_matmul_naive(x, w, y, ids, bias=bias, err_flag=err)
    assert err.item() == 0
    _check(y, s[ids.long()], bias[ids.long()], K, 256 if M <= 64 else 1024)
