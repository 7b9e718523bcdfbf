"""The bf16 products over experts where a call is at one of its limits: single pairs whose K a cluster of the narrow kernel
splits, and a count of positions beyond what the sorted arrays hold."""
import pytest
import torch

from bf16_helpers import BF, align, err_flag, experts, gen, grouped64, operand, routes, whole
from lora_moe_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("M,topk,N,K", [(1, 1, 1024, 131072), (2, 1, 1024, 65600), (1, 2, 1000, 70001), (3, 1, 896, 70000),
                                        (3, 1, 1000, 70000), (5, 1, 760, 49000), (2, 1, 2400, 40000), (2, 2, 1200, 40000),
                                        (4, 1, 2400, 20000), (1, 1, 1, 1 << 28)])
def test_single_pairs_whose_k_is_split(M, topk, N, K):
    """More than 256 MB of weights, fewer items than SMs: 8, 16, 21, 24, 30, 38, 40 and 76 of them, in clusters of 8 to 2."""
    g = gen(K)
    E = max(topk, 2 if N > 1 else 1)
    ids = routes(M, topk, E, g)
    x, w = operand(whole(g, M, K, most=1)), experts(whole(g, E, N, K, most=1))
    bias = whole(g, E, N, most=9).to(BF)
    y, err = torch.empty((M, topk, N), dtype=BF, device="cuda"), err_flag()
    B.moe_bf16_grouped_matmul_naive(x, w, y, ids, bias=bias, err_flag=err)
    want = torch.stack([x[f // topk].double() @ w[e].double().t() + bias[e].double()
                        for f, e in enumerate(ids.view(-1).tolist())])
    assert err.item() == 0 and torch.equal(y.view(-1, N), want.to(BF))


@pytest.mark.parametrize("M,topk,E,N,K,block", [(2, 2, 128, 256, 2048, 16), (2, 2, 128, 256, 2048, 64), (40, 2, 8, 2000, 200, 16),
                                                (1500, 2, 4, 300, 200, 64), (1500, 2, 4, 300, 1100, 16)])
@pytest.mark.parametrize("count", [1 << 30, 0x7FFFFFFF])
def test_more_positions_than_the_arrays_hold(M, topk, E, N, K, block, count):
    """The count is cut to the arrays' own; behind the align's blocks they hold sentinels."""
    g = gen(M)
    ids = routes(M, topk, E, g)
    x, w = operand(whole(g, M, K)), experts(whole(g, E, N, K))
    sorted_ids, expert_ids, padded = align(ids, E, block)
    n = padded.item()
    sorted_ids.view(-1)[n:] = M * topk
    expert_ids.view(-1)[n // block:] = E - 1
    padded.fill_(count)
    y, err = torch.full((M, topk, N), 7.0, dtype=BF, device="cuda"), err_flag()
    B.moe_bf16_grouped_matmul(x, w, y, sorted_ids, expert_ids, padded, block, err_flag=err)
    # clusters that split K are as many as an align's blocks: what is left over is reported
    assert err.item() in (0, B.DEVERR_CAPACITY)
    assert E != 128 or err.item() == B.DEVERR_CAPACITY
    assert torch.equal(y.view(M * topk, N), grouped64(x, w, ids, False)[0].to(BF))


@pytest.mark.parametrize("M,block", [(20, 16), (1500, 64)])
@pytest.mark.parametrize("count", [0, -1, -(1 << 31)])
def test_no_positions(M, block, count):
    g = gen(M)
    ids = routes(M, 2, 4, g)
    x, w = operand(whole(g, M, 200)), experts(whole(g, 4, 300, 200))
    sorted_ids, expert_ids, padded = align(ids, 4, block)
    padded.fill_(count)
    y, err = torch.full((M, 2, 300), 7.0, dtype=BF, device="cuda"), err_flag()
    B.moe_bf16_grouped_matmul(x, w, y, sorted_ids, expert_ids, padded, block, err_flag=err)
    assert err.item() == 0 and (y == 7).all()
