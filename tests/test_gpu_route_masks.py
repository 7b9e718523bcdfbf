"""Biases that mask experts by the type's lowest value, or by one near it: such experts are candidates, which come last."""
import pytest
import torch

from test_gpu_route import INF, check, route64, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("E,topk,groups,topk_groups", [(1, 1, 1, 1), (2, 2, 1, 1), (32, 6, 4, 1), (40, 8, 1, 1), (60, 20, 4, 3),
                                                       (64, 8, 8, 4), (128, 8, 1, 1), (256, 32, 8, 2), (1000, 8, 8, 4)])
@pytest.mark.parametrize("low", [torch.finfo(torch.float32).min, -3.4e38, -1e38, -1e9])
@pytest.mark.parametrize("open_", ["half", "few", "none"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("best", [1, 2])
def test_lowest_value(E, topk, groups, topk_groups, low, open_, sigmoid, best):
    g = torch.Generator(device="cuda")
    g.manual_seed(E + topk)
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    order = torch.randperm(E, generator=g, device="cuda")
    bias[order[{"half": E // 2, "few": topk // 2, "none": 0}[open_]:]] = low
    logits = torch.randn((37, E), generator=g, device="cuda")
    logits[::5, ::3] = -INF
    check(logits, topk, bias=bias, sigmoid=sigmoid, groups=groups, topk_groups=topk_groups, best=best, renormalize=False)


@pytest.mark.parametrize("E,topk,groups,topk_groups", [(5, 3, 1, 1), (64, 8, 1, 1), (64, 8, 8, 3), (300, 6, 1, 1)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_largest_value(E, topk, groups, topk_groups, sigmoid):
    """Experts that are always chosen."""
    g = torch.Generator(device="cuda")
    g.manual_seed(E)
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    bias[::4] = torch.finfo(torch.float32).max
    check(torch.randn((37, E), generator=g, device="cuda"), topk, bias=bias, sigmoid=sigmoid, groups=groups,
          topk_groups=topk_groups, best=2)


@pytest.mark.parametrize("E,topk", [(1, 1), (8, 8), (60, 5), (256, 8)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_logits_of_the_lowest_value(E, topk, sigmoid):
    logits = torch.randn((37, E), generator=torch.Generator("cuda").manual_seed(E), device="cuda")
    logits[:, ::2] = torch.finfo(torch.float32).min
    low = torch.full((1, E), torch.finfo(torch.float32).min, device="cuda")
    for bias in (None, torch.zeros(E, device="cuda")):
        if E > 1:
            check(logits, topk, bias=bias, sigmoid=sigmoid)
        # a row of nothing else: equal scores (too small for 64 bits where they are a sigmoid's), of which each has its share
        ids, weights = run(low, topk, bias=bias, sigmoid=sigmoid)
        assert ids[0].tolist() == list(range(topk)) and ((weights - 1 / topk).abs() <= 2.0 ** -19 / topk).all()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("scale", [1e-30, 1e30])
@pytest.mark.parametrize("renormalize", [False, True])
def test_weights_of_a_scale(sigmoid, scale, renormalize):
    """Scores near the smallest fp32 times a large number: an absolute error of the scores is scaled with them."""
    logits = torch.randn((50, 64), generator=torch.Generator("cuda").manual_seed(1), device="cuda") - 95
    if not sigmoid:
        logits[:, 0] = 0
    ids, weights = run(logits, 6, sigmoid=sigmoid, renormalize=renormalize, scale=scale)
    want, w64 = route64(logits, 6, sigmoid=sigmoid, renormalize=renormalize, scale=scale)
    assert torch.equal(ids.cpu(), want)
    assert ((weights.cpu().double() - w64).abs() <= 2.0 ** -19 * w64.abs() + 2.0 ** -140 * max(scale, 1)).all()
