"""The router's choice of groups where fp32 sums of two choices cannot tell it: large biases of both signs, which cancel in the
sum but not in its roundings, and sums past the largest fp32."""
import pytest
import torch

from test_gpu_route import INF, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _cancelling(M, E, groups, large, sigmoid, seed):
    """In each group one expert with a bias of +large, one of -large, the others out of the way; scores whose differences are
    about an fp32 rounding of `large`, so that the groups' exact sums lie that close together."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    size = E // groups
    bias = torch.full((groups, size), -3.0 * large, device="cuda")
    order = torch.stack([torch.randperm(size, generator=g, device="cuda") for _ in range(groups)])
    bias.scatter_(1, order[:, :1], large)
    bias.scatter_(1, order[:, 1:2], -large)
    slope = 0.25 if sigmoid else 1.0 / E
    spread = min(0.5, 3 * large * 2.0 ** -23 / slope)
    return spread * torch.randn((M, E), generator=g, device="cuda"), bias.view(-1)


@pytest.mark.parametrize("E,groups,topk_groups,topk", [(64, 8, 4, 8), (256, 8, 4, 8), (60, 4, 2, 4), (160, 8, 3, 6),
                                                       (16, 8, 4, 2), (1024, 32, 9, 4), (32, 8, 2, 4)])
@pytest.mark.parametrize("large", [4.0, 16.0, 64.0, 256.0, 4096.0, 65536.0])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("general", [False, True])
def test_choices_that_cancel(E, groups, topk_groups, topk, large, sigmoid, general):
    logits, bias = _cancelling(max(60, 40000 // E), E, groups, large, sigmoid, E + int(large))
    if general:      # one expert out for all tokens, by a bias that the fast form leaves to the general one
        bias[bias.argmin()] = -INF
    check(logits, topk, bias=bias, sigmoid=sigmoid, groups=groups, topk_groups=topk_groups, best=2)


@pytest.mark.parametrize("E,groups", [(64, 8), (60, 6)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_some_groups_cancel(E, groups, sigmoid):
    """Groups of large roundings among groups of small ones, whose sums lie between theirs."""
    logits, bias = _cancelling(600, E, groups, 1024.0, sigmoid, 3)
    bias.view(groups, -1)[::2] = 0
    check(logits, 4, bias=bias, sigmoid=sigmoid, groups=groups, topk_groups=groups // 2, best=2)


@pytest.mark.parametrize("E,groups", [(64, 8), (60, 6), (256, 8)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("general", [False, True])
def test_sums_past_the_largest_number(E, groups, sigmoid, sign, general):
    """Two choices whose sum fp32 cannot hold: the order is that of 64 bits, and such a group has candidates."""
    g = torch.Generator(device="cuda")
    g.manual_seed(E)
    bias = (sign * torch.randint(9, 16, (groups, E // groups), generator=g, device="cuda").float() * 2.0 ** 124).view(-1)
    if sign > 0:
        bias[::3] = -1.0
    if general:
        bias[1] = -INF
    logits = torch.randn((300, E), generator=g, device="cuda")
    logits[::7, :E // 2] = -INF
    check(logits, 4, bias=bias, sigmoid=sigmoid, groups=groups, topk_groups=groups // 2, best=2)


@pytest.mark.parametrize("E,groups", [(64, 8), (60, 4), (36, 12)])
@pytest.mark.parametrize("best", [1, 2])
def test_candidates_in_fewer_groups_than_stay(E, groups, best):
    g = torch.Generator(device="cuda")
    g.manual_seed(E)
    logits = torch.randn((500, groups, E // groups), generator=g, device="cuda")
    logits[:, torch.randperm(groups, generator=g, device="cuda")[1:]] = -INF
    check(logits.view(500, E), 3, bias=0.1 * torch.randn(E, generator=g, device="cuda"), sigmoid=True, groups=groups,
          topk_groups=groups // 2, best=best)
