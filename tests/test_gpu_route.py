"""The router against its definition in 64 bits: the experts exactly, the weights within derived bounds."""
import pytest
import torch

from lora_moe_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def route64(logits, topk, bias=None, sigmoid=False, renormalize=True, scale=1.0, groups=1, topk_groups=1, best=1):
    """One row at a time, in Python's own arithmetic on 64-bit numbers."""
    x = logits.to(F64).cpu()
    M, E = x.shape
    if sigmoid:
        s = 1 / (1 + torch.exp(-x))
    else:
        s = torch.exp(x - x.amax(1, keepdim=True))
        s = s / s.sum(1, keepdim=True)
    c = s if bias is None else s + bias.to(F64).cpu()
    s, c, x = s.tolist(), c.tolist(), x.tolist()
    ids, weights = [], []
    for m in range(M):
        candidate = [x[m][e] > -INF and c[m][e] > -INF for e in range(E)]
        order = c[m] if bias is not None else x[m]     # (a sigmoid of large logits is one for all of them)
        if groups > topk_groups:
            size, worth = E // groups, []
            for g in range(groups):
                own = order if best == 1 else c[m]
                top = sorted((own[e] for e in range(g * size, (g + 1) * size) if candidate[e]), reverse=True)[:best]
                worth.append(sum(top) if top else -INF)
            stay = sorted(range(groups), key=lambda g: (-worth[g], g))[:topk_groups]
            candidate = [candidate[e] and e // size in stay for e in range(E)]
        chosen = sorted(range(E), key=lambda e: (not candidate[e], -order[e] if candidate[e] else 0, e))[:topk]
        w = [s[m][e] if candidate[e] else 0.0 for e in chosen]
        total = sum(w)
        if renormalize and total > 0:
            w = [v / total for v in w]
        ids.append(chosen)
        weights.append([v * scale for v in w])
    return torch.tensor(ids, dtype=I32), torch.tensor(weights, dtype=F64)


def run(logits, topk, bias=None, sigmoid=False, renormalize=True, scale=1.0, groups=1, topk_groups=1, best=1, stream=None):
    M = logits.shape[0]
    ids = torch.full((M, topk), -7, dtype=I32, device="cuda")
    weights = torch.full((M, topk), -7.0, device="cuda")
    B.moe_route(logits, ids, weights, bias=bias, scoring=B.ROUTE_SIGMOID if sigmoid else B.ROUTE_SOFTMAX,
                renormalize=renormalize, scale=scale, num_groups=groups, topk_groups=topk_groups, group_best=best,
                stream=stream)
    return ids, weights


def check(logits, topk, **kw):
    ids, weights = run(logits, topk, **kw)
    want, w64 = route64(logits, topk, **kw)
    assert torch.equal(ids.cpu(), want), "%d rows differ" % (ids.cpu() != want).any(1).sum()
    # the header's bound
    assert ((weights.cpu().double() - w64).abs() <= 2.0 ** -19 * w64.abs() + 2.0 ** -140).all()


def _logits(M, E, dtype=F32, seed=0, scale=1.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + M * 1000 + E)
    return (scale * torch.randn((M, E), generator=g, device="cuda")).to(dtype)


def _bias(E, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + E)
    return 0.1 * torch.randn(E, generator=g, device="cuda")


@pytest.mark.parametrize("M", [1, 2, 5, 67])
@pytest.mark.parametrize("E,topk", [(1, 1), (2, 2), (8, 2), (31, 4), (32, 32), (33, 5), (60, 4), (64, 8), (128, 8),
                                    (130, 32), (256, 8), (384, 6), (511, 3), (512, 10), (1000, 17), (1024, 8)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_softmax(M, E, topk, dtype):
    check(_logits(M, E, dtype), topk)
    check(_logits(M, E, dtype), topk, renormalize=False, scale=2.5)


@pytest.mark.parametrize("E,topk", [(8, 2), (60, 4), (128, 8), (256, 8), (300, 6), (1024, 32)])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
def test_bias(E, topk, dtype, sigmoid, renormalize):
    check(_logits(300, E, dtype), topk, bias=_bias(E), sigmoid=sigmoid, renormalize=renormalize, scale=1.5)


@pytest.mark.parametrize("E,groups,topk_groups,topk", [(256, 8, 4, 8), (128, 4, 1, 8), (64, 16, 3, 6), (60, 4, 2, 4),
                                                       (160, 8, 3, 6), (36, 12, 5, 7), (512, 32, 9, 10), (1024, 2, 1, 20),
                                                       (32, 32, 8, 8), (16, 2, 2, 4), (6, 3, 2, 4)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("sigmoid,biased", [(False, False), (True, True), (True, False), (False, True)])
def test_groups(E, groups, topk_groups, topk, best, sigmoid, biased):
    check(_logits(150, E, F32 if biased else BF), topk, bias=_bias(E) if biased else None, sigmoid=sigmoid, groups=groups,
          topk_groups=topk_groups, best=best)


@pytest.mark.parametrize("M,E", [(3000, 256), (5000, 64)])
def test_many_tokens(M, E):
    check(_logits(M, E), 8, bias=_bias(E), sigmoid=True, groups=8, topk_groups=4, best=2, scale=2.5)


@pytest.mark.parametrize("E,topk,groups,topk_groups,best", [(64, 2, 1, 1, 1), (128, 8, 1, 1, 1), (128, 4, 4, 2, 2),
                                                            (256, 8, 8, 4, 2), (256, 6, 2, 1, 1), (256, 8, 8, 1, 2),
                                                            (64, 8, 16, 9, 2)])
@pytest.mark.parametrize("sigmoid,biased,dtype,renormalize", [(False, False, BF, True), (True, True, F32, True),
                                                              (False, True, F32, False), (True, False, BF, False),
                                                              (False, False, F32, False)])
def test_a_prefill(E, topk, groups, topk_groups, best, sigmoid, biased, dtype, renormalize):
    """Several tokens a warp, one after the other; some rows with masked experts, ties, or few candidates."""
    logits = _logits(4261, E, dtype)
    logits[::97, ::3] = -INF
    logits[::89, 2:] = -INF
    logits[5::101] = logits[5::101].round()
    check(logits, topk, bias=_bias(E) if biased else None, sigmoid=sigmoid, renormalize=renormalize, scale=1.5, groups=groups,
          topk_groups=topk_groups, best=best)


def test_a_prefill_with_rows_that_are_no_numbers():
    E = 128
    logits = _logits(4400, E)
    logits[7, 9] = float("nan")
    logits[4399] = INF
    ids, weights = run(logits, 8)
    bad = torch.isnan(weights).all(1)
    assert bad.nonzero().flatten().tolist() == [7, 4399] and not torch.isnan(weights[~bad]).any()
    assert (ids.sort(1).values.diff(dim=1) > 0).all() and ((ids >= 0) & (ids < E)).all()
    bias = _bias(E)
    bias[3] = float("nan")
    ids, weights = run(logits, 8, bias=bias, sigmoid=True)
    assert torch.isnan(weights).all() and (ids.sort(1).values.diff(dim=1) > 0).all()


@pytest.mark.parametrize("sigmoid", [False, True])
def test_a_prefill_of_near_ties(sigmoid):
    """Choices a fraction of an fp32 rounding apart in every row, and in the groups' worth."""
    M, E = 4300, 64
    logits = _logits(1, E, F32, 5)
    s = torch.sigmoid(logits[0].double()) if sigmoid else torch.softmax(logits[0].double(), 0)
    bias = (0.7 - s).float()
    logits = logits + 1e-7 * torch.randn((M, E), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    check(logits, 8, bias=bias, sigmoid=sigmoid)
    check(logits, 8, bias=bias, sigmoid=sigmoid, groups=4, topk_groups=2, best=2)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups,best", [(1, 1), (8, 1), (8, 2)])
def test_ties_take_the_lowest_index(sigmoid, biased, groups, best):
    """A few distinct logits for all experts."""
    E = 128
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    logits = torch.randint(-2, 3, (200, E), generator=g, device="cuda").float()
    bias = torch.randint(0, 2, (E,), generator=g, device="cuda").float() * 0.25 if biased else None
    check(logits, 8, bias=bias, sigmoid=sigmoid, groups=groups, topk_groups=min(groups, 3), best=best)
    check(torch.zeros_like(logits), 32, bias=None if bias is None else 0 * bias, sigmoid=sigmoid, groups=groups,
          topk_groups=min(groups, 3), best=best)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_neighbours_that_fp32_scores_cannot_tell_apart(sigmoid):
    """Choices a fraction of an fp32 rounding apart: the order is that of 64 bits."""
    M, E = 400, 64
    logits = _logits(M, E, F32, 5)
    s = torch.sigmoid(logits[0].double()) if sigmoid else torch.softmax(logits[0].double(), 0)
    bias = (0.7 - s).float()                          # row 0: every choice is 0.7, but for the bias's rounding
    logits = (logits[:1] + 1e-7 * torch.randn((M, E), device="cuda", generator=torch.Generator("cuda").manual_seed(1)))
    check(logits, 8, bias=bias, sigmoid=sigmoid)
    check(logits, 8, bias=bias, sigmoid=sigmoid, groups=4, topk_groups=2, best=2)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups", [1, 4])
def test_masked_experts(sigmoid, biased, groups):
    """-inf: no candidates, in a row with fewer candidates than places, and in one with none."""
    E = 40
    logits = _logits(6, E)
    logits[0, ::2] = -INF
    logits[1, 3:] = -INF
    logits[2] = -INF
    logits[3, 10:] = -INF
    logits[4, :-1] = -INF
    check(logits, 8, bias=_bias(E) if biased else None, sigmoid=sigmoid, groups=groups, topk_groups=min(groups, 2), best=2)
    check(logits, 8, bias=_bias(E) if biased else None, sigmoid=sigmoid, groups=groups, topk_groups=min(groups, 2), best=1,
          renormalize=False)


def test_bias_of_minus_infinity_masks():
    bias = _bias(20)
    bias[4:9] = -INF
    check(_logits(30, 20), 18, bias=bias, sigmoid=True)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups", [1, 4])
def test_nan_and_infinity(sigmoid, biased, groups):
    """Ids stay distinct and in range; the weights of such a row are NaN, those of others are not touched by it."""
    E = 64
    logits = _logits(5, E)
    logits[1, 7] = float("nan")
    logits[2] = float("nan")
    logits[3, 9] = INF
    kw = dict(bias=_bias(E) if biased else None, sigmoid=sigmoid, groups=groups, topk_groups=min(2, groups), best=2)
    ids, weights = run(logits, 8, **kw)
    assert ((ids >= 0) & (ids < E)).all()
    assert (ids.sort(1).values.diff(dim=1) > 0).all()
    bad = torch.isnan(weights)
    assert bad[1].all() and bad[2].all() and bad[3].all() == (not sigmoid) and not bad[0].any() and not bad[4].any()
    if sigmoid:     # (a softmax over a NaN leaves no expert a score)
        assert not (ids[1] == 7).any()
        check(logits[3:4], 8, **kw)
    bias = _bias(E)
    bias[5] = float("nan")
    ids, weights = run(logits[:1], 8, bias=bias, sigmoid=sigmoid)
    assert torch.isnan(weights).all() and (ids.sort(1).values.diff(dim=1) > 0).all()


@pytest.mark.parametrize("sigmoid", [False, True])
def test_large_logits(sigmoid):
    """Scores that round to one or to nothing: the logits still decide."""
    logits = _logits(50, 96, F32, scale=60)
    ids, weights = run(logits, 6, sigmoid=sigmoid)
    want = torch.sort(logits.double(), dim=1, descending=True, stable=True).indices[:, :6]
    assert torch.equal(ids.long(), want) and torch.isfinite(weights).all()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("M,E,groups,topk_groups,topk", [(40, 200, 4, 3, 16), (3, 200, 5, 4, 16), (40, 256, 8, 4, 8),
                                                         (300, 60, 4, 2, 10), (20, 64, 2, 1, 32)])
@pytest.mark.parametrize("scale", [1.0, 300.0])
@pytest.mark.parametrize("bad", [False, True])
def test_logits_decide_within_groups_chosen_by_scores(sigmoid, M, E, groups, topk_groups, topk, scale, bad):
    """Scores that are all one, or zero, in any arithmetic, and those that are close, by their logits."""
    x = _logits(M, E, BF, scale=scale)
    if bad:      # rows that the general form takes
        x[:, 0] = INF if sigmoid else x[:, 1]
        x[:, E // groups:E // groups * 2] = x[:, :1]
    check(x, topk, sigmoid=sigmoid, groups=groups, topk_groups=topk_groups, best=2, renormalize=False)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,topk", [(16, 5), (64, 16), (200, 8), (256, 20)])
@pytest.mark.parametrize("scale", [10.0, 60.0])
@pytest.mark.parametrize("masked", [False, True])
def test_weights_of_far_logits(sigmoid, renormalize, biased, E, topk, scale, masked):
    """Differences of logits that fp32 rounds, and chosen experts whose scores are all tiny: a bias chooses them."""
    x = _logits(60, E, F32, scale=scale)
    bias = None
    if biased:
        bias = 4 * torch.rand(E, generator=torch.Generator().manual_seed(E)).cuda()
        x = x - 3 * scale * (bias > bias.median())
    if masked:      # all but few: rows that the general form takes
        x[:, topk - 2:] = -INF
    check(x, topk, bias=bias, sigmoid=sigmoid, renormalize=renormalize)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("pad,lead", [(1, 0), (8, 8), (3, 5)])
@pytest.mark.parametrize("E", [8, 64, 100, 256, 520])
def test_strided_rows(dtype, pad, lead, E):
    raw = torch.full((40 * (E + pad) + lead,), float("nan"), dtype=dtype, device="cuda")
    x = raw[lead:].view(40, E + pad)[:, :E]
    x.copy_(_logits(40, E, dtype))
    check(x, 4, bias=_bias(E + 1)[1:], sigmoid=True)


def test_empty():
    run(torch.empty((0, 64), device="cuda"), 4)


def test_feeds_the_align():
    """ids go to the plain align as they are."""
    ids, weights = run(_logits(100, 32), 4)
    buf = B.AlignBuffers(100, 4, 32, 1, 1, 16)
    err = torch.zeros(1, dtype=I32, device="cuda")
    B.moe_align_block_size(ids, 32, 16, buf.sorted_token_ids, buf.expert_ids, buf.num_tokens_post_padded,
                           workspace=buf.workspace, err_flag=err)
    n = buf.num_tokens_post_padded.item()
    pairs = buf.sorted_token_ids.view(-1)[:n]
    assert err.item() == 0 and torch.equal(pairs[pairs < 400].sort().values, torch.arange(400, dtype=I32, device="cuda"))
