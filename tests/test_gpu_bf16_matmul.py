"""The bf16 products against their definitions in 64 bits: exactly on whole numbers, whose products and sums fp32 holds,
and within derived bounds on others."""
import pytest
import torch

from bf16_helpers import (ACTS, BF, F32, act64, align, assert_rounded, err_flag, experts, gen, grouped64, operand, routes,
                          strided, whole)
from lora_moe_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


# ------------------------------------------------------------------ dense

def _whole_dense(M, N, K, dtype=BF, bias=None, residual=False, pad=0, ypad=0, lead=0):
    g = gen(M * 7 + N * 3 + K)
    x, w = operand(whole(g, M, K), pad), operand(whole(g, N, K), pad)
    b = None if bias is None else whole(g, N, most=9).to(bias)
    r = strided(M, N, dtype, ypad + 1).copy_(whole(g, M, N, most=9)) if residual else None
    y, err = strided(M, N, dtype, ypad, lead), err_flag()
    B.moe_bf16_matmul(x, w, y, bias=b, residual=r, err_flag=err)
    want = x.double() @ w.double().t()
    if b is not None:
        want = want + b.double()
    if r is not None:
        want = want + r.double()
    assert err.item() == 0
    assert torch.equal(y, want.to(dtype)), "%d of %d differ" % ((y != want.to(dtype)).sum(), y.numel())
    if ypad:
        assert torch.isnan(y.as_strided((M, ypad), (N + ypad, 1), y.storage_offset() + N).float()).all()


@pytest.mark.parametrize("M", [1, 8, 9, 16, 17, 33, 64, 65, 128, 129, 200, 257, 600])
@pytest.mark.parametrize("N,K", [(1, 1), (127, 16), (128, 128), (129, 130), (300, 1000), (1536, 2048), (520, 2880)])
def test_dense(M, N, K):
    _whole_dense(M, N, K)
    _whole_dense(M, N, K, F32)


@pytest.mark.parametrize("M,N,K", [(5, 264, 400), (16, 33, 77), (40, 100, 77), (300, 700, 333), (130, 512, 4096),
                                   (2000, 700, 333), (5000, 260, 129)])
@pytest.mark.parametrize("pad,ypad,lead", [(0, 1, 0), (40, 8, 8), (16, 5, 1)])
@pytest.mark.parametrize("dtype,bias,residual", [(BF, None, True), (BF, BF, False), (F32, F32, True), (F32, BF, False),
                                                 (BF, F32, True)])
def test_dense_epilogue_and_strides(M, N, K, pad, ypad, lead, dtype, bias, residual):
    _whole_dense(M, N, K, dtype, bias, residual, pad, ypad, lead)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 7168), (1, 64, 16384), (16, 128, 8192), (2048, 1100, 640), (8192, 128, 256),
                                   (300, 20000, 128), (6000, 300, 1), (1500, 2049, 500), (20000, 1, 300), (3, 9000, 9000),
                                   (16, 5000, 8192), (16, 512, 65600), (9, 700, 49152), (70, 128, 16384), (1, 40000, 520),
                                   (100, 256, 7168), (4096, 256, 1024)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_dense_long(M, N, K, dtype):
    _whole_dense(M, N, K, dtype, residual=True)


@pytest.mark.parametrize("M", [3, 40, 100, 4000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_residual_in_place(M, dtype):
    g = gen(M)
    x, w = operand(whole(g, M, 200)), operand(whole(g, 260, 200))
    y = whole(g, M, 260, most=9).to(dtype)
    want = x.double() @ w.double().t() + y.double()
    B.moe_bf16_matmul(x, w, y, residual=y)
    assert torch.equal(y, want.to(dtype))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [2, 13, 50, 100, 3000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_dense_random(act, M, dtype):
    g = gen(M)
    K, N = 1000, 300
    x, w = (operand(torch.randn((n, K), generator=g, device="cuda") * s) for n, s in ((M, 2), (N, K ** -0.5)))
    b = torch.randn(N, generator=g, device="cuda")
    r = torch.randn((M, N), generator=g, device="cuda").to(dtype)
    y = torch.empty((M, N), dtype=dtype, device="cuda")
    B.moe_bf16_matmul(x, w, y, bias=b, residual=r, activation=ACTS[act])
    v = x.double() @ w.double().t() + b.double()
    ref = act64(v, act)
    # K + 16 additions of exact products (and of the shares of K), each of which may truncate: 2^-23 of the sum of
    # magnitudes at most; the activations' slope is at most 1.13, their own error 2^-20 of the value, and gelu's
    # argument is rounded (2^-23 of |v|, times a slope of v * phi(v) * v, below 0.5)
    size = x.double().abs() @ w.double().abs().t() + b.double().abs()
    bound = 1.13 * (K + 16) * 2.0 ** -23 * size + 2.0 ** -20 * ref.abs() + 2.0 ** -23 * v.abs() + 2.0 ** -24 * r.double().abs()
    assert_rounded(y, ref + r.double(), bound, act)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [2, 40, 100, 6000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_activations(act, M, dtype):
    """Every product is by one or zero, so that the activation's own error shows: the header's bound for a bf16 y; for an
    fp32 one a few roundings (of the argument, 2^-23 of |v| times a slope of at most 1.13, and of the result)."""
    N = 64
    v = (torch.arange(M * N, device="cuda").double() / (M * N) - 0.5) * 60
    x = operand(v.view(M, N))
    y = torch.empty((M, N), dtype=dtype, device="cuda")
    B.moe_bf16_matmul(x, torch.eye(N, device="cuda").to(BF), y, activation=ACTS[act])
    ref = act64(x.double(), act)
    if dtype == BF:
        bound = torch.maximum(2.0 ** -16 * ref.abs(), 2.0 ** -21 * x.double().abs())
    else:
        bound = 2.0 ** -20 * ref.abs() + 2.0 ** -22 * x.double().abs() * (act != "none")
    assert_rounded(y, ref, bound, act)


@pytest.mark.parametrize("M,N,K", [(1, 200, 7168), (12, 200, 7168), (60, 200, 7168), (300, 200, 7168), (6000, 512, 7168)])
def test_fp32_sums_do_not_drift(M, N, K):
    """Rows whose products all have one sign: what truncating additions lose adds up.  Runs of at most 256 columns lose
    2^-23 of their sum in each of 16 additions, so all of K loses no more than 16 * 2^-23 of it, and the runs' additions
    (28, and 8 of shares of K) half of 2^-23 each."""
    g = gen(K)
    x, w = (operand(torch.rand((n, K), generator=g, device="cuda") + 0.5) for n in (M, N))
    y = torch.empty((M, N), dtype=F32, device="cuda")
    B.moe_bf16_matmul(x, w, y)
    ref = x.double() @ w.double().t()
    assert ((y.double() - ref).abs() <= (16 + 36 / 2) * 2.0 ** -23 * ref).all(), ((y.double() - ref) / ref).abs().max()


def test_dense_empty():
    w = operand(whole(gen(0), 64, 64))
    B.moe_bf16_matmul(torch.empty((0, 64), dtype=BF, device="cuda"), w, torch.empty((0, 64), dtype=BF, device="cuda"))


@pytest.mark.parametrize("M", [3, 40, 100, 4000])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_dense_nan_stays_in_its_row_and_column(M, bad):
    g = gen(M)
    x, w = operand(whole(g, M, 256) + 5), operand(whole(g, 300, 256) + 5)
    x[1, 200] = bad
    w[77, 3] = bad
    y, err = torch.empty((M, 300), dtype=BF, device="cuda"), err_flag()
    B.moe_bf16_matmul(x, w, y, err_flag=err)
    off = ~torch.isfinite(y)
    assert off[1].all() and off[:, 77].all()
    off[1] = False
    off[:, 77] = False
    assert not off.any() and err.item() == 0


# ------------------------------------------------------------------ over experts

def _whole_grouped(M, topk, E, N, K, block, per_pair=False, weighted=False, bias=None, kind="even", pad=0, ypad=0):
    g = gen(M + E + N + K)
    ids = routes(M, topk, E, g, kind)
    x, w = operand(whole(g, M * topk if per_pair else M, K), pad), experts(whole(g, E, N, K), pad)
    b = None if bias is None else whole(g, E, N, most=9).to(bias)
    weights = torch.randint(1, 5, (M, topk), generator=g, device="cuda").float() if weighted else None
    y = strided(M * topk, N, BF, ypad).as_strided((M, topk, N), (topk * (N + ypad), N + ypad, 1))
    err = err_flag()
    more = dict(bias=b, topk_weights=weights, x_per_pair=per_pair, err_flag=err)
    if block:
        B.moe_bf16_grouped_matmul(x, w, y, *align(ids, E, block), block, **more)
    else:
        B.moe_bf16_grouped_matmul_naive(x, w, y, ids, **more)
    want = grouped64(x, w, ids, per_pair, b, weights=weights)[0].view(M, topk, N).to(BF)
    assert err.item() == 0
    assert torch.equal(y, want), "%d of %d differ" % ((y != want).sum(), y.numel())


@pytest.mark.parametrize("M,topk,E", [(1, 1, 1), (1, 8, 16), (5, 2, 4), (17, 3, 60), (100, 4, 8), (200, 2, 2)])
@pytest.mark.parametrize("N,K", [(1, 1), (130, 77), (256, 320), (700, 1032)])
@pytest.mark.parametrize("block", [0, 16, 32, 64, 128])
def test_grouped(M, topk, E, N, K, block):
    _whole_grouped(M, topk, E, N, K, block)


@pytest.mark.parametrize("M,topk,E,N,K", [(3, 2, 5, 264, 400), (40, 4, 12, 100, 77), (900, 2, 3, 300, 129),
                                          (2500, 2, 9, 520, 200)])
@pytest.mark.parametrize("block", [0, 16, 64, 128])
@pytest.mark.parametrize("per_pair,weighted,bias,kind,pad,ypad", [
    (True, False, None, "even", 0, 1), (False, True, BF, "skew", 8, 0), (True, True, F32, "one", 40, 8)])
def test_grouped_epilogue_and_strides(M, topk, E, N, K, block, per_pair, weighted, bias, kind, pad, ypad):
    _whole_grouped(M, topk, E, N, K, block, per_pair, weighted, bias, kind, pad, ypad)


@pytest.mark.parametrize("M,topk,E,N,K,block", [(4096, 2, 8, 300, 256, 128), (1024, 8, 128, 256, 192, 64),
                                                (700, 4, 16, 1030, 500, 32), (16, 8, 128, 1536, 2048, 16),
                                                (64, 4, 128, 400, 2880, 16), (1, 8, 128, 1536, 2048, 0),
                                                (16, 4, 32, 4096, 3000, 0)])
def test_grouped_long(M, topk, E, N, K, block):
    _whole_grouped(M, topk, E, N, K, block, kind="skew")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,E,block", [(6, 4, 0), (6, 4, 16), (1200, 4, 64)])
def test_grouped_random(act, M, E, block):
    g = gen(M)
    K, N, topk = 500, 200, 2
    ids = routes(M, topk, E, g)
    x = operand(torch.randn((M, K), generator=g, device="cuda") * 2)
    w = experts(torch.randn((E, N, K), generator=g, device="cuda") * K ** -0.5)
    b = torch.randn((E, N), generator=g, device="cuda").to(BF)
    weights = torch.rand((M, topk), generator=g, device="cuda")
    y = torch.empty((M, topk, N), dtype=BF, device="cuda")
    more = dict(bias=b, activation=ACTS[act], topk_weights=weights)
    if block:
        B.moe_bf16_grouped_matmul(x, w, y, *align(ids, E, block), block, **more)
    else:
        B.moe_bf16_grouped_matmul_naive(x, w, y, ids, **more)
    ref, size = grouped64(x, w, ids, False, b, act, weights)
    bound = 1.13 * (K + 16) * 2.0 ** -23 * (size + 4) + 2.0 ** -19 * (ref.abs() + 1)
    assert_rounded(y.view(M * topk, N), ref, bound, act)


@pytest.mark.parametrize("M,topk,E,block", [(30, 2, 6, 16), (30, 2, 6, 64), (1500, 2, 4, 64), (12, 2, 6, 0)])
def test_pairs_of_no_expert_are_left_alone(M, topk, E, block):
    """Ids out of range are dropped by the align and skipped, and reported, by the naive form."""
    g = gen(M)
    ids = routes(M, topk, E, g)
    ids[::3, 0] = -1
    ids[1::3, 1] = E
    x, w = operand(whole(g, M, 128)), experts(whole(g, E, 200, 128))
    y, err = torch.full((M, topk, 200), 7.0, dtype=BF, device="cuda"), err_flag()
    if block:
        B.moe_bf16_grouped_matmul(x, w, y, *align(ids, E, block), block, err_flag=err)
        assert err.item() == 0
    else:
        B.moe_bf16_grouped_matmul_naive(x, w, y, ids, err_flag=err)
        assert err.item() == B.DEVERR_EXPERT_ID
    bad = ((ids < 0) | (ids >= E)).reshape(-1)
    want = grouped64(x, w, ids, False)[0].to(BF)
    got = y.view(M * topk, 200)
    assert (got[bad] == 7).all() and torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("M,E,block", [(20, 6, 16), (1500, 4, 64)])
def test_entries_out_of_range_are_skipped_and_reported(M, E, block):
    g = gen(M)
    ids = routes(M, 2, E, g)
    x, w = operand(whole(g, M, 128)), experts(whole(g, E, 200, 128))
    sorted_ids, expert_ids, padded = align(ids, E, block)
    expert_ids.view(-1)[0] = E + 5
    at = block + 1                                  # in the second block
    f = sorted_ids.view(-1)[at].item()
    sorted_ids.view(-1)[at] = -4
    skipped = [v for v in sorted_ids.view(-1)[:block].tolist() if v < M * 2] + [f]
    y, err = torch.full((M, 2, 200), 7.0, dtype=BF, device="cuda"), err_flag()
    B.moe_bf16_grouped_matmul(x, w, y, sorted_ids, expert_ids, padded, block, err_flag=err)
    assert err.item() == B.DEVERR_EXPERT_ID | B.DEVERR_PAIR_ID
    keep = torch.ones(M * 2, dtype=torch.bool, device="cuda")
    keep[skipped] = False
    want = grouped64(x, w, ids, False)[0].to(BF)
    got = y.view(M * 2, 200)
    assert (got[~keep] == 7).all() and torch.equal(got[keep], want[keep])


def test_grouped_empty():
    w = experts(whole(gen(0), 4, 64, 64))
    ids = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    y = torch.empty((0, 2, 64), dtype=BF, device="cuda")
    x = torch.empty((0, 64), dtype=BF, device="cuda")
    B.moe_bf16_grouped_matmul_naive(x, w, y, ids)
    B.moe_bf16_grouped_matmul(x, w, y, *align(ids, 4, 16), 16)
