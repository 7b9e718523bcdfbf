"""The 8-bit products, dense and over experts, against their definition in 64 bits."""
import pytest
import torch

from fp8_helpers import F8, assert_bf16_close, f8_rows, f8_weight, product64, strided
from lora_moe_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _dense(M, N, K, pad=0, ypad=0):
    g = _gen(M + 3 * N + 5 * K)
    x, xs = f8_rows(M, K, g, pad)
    w, ws = f8_weight(N, K, g, pad=pad)
    y, err = strided(M, N, BF, ypad), _err()
    B.moe_fp8_matmul(x, xs, w, ws, y, err_flag=err)
    assert err.item() == 0
    ref, bound = product64(x, xs, w, ws)
    assert_bf16_close(y, ref, bound, "dense %d %d %d" % (M, N, K))
    if ypad:
        assert torch.isnan(y.as_strided((M, N + ypad), (N + ypad, 1))[:, N:].float()).all()


@pytest.mark.parametrize("M", [1, 15, 17, 33, 64, 65, 200, 257, 600])
@pytest.mark.parametrize("N,K", [(1, 1), (127, 16), (128, 128), (129, 130), (300, 1000), (1536, 2048), (520, 2880)])
def test_dense(M, N, K):
    _dense(M, N, K)


@pytest.mark.parametrize("M,N,K", [(5, 264, 400), (40, 100, 77), (300, 700, 333), (130, 512, 4096), (2000, 700, 333),
                                   (5000, 260, 129)])
@pytest.mark.parametrize("pad,ypad", [(0, 1), (40, 8), (16, 5)])
def test_dense_strided(M, N, K, pad, ypad):
    _dense(M, N, K, pad, ypad)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 7168), (1, 64, 16384), (16, 128, 8192), (2048, 1100, 640),
                                   (8192, 128, 256), (300, 20000, 128), (6000, 300, 1), (1500, 2049, 500), (20000, 1, 300),
                                   (3, 9000, 9000), (16, 5000, 8192), (16, 512, 65600), (9, 700, 49152), (70, 128, 16384)])
def test_dense_long(M, N, K):
    _dense(M, N, K)


def test_dense_empty():
    g = _gen(0)
    w, ws = f8_weight(64, 64, g)
    B.moe_fp8_matmul(torch.empty((0, 64), dtype=F8, device="cuda"), torch.empty((0, 1), device="cuda"), w, ws,
                     torch.empty((0, 64), dtype=BF, device="cuda"))


@pytest.mark.parametrize("M", [3, 40, 300, 4000])
def test_dense_nan_stays_in_its_row_and_column(M):
    g = _gen(M)
    x, xs = f8_rows(M, 256, g)
    w, ws = f8_weight(300, 256, g)
    x.view(torch.uint8)[1, 200] = 0x7f
    w.view(torch.uint8)[77, 3] = 0xff
    y, err = torch.empty((M, 300), dtype=BF, device="cuda"), _err()
    B.moe_fp8_matmul(x, xs, w, ws, y, err_flag=err)
    bad = torch.isnan(y)
    assert bad[1].all() and bad[:, 77].all()
    bad[1] = False
    bad[:, 77] = False
    assert not bad.any() and err.item() == 0


@pytest.mark.parametrize("M", [2, 40, 300, 20000])
def test_dense_infinite_and_zero_scales(M):
    g = _gen(M)
    x, xs = f8_rows(M, 384, g)
    w, ws = f8_weight(128, 384, g)
    xs[0] = 0
    xs[1, 2] = float("inf")
    y = torch.empty((M, 128), dtype=BF, device="cuda")
    B.moe_fp8_matmul(x, xs, w, ws, y)
    assert (y[0] == 0).all() and not torch.isfinite(y[1]).any()
    if M > 2:
        assert torch.isfinite(y[2:]).all()


# ------------------------------------------------------------------ over experts

def _route(M, topk, E, g, kind):
    if kind == "one":                       # every token to the same experts
        ids = torch.arange(topk, device="cuda").expand(M, topk) % E
    else:
        p = torch.ones(E, device="cuda") if kind == "even" else 1.0 / torch.arange(1, E + 1, device="cuda") ** 1.5
        ids = torch.multinomial(p.expand(max(M, 1), E), topk, generator=g)[:M]
    return ids.to(torch.int32).contiguous()


def _align(ids, E, block):
    M, topk = ids.shape
    buf = B.AlignBuffers(M, topk, E, 1, 1, block)
    B.moe_align_block_size(ids, E, block, buf.sorted_token_ids, buf.expert_ids, buf.num_tokens_post_padded,
                           workspace=buf.workspace)
    return buf.sorted_token_ids, buf.expert_ids, buf.num_tokens_post_padded


def _reference(x, xs, w, ws, ids, per_pair, weights):
    M, topk = ids.shape
    N = w.shape[1]
    flat = ids.reshape(-1).long()
    ref = torch.zeros((M * topk, N), dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(ref)
    for e in flat.unique().tolist():
        if not 0 <= e < w.shape[0]:
            continue
        f = torch.nonzero(flat == e)[:, 0]
        r = f if per_pair else f // topk
        rows = x.double()[r]
        ref[f], bound[f] = product64(rows, xs[r], w[e], ws[e])
    if weights is not None:
        ref, bound = ref * weights.reshape(-1, 1).double(), bound * weights.reshape(-1, 1).double().abs()
        bound = bound + ref.abs() * 2.0 ** -24
    return ref, bound


def _grouped(M, topk, E, K, N, block, kind="even", per_pair=False, weighted=False, pad=0, ypad=0, seed=0):
    """block 0: the naive assignment."""
    g = _gen(M + topk + E + K + N + block + seed)
    x, xs = f8_rows(M * topk if per_pair else M, K, g, pad)
    w, ws = f8_weight(N, K, g, E, pad)
    ids = _route(M, topk, E, g, kind)
    weights = torch.rand((M, topk), generator=g, device="cuda") if weighted else None
    y, err = strided(M * topk, N, BF, ypad).unflatten(0, (M, topk)), _err()
    kw = dict(topk_weights=weights, x_per_pair=per_pair, err_flag=err)
    if block:
        B.moe_fp8_grouped_matmul(x, xs, w, ws, y, *_align(ids, E, block), block, **kw)
    else:
        B.moe_fp8_grouped_matmul_naive(x, xs, w, ws, y, ids, **kw)
    assert err.item() == 0
    ref, bound = _reference(x, xs, w, ws, ids, per_pair, weights)
    assert_bf16_close(y.reshape(M * topk, N), ref, bound, "grouped")


@pytest.mark.parametrize("block", [0, 16, 32, 64, 128])
@pytest.mark.parametrize("M,topk,E,K,N,kind", [(1, 1, 1, 16, 1, "even"), (1, 8, 8, 256, 384, "even"),
                                               (16, 8, 128, 512, 300, "skew"), (19, 2, 8, 2880, 130, "even"),
                                               (150, 4, 60, 130, 257, "skew"), (200, 1, 3, 400, 640, "one")])
@pytest.mark.parametrize("per_pair,weighted", [(False, False), (True, True)])
def test_grouped(block, M, topk, E, K, N, kind, per_pair, weighted):
    if block == 0 and M > 20:
        pytest.skip("the naive assignment is for few tokens")
    _grouped(M, topk, E, K, N, block, kind, per_pair, weighted)


@pytest.mark.parametrize("block", [0, 16, 64, 128])
@pytest.mark.parametrize("pad,ypad", [(48, 8), (1, 3)])
def test_grouped_strided(block, pad, ypad):
    _grouped(12, 2, 4, 200, 200, block, per_pair=True, weighted=True, pad=pad, ypad=ypad)


@pytest.mark.parametrize("M,topk,E,K,N,block", [(16, 8, 128, 2048, 1536, 16), (1000, 2, 8, 1024, 2048, 128),
                                                (700, 4, 16, 768, 1024, 64), (64, 4, 32, 2880, 2880, 32)])
def test_grouped_larger(M, topk, E, K, N, block):
    _grouped(M, topk, E, K, N, block, "skew", seed=1)


@pytest.mark.parametrize("block", [0, 16, 128])
@pytest.mark.parametrize("M,topk,E,K,N,kind", [(5, 1, 1, 8192, 100, "one"), (3, 2, 3, 8200, 400, "even"),
                                               (1, 1, 2, 8192, 4100, "even"), (2, 2, 4, 16384, 1030, "one")])
def test_grouped_few_items_of_a_long_k(block, M, topk, E, K, N, kind):
    """Clusters of 2, 4 and 8 CTAs that split K, with empty units beside the live ones."""
    _grouped(M, topk, E, K, N, block, kind, weighted=True)


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("M,topk,E,K,N,kind", [(400, 1, 2, 256, 300, "even"), (130, 2, 2, 130, 520, "even"),
                                               (513, 1, 1, 400, 257, "one"), (2000, 2, 8, 512, 256, "skew"),
                                               (700, 3, 16, 272, 128, "skew"), (3000, 4, 60, 128, 96, "even"),
                                               (400, 2, 2, 130, 777, "even"), (90, 1, 1, 64, 6000, "one")])
def test_grouped_many_pairs_an_expert(block, M, topk, E, K, N, kind):
    _grouped(M, topk, E, K, N, block, kind, per_pair=block > 32, weighted=block == 64, pad=block // 4)


def test_grouped_with_a_workspace():
    g = _gen(3)
    M, topk, E, K, N, block = 600, 2, 4, 256, 520, 64
    x, xs = f8_rows(M, K, g)
    w, ws = f8_weight(N, K, g, E)
    ids = _route(M, topk, E, g, "even")
    n = B.fp8_grouped_workspace_bytes(M, topk, E, K, N, block)
    assert n > 0
    space = torch.full((n + 64,), 0x7f, dtype=torch.uint8, device="cuda")
    y, want = (torch.empty((M, topk, N), dtype=BF, device="cuda") for _ in range(2))
    blocks = _align(ids, E, block)
    B.moe_fp8_grouped_matmul(x, xs, w, ws, y, *blocks, block, workspace=space[:n])
    B.moe_fp8_grouped_matmul(x, xs, w, ws, want, *blocks, block)
    assert torch.equal(y, want) and (space[n:] == 0x7f).all()
    with pytest.raises(B.MoeLoraError):
        B.moe_fp8_grouped_matmul(x, xs, w, ws, y, *blocks, block, workspace=space[:n - 1])


@pytest.mark.parametrize("block", [32, 64, 128])
def test_grouped_pair_after_sentinels_is_reported(block):
    """The units after a block's first that begin with the sentinel are skipped; a pair in one of them is reported."""
    g = _gen(block)
    M, topk, E, K, N = 20, 1, 4, 256, 128
    x, xs = f8_rows(M, K, g)
    w, ws = f8_weight(N, K, g, E)
    ids = (torch.arange(M, device="cuda") % E).to(torch.int32)[:, None].contiguous()
    s, e, n = _align(ids, E, block)
    y, err = torch.empty((M, topk, N), dtype=BF, device="cuda"), _err()
    B.moe_fp8_grouped_matmul(x, xs, w, ws, y, s, e, n, block, err_flag=err)
    ref, bound = _reference(x, xs, w, ws, ids, False, None)
    assert err.item() == 0
    assert_bf16_close(y.reshape(-1, N), ref, bound)
    s.reshape(-1)[block - 1] = 0          # the first block's last position
    B.moe_fp8_grouped_matmul(x, xs, w, ws, y, s, e, n, block, err_flag=err)
    assert err.item() == B.DEVERR_PAIR_ID
    assert_bf16_close(y.reshape(-1, N), ref, bound)


@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_grouped_no_tokens(block):
    g = _gen(0)
    w, ws = f8_weight(64, 64, g, 4)
    ids = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    y = torch.empty((0, 2, 64), dtype=BF, device="cuda")
    x, xs = torch.empty((0, 64), dtype=F8, device="cuda"), torch.empty((0, 1), device="cuda")
    cap = B.max_num_tokens_padded(0, 2, 4, block)
    s = torch.empty(cap, dtype=torch.int32, device="cuda")
    e = torch.empty(-(-cap // block), dtype=torch.int32, device="cuda")
    B.moe_fp8_grouped_matmul(x, xs, w, ws, y, s, e, _err(), block)
    B.moe_fp8_grouped_matmul_naive(x, xs, w, ws, y, ids)


@pytest.mark.parametrize("block", [0, 16, 64, 128])
def test_grouped_leaves_dropped_pairs(block):
    """Pairs whose expert is out of range: dropped by the align, skipped and reported by the naive assignment."""
    g = _gen(block)
    M, topk, E, K, N = 40, 2, 6, 256, 200
    x, xs = f8_rows(M, K, g)
    w, ws = f8_weight(N, K, g, E)
    ids = _route(M, topk, E, g, "even")
    ids[3, 1], ids[17, 0], ids[39, 1] = -1, E, 1 << 30
    y, err = torch.full((M, topk, N), 7.0, dtype=BF, device="cuda"), _err()
    if block:
        B.moe_fp8_grouped_matmul(x, xs, w, ws, y, *_align(ids, E, block), block, err_flag=err)
        assert err.item() == 0
    else:
        B.moe_fp8_grouped_matmul_naive(x, xs, w, ws, y, ids, err_flag=err)
        assert err.item() == B.DEVERR_EXPERT_ID
    gone = (ids < 0) | (ids >= E)
    assert (y[gone] == 7).all()
    ref, bound = _reference(x, xs, w, ws, ids, False, None)
    keep = ~gone.reshape(-1)
    assert_bf16_close(y.reshape(-1, N)[keep], ref[keep], bound[keep])


@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_grouped_bad_entries_are_skipped(block):
    """Entries of the sorted arrays that no align writes are reported and never dereferenced."""
    g = _gen(block)
    M, topk, E, K, N = 300, 1, 3, 256, 200
    x, xs = f8_rows(M, K, g)
    w, ws = f8_weight(N, K, g, E)
    ids = (torch.arange(M, device="cuda") % E).to(torch.int32)[:, None].contiguous()
    s, e, n = _align(ids, E, block)
    flat = s.reshape(-1)
    lost = [int(flat[0]), int(flat[5])]
    flat[0], flat[5] = -3, 1 << 29
    blocks = int(n) // block
    skipped = flat[(blocks - 1) * block:blocks * block].clone()
    e.reshape(-1)[blocks - 1] = E + 4
    y, err = torch.full((M, topk, N), 7.0, dtype=BF, device="cuda"), _err()
    B.moe_fp8_grouped_matmul(x, xs, w, ws, y, s, e, n, block, err_flag=err)
    assert err.item() == B.DEVERR_EXPERT_ID | B.DEVERR_PAIR_ID
    untouched = set(lost) | {int(v) for v in skipped if v < M * topk}
    ref, bound = _reference(x, xs, w, ws, ids, False, None)
    keep = torch.tensor([f not in untouched for f in range(M)], device="cuda")
    assert (y.reshape(-1, N)[~keep] == 7).all()
    assert_bf16_close(y.reshape(-1, N)[keep], ref[keep], bound[keep])


@pytest.mark.parametrize("block", [0, 16, 64, 128])
def test_grouped_nan_stays_in_its_row(block):
    g = _gen(block)
    M, topk, E, K, N = 30, 2, 4, 300, 150
    x, xs = f8_rows(M, K, g)
    w, ws = f8_weight(N, K, g, E)
    x.view(torch.uint8)[7] = 0x7f
    xs[11] = float("nan")
    ids = _route(M, topk, E, g, "even")
    y = torch.empty((M, topk, N), dtype=BF, device="cuda")
    if block:
        B.moe_fp8_grouped_matmul(x, xs, w, ws, y, *_align(ids, E, block), block)
    else:
        B.moe_fp8_grouped_matmul_naive(x, xs, w, ws, y, ids)
    bad = torch.isnan(y).all(-1).all(-1)
    assert bad[7] and bad[11] and bad.sum() == 2 and not torch.isnan(y[~bad]).any()


@pytest.mark.parametrize("M,block", [(1, 0), (16, 16), (200, 64), (600, 128)])
def test_grouped_same_bits_every_time_and_on_another_stream(M, block):
    g = _gen(M)
    topk, E, K, N = 8, 16, 2048, 256
    x, xs = f8_rows(M, K, g)
    w, ws = f8_weight(N, K, g, E)
    ids = _route(M, topk, E, g, "even")
    blocks = _align(ids, E, block) if block else None
    first = None
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for k in range(6):
        y = torch.empty((M, topk, N), dtype=BF, device="cuda")
        stream = side if k % 2 else None
        torch.cuda.synchronize()
        if block:
            B.moe_fp8_grouped_matmul(x, xs, w, ws, y, *blocks, block, stream=stream)
        else:
            B.moe_fp8_grouped_matmul_naive(x, xs, w, ws, y, ids, stream=stream)
        torch.cuda.synchronize()
        first = y if first is None else first
        assert torch.equal(first.view(torch.int16), y.view(torch.int16))


def test_grouped_in_a_cuda_graph():
    g = _gen(5)
    M, topk, E, K, N = 4, 2, 8, 512, 256
    x, xs = f8_rows(M, K, g)
    w, ws = f8_weight(N, K, g, E)
    ids = _route(M, topk, E, g, "even")
    y = torch.empty((M, topk, N), dtype=BF, device="cuda")
    B.moe_fp8_grouped_matmul_naive(x, xs, w, ws, y, ids)
    want = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_fp8_grouped_matmul_naive(x, xs, w, ws, y, ids)
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("M,N,ld", [(12, 200, 1 << 29), (40, 200, 1 << 27), (5200, 260, 1 << 20)])
def test_dense_offsets_past_32_bits(M, N, ld):
    """Rows of x and y far apart, the last past 2^32 bytes, on each kernel."""
    g = _gen(M)
    K = 272
    w, ws = f8_weight(N, K, g)
    small, xs = f8_rows(M, K, g)
    x = torch.empty(M * ld, dtype=torch.uint8, device="cuda").view(F8).view(M, ld)[:, :K]
    x.copy_(small)
    y = torch.empty(M * ld, dtype=BF, device="cuda").view(M, ld)[:, :N]
    B.moe_fp8_matmul(x, xs, w, ws, y)
    ref, bound = product64(small, xs, w, ws)
    assert_bf16_close(y, ref, bound)


def test_grouped_offsets_past_32_bits():
    """A weight of more than 2^32 elements and rows of x and y past 2^31 elements: the last expert and the last rows."""
    g = _gen(8)
    E, K, N = 136, 8192, 4096                    # 4.56e9 elements
    w = torch.zeros((E, N, K), dtype=torch.uint8, device="cuda").view(F8)
    ws = torch.full((E, N // 128, K // 128), 1e-3, device="cuda")
    v, _ = f8_rows(N, K, g)
    w.view(torch.uint8)[E - 1] = v.view(torch.uint8)
    M, ldy = 300, 1 << 23                        # y: 2.5e9 elements apart, first to last row
    x, xs = f8_rows(M, K, g)
    ids = torch.full((M, 1), E - 1, dtype=torch.int32, device="cuda")
    raw = torch.empty(M * ldy, dtype=BF, device="cuda")
    y = raw.view(M, 1, ldy)[:, :, :N]
    ref, bound = product64(x, xs, w[E - 1], ws[E - 1])
    for block in (64, 128):
        y.fill_(float("nan"))
        B.moe_fp8_grouped_matmul(x, xs, w, ws, y, *_align(ids, E, block), block)
        assert_bf16_close(y[:, 0], ref, bound, "block %d" % block)
    y[:16].fill_(float("nan"))
    B.moe_fp8_grouped_matmul_naive(x[:16], xs[:16], w, ws, y[:16], ids[:16].contiguous())
    assert_bf16_close(y[:16, 0], ref[:16], bound[:16], "naive")
