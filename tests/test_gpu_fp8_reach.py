"""Forms of the 8-bit kernels that only large or particular calls run, against the definitions in 64 bits: each case says
which form it is for, and asserts it where the sizes decide."""
import pytest
import torch

from fp8_helpers import F8, assert_bf16_close, assert_f8_close, f8_rows, f8_weight, groups, product64, quantize64, strided
from lora_moe_gb300 import binding as B
from test_gpu_fp8_matmul import _align, _err, _gen, _grouped, _reference, _route
from test_gpu_fp8_rows import ACT_REL, _check_norm

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("rows,I", [(5000, 1000), (39001, 128), (700, 14336), (13001, 300)])
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_act_of_many_groups(rows, I, pad):
    """Two groups a thread, from 38912 groups on (152 SMs x 8 CTAs x 32); 16 bytes at a time or scalar (pad 3)."""
    assert rows * groups(I) >= 38912
    x = strided(rows, 2 * I, BF, pad)
    x.copy_(4 * torch.randn((rows, 2 * I), generator=_gen(rows + I), device="cuda"))
    q, scales = strided(rows, I, F8, pad), torch.full((rows, groups(I)), float("nan"), device="cuda")
    act = strided(rows, I, BF, pad)
    B.moe_silu_mul_fp8(x, q, scales, act=act)
    gate, up = x[:, :I].double(), x[:, I:].double()
    v = gate / (1 + torch.exp(-gate)) * up
    assert_f8_close(q, scales, v, quantize64(v), ACT_REL, "act")
    assert_bf16_close(act, v, v.abs() * ACT_REL, "act")
    if pad:
        assert torch.isnan(q.as_strided((rows, I + pad), (I + pad, 1))[:, I:].float()).all()
        assert torch.isnan(act.as_strided((rows, I + pad), (I + pad, 1))[:, I:]).all()


@pytest.mark.parametrize("M,H,parts", [(305, 1024, 1), (700, 2880, 4), (333, 4096, 3), (1000, 1100, 2)])
@pytest.mark.parametrize("pad", [0, 3])
def test_norm_of_many_rows(M, H, parts, pad):
    """Two vectors a thread for rows of 1024 to 4096 columns, from 305 rows on (two for each SM)."""
    g = _gen(M + H)
    x = torch.empty((M, parts, H + pad), dtype=BF, device="cuda").fill_(float("nan"))[:, :, :H]
    x.copy_(torch.randn((M, parts, H), generator=g, device="cuda"))
    residual = strided(M, H, BF, pad)
    residual.copy_(3 * torch.randn((M, H), generator=g, device="cuda"))
    weight = (1 + 0.3 * torch.randn(H, generator=g, device="cuda")).to(BF)
    out, normed, q = strided(M, H, BF, pad), strided(M, H, BF, pad), strided(M, H, F8, pad)
    scales = torch.full((M, groups(H)), float("nan"), device="cuda")
    B.moe_add_rms_norm_fp8(x, weight, q, scales, residual=residual, residual_out=out, normed=normed, eps=1e-5)
    _check_norm(x, residual, weight, 1e-5, out, normed, q, scales)


@pytest.mark.parametrize("M,topk,E,K,N,block", [(600, 2, 300, 256, 200, 128), (800, 3, 600, 130, 130, 64),
                                                (900, 2, 300, 400, 96, 128)])
def test_narrow_without_a_list(M, topk, E, K, N, block):
    """More than 2048 units of 16 positions in blocks of more than 16: no list of the live ones is made."""
    assert B.fp8_grouped_workspace_bytes(M, topk, E, K, N, block) == 0
    g = _gen(M + E)
    x, xs = f8_rows(M, K, g)
    w, ws = f8_weight(N, K, g, E)
    ids = ((torch.arange(M * topk, device="cuda") * 7) % E).to(torch.int32).view(M, topk)
    s, e, n = _align(ids, E, block)
    assert int(n) // 16 > 2048
    y, err = torch.full((M, topk, N), float("nan"), dtype=BF, device="cuda"), _err()
    B.moe_fp8_grouped_matmul(x, xs, w, ws, y, s, e, n, block, err_flag=err)
    assert err.item() == 0
    ref, bound = _reference(x, xs, w, ws, ids, False, None)
    assert_bf16_close(y.reshape(M * topk, N), ref, bound)


@pytest.mark.parametrize("M,E,block", [(20, 8, 16), (40, 16, 64), (900, 4, 64), (600, 3, 128)])
@pytest.mark.parametrize("own_space", [False, True])
def test_sorted_forms_in_a_cuda_graph(M, E, block, own_space):
    """Narrow and wide, the align captured with them, with the caller's workspace and with torch's."""
    g = _gen(M)
    topk, K, N = 2, 400, 700
    x, xs = f8_rows(M, K, g)
    w, ws = f8_weight(N, K, g, E)
    ids = _route(M, topk, E, g, "even")
    y = torch.empty((M, topk, N), dtype=BF, device="cuda")
    n = B.fp8_grouped_workspace_bytes(M, topk, E, K, N, block)
    assert (n > 0) == (M > 100)
    space = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda") if own_space else None
    buf = B.AlignBuffers(M, topk, E, 1, 1, block)
    err = _err()

    def step():
        B.moe_align_block_size(ids, E, block, buf.sorted_token_ids, buf.expert_ids, buf.num_tokens_post_padded,
                               workspace=buf.workspace, err_flag=err)
        B.moe_fp8_grouped_matmul(x, xs, w, ws, y, buf.sorted_token_ids, buf.expert_ids, buf.num_tokens_post_padded, block,
                                 workspace=space, err_flag=err)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):        # other tokens and other experts under the same graph
        g = _gen(seed)
        x.copy_(f8_rows(M, K, g)[0])
        ids.copy_(_route(M, topk, E, g, "skew"))
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        ref, bound = _reference(x, xs, w, ws, ids, False, None)
        assert_bf16_close(y.reshape(M * topk, N), ref, bound)
    assert err.item() == 0


def test_wide_offsets_past_32_bits():
    """The wide kernel and its gather: a weight of more than 2^32 elements (the last expert), rows of x past 2^32 bytes
    and of y past 2^31 elements."""
    g = _gen(9)
    E, K, N, M, ldx, ldy, block = 136, 8192, 4096, 2800, 1 << 21, 1 << 20, 128
    assert B.fp8_grouped_workspace_bytes(M, 1, E, K, N, block) > 0
    w = torch.zeros((E, N, K), dtype=torch.uint8, device="cuda").view(F8)
    ws = torch.full((E, N // 128, K // 128), 1e-3, device="cuda")
    w.view(torch.uint8)[E - 1] = f8_rows(N, K, g)[0].view(torch.uint8)
    small, xs = f8_rows(M, K, g)
    x = torch.empty(M * ldx, dtype=torch.uint8, device="cuda").view(F8).view(M, ldx)[:, :K]
    x.copy_(small)
    ids = torch.full((M, 1), E - 1, dtype=torch.int32, device="cuda")
    y = torch.full((M * ldy,), float("nan"), dtype=BF, device="cuda").view(M, 1, ldy)[:, :, :N]
    err = _err()
    B.moe_fp8_grouped_matmul(x, xs, w, ws, y, *_align(ids, E, block), block, err_flag=err)
    assert err.item() == 0
    ref, bound = product64(small, xs, w[E - 1], ws[E - 1])
    assert_bf16_close(y[:, 0], ref, bound)
    assert torch.isnan(y.as_strided((M, 8), (ldy, 1), N).float()).all()     # nothing beside the rows


@pytest.mark.parametrize("block", [64, 128])
def test_wide_with_a_few_pairs_in_most_tiles(block):
    """Skewed routers: tiles of one to 256 rows, whose second CTA has none."""
    _grouped(1300, 2, 60, 256, 300, block, "skew", per_pair=True, weighted=True, seed=3)
