"""The direct calls (fastcall.so) of the bf16 products and of the router: they take ordinary calls and leave every other
one to the binding, with the same results."""
import pytest
import torch

from lora_moe_gb300 import binding as B

BF, I32 = torch.bfloat16, torch.int32


def _fast():
    f = B._load_fast()
    if f is B._NoFast:
        pytest.skip("fastcall.so is not built (no Python headers)")
    return f


def test_leaves_what_is_not_ordinary():
    f = _fast()
    x, w, y = torch.zeros((2, 64), dtype=BF), torch.zeros((8, 64), dtype=BF), torch.zeros((2, 8), dtype=BF)
    ids, weights = torch.zeros((2, 2), dtype=I32), torch.zeros((2, 2))
    assert f.matmul16(x, w, y, None, None, 0, None) is None              # host tensors
    assert f.matmul16(1, 2, 3, None, None, 0, None) is None              # no tensors
    assert f.matmul16(x, w, y, None, None, 1.5, None) is None            # the activation is no integer
    assert f.matmul16(x) is None                                         # too few
    assert f.route(torch.zeros((2, 8)), ids, weights, None, 0, True, 1.0, 1, 1, 1) is None
    assert f.route(torch.zeros((2, 8)), ids, weights, None, 0, True, 1, 1, 1, 1) is None     # the scale is no float
    assert f.route(torch.zeros((2, 8)), ids, weights, None, 1 << 70, True, 1.0, 1, 1, 1) is None
    assert f.route(None, None, None, None, 0, True, 1.0, 1, 1, 1) is None
    z = torch.zeros((2, 2, 8), dtype=BF)
    assert f.naive16(x, w[None], z, None, 0, None, False, None, ids) is None
    assert f.grouped16(x, w[None], z, None, 0, None, False, None, ids, ids, ids, 16) is None
    with pytest.raises(TypeError):
        f.bind16(1)
    with pytest.raises(ValueError):
        f.bind16(0, 0, 0, 0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [0, 8])
@pytest.mark.parametrize("f32", [False, True])
def test_same_results_as_through_ctypes(pad, f32):
    """A call that names its stream goes through ctypes: the same bits."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _fast()
    g = torch.Generator(device="cuda")
    g.manual_seed(pad)
    kind = torch.float32 if f32 else BF

    def rnd(*shape, dtype=BF):
        return torch.randn(shape[:-1] + (shape[-1] + pad,), generator=g, device="cuda").to(dtype)[..., :shape[-1]]

    M, topk, E, N, K = 5, 2, 16, 192, 256
    x, w = rnd(M, K), rnd(E, N, K)
    bias = torch.randn((E, N), generator=g, device="cuda").to(kind)
    residual, logits = rnd(M, N, dtype=kind), rnd(M, E, dtype=kind)
    select = torch.randn(E, generator=g, device="cuda")
    out = []
    for stream in (None, torch.cuda.current_stream()):
        def new(*shape, dtype=BF):
            return torch.zeros(shape[:-1] + (shape[-1] + pad,), dtype=dtype, device="cuda")[..., :shape[-1]]
        ids, weights = torch.zeros((M, topk), dtype=I32, device="cuda"), torch.zeros((M, topk), device="cuda")
        B.moe_route(logits, ids, weights, bias=select, scoring=B.ROUTE_SIGMOID, renormalize=False, scale=2.0, num_groups=4,
                    topk_groups=2, group_best=2, stream=stream)
        buf = B.AlignBuffers(M, topk, E, 1, 1, 16)
        B.moe_align_block_size(ids, E, 16, buf.sorted_token_ids, buf.expert_ids, buf.num_tokens_post_padded,
                               workspace=buf.workspace)
        y, z, d = new(M, topk, N), new(M, topk, N), new(M, N, dtype=kind)
        B.moe_bf16_grouped_matmul(x, w, y, buf.sorted_token_ids, buf.expert_ids, buf.num_tokens_post_padded, 16, bias=bias,
                                  activation=B.ACT_SILU, topk_weights=weights, stream=stream)
        B.moe_bf16_grouped_matmul_naive(x, w, z, ids, bias=bias, activation=B.ACT_GELU, topk_weights=weights, stream=stream)
        B.moe_bf16_matmul(x, w[1], d, bias=bias[1], residual=residual, activation=B.ACT_GELU_TANH, stream=stream)
        out.append([t.float() for t in (ids, weights, y, z, d)])
    for p, q in zip(*out):
        assert torch.equal(p, q) and p.abs().sum() > 0


@pytest.mark.gpu
def test_refusals_reach_the_caller():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _fast()
    x = torch.zeros((2, 132), dtype=BF, device="cuda")[:, :128]     # rows of 264 bytes: not on 16 bytes
    w, y = torch.zeros((8, 128), dtype=BF, device="cuda"), torch.zeros((2, 8), dtype=BF, device="cuda")
    with pytest.raises(B.MoeLoraError) as e:
        B.moe_bf16_matmul(x, w, y)
    assert e.value.status == 3
    with pytest.raises(ValueError):
        B.moe_bf16_matmul(w, w, y)
    with pytest.raises(TypeError):
        B.moe_bf16_matmul(w[:2], w, y, bias=torch.zeros(8, device="cuda", dtype=torch.float16))
    with pytest.raises(B.MoeLoraError) as e:
        B.moe_route(torch.zeros((2, 8), device="cuda"), torch.zeros((2, 2), dtype=I32, device="cuda"),
                    torch.zeros((2, 2), device="cuda"), num_groups=3)
    assert e.value.status == 1
