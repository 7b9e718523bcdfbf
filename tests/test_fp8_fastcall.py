"""The direct calls of the 8-bit operators (fastcall.so): they take ordinary calls and leave every other one to the
binding, with the same results."""
import os

import pytest
import torch

from lora_moe_gb300 import binding as B
from lora_moe_gb300 import build

BF, F8 = torch.bfloat16, torch.float8_e4m3fn


def _fast():
    f = B._load_fast()
    if f is B._NoFast:
        pytest.skip("fastcall.so is not built (no Python headers)")
    return f


def test_built_where_the_headers_are():
    build.build()
    assert os.path.exists(build.FASTCALL) == build._has_python_headers()


def test_leaves_what_is_not_ordinary():
    f = _fast()
    h = torch.zeros((2, 128), dtype=BF)
    q, s = torch.zeros((2, 128), dtype=F8), torch.zeros((2, 1))
    assert f.norm(h, h[0], q, s, None, None, None, 1e-6) is None       # host tensors
    assert f.norm(h, h[0], q, s, None, None, None, 1) is None          # eps is no float
    assert f.norm(1, 2, 3, 4, None, None, None, 1e-6) is None          # no tensors
    assert f.norm(h) is None                                           # too few
    assert f.act(torch.zeros((2, 256), dtype=BF), q, s, None) is None
    assert f.act(None, None, None, None) is None
    assert f.matmul(q, s, q, s, h, None) is None
    w, y = torch.zeros((4, 8, 128), dtype=F8), torch.zeros((1, 2, 8), dtype=BF)
    ws, ids = torch.zeros((4, 1, 1)), torch.zeros((1, 2), dtype=torch.int32)
    assert f.naive(q[:1], s[:1], w, ws, y, None, False, None, ids) is None
    assert f.grouped(q[:1], s[:1], w, ws, y, None, False, None, ids, ids, ids, 16) is None
    with pytest.raises(TypeError):
        f.bind(1)
    with pytest.raises(ValueError):
        f.bind(0, 0, 0, 0, 0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [0, 16])
def test_same_results_as_through_ctypes(pad):
    """A call that names its stream goes through ctypes: the same bits."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _fast()
    g = torch.Generator(device="cuda")
    g.manual_seed(pad)

    def f8(*shape):
        raw = torch.randn(shape[:-1] + (shape[-1] + pad,), generator=g, device="cuda").to(F8)
        return raw[..., :shape[-1]]

    M, topk, E, N, K = 5, 2, 6, 192, 256
    x, w = f8(M, K), f8(E, N, K)
    xs, ws = torch.rand((M, 2), generator=g, device="cuda"), torch.rand((E, 2, 2), generator=g, device="cuda")
    ids = torch.randint(0, E, (M, topk), generator=g, device="cuda", dtype=torch.int32)
    weights = torch.rand((M, topk), generator=g, device="cuda")
    buf = B.AlignBuffers(M, topk, E, 1, 1, 16)
    B.moe_align_block_size(ids, E, 16, buf.sorted_token_ids, buf.expert_ids, buf.num_tokens_post_padded,
                           workspace=buf.workspace)
    h = torch.randn((M, 3, K + pad), generator=g, device="cuda").to(BF)[:, :, :K]
    gain = torch.randn(K, generator=g, device="cuda").to(BF)
    out = []
    for stream in (None, torch.cuda.current_stream()):
        def new(*shape, dtype=BF):
            return torch.zeros(shape[:-1] + (shape[-1] + pad,), dtype=dtype, device="cuda")[..., :shape[-1]]
        y, z, d = new(M, topk, N), new(M, topk, N), new(M, N)
        n8, ns, r, n = new(M, K, dtype=F8), torch.zeros((M, 2), device="cuda"), new(M, K), new(M, K)
        a8, as_, a = new(M, K // 2, dtype=F8), torch.zeros((M, 1), device="cuda"), new(M, K // 2)
        B.moe_fp8_grouped_matmul(x, xs, w, ws, y, buf.sorted_token_ids, buf.expert_ids, buf.num_tokens_post_padded, 16,
                                 topk_weights=weights, stream=stream)
        B.moe_fp8_grouped_matmul_naive(x, xs, w, ws, z, ids, topk_weights=weights, stream=stream)
        B.moe_fp8_matmul(x, xs, w[1], ws[1], d, stream=stream)
        B.moe_add_rms_norm_fp8(h, gain, n8, ns, residual=h[:, 0], residual_out=r, normed=n, stream=stream)
        B.moe_silu_mul_fp8(h[:, 1], a8, as_, act=a, stream=stream)
        out.append([t.float() for t in (y, z, d, n8, ns, r, n, a8, as_, a)])
    for p, q in zip(*out):
        assert torch.equal(p, q) and p.abs().sum() > 0


@pytest.mark.gpu
def test_refusals_reach_the_caller():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _fast()
    x = torch.zeros((2, 136), dtype=torch.uint8, device="cuda").view(F8)[:, :128]     # rows of 136: not on 16 bytes
    w, s = torch.zeros((8, 128), dtype=torch.uint8, device="cuda").view(F8), torch.zeros((2, 1), device="cuda")
    y = torch.zeros((2, 8), dtype=BF, device="cuda")
    with pytest.raises(B.MoeLoraError) as e:
        B.moe_fp8_matmul(x, s, w, s[:1], y)
    assert e.value.status == 3
    with pytest.raises(ValueError):
        B.moe_fp8_matmul(x, s, w, s, y)
    with pytest.raises(TypeError):
        B.moe_fp8_matmul(x, s.double(), w, s[:1], y)
