"""Refusals of the bf16 products and of the router, on the host (no GPU needed)."""
import ctypes

import pytest
import torch

from lora_moe_gb300 import binding as B

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4
_buf = ctypes.create_string_buffer(64)
P0 = (ctypes.addressof(_buf) + 15) & ~15      # host memory, never dereferenced


def _dense(**kw):
    a = dict(x=P0, ldx=256, w=P0, ldw=256, bias=None, bias_f32=0, res=None, ldr=0, y=P0, ldy=128, y_f32=0, act=0, M=2, N=128,
             K=256, err=None, stream=None)
    a.update(kw)
    return B.lib().moe_bf16_matmul(*a.values())


def _grouped(**kw):
    a = dict(x=P0, per_pair=0, ldx=256, w=P0, ldw=256, bias=None, bias_f32=0, y=P0, ldy=128, act=0, weights=None, sorted=P0,
             experts=P0, padded=P0, M=2, topk=2, E=8, K=256, N=128, block=16, cap=124, capb=8, ws_ptr=None, ws_bytes=0,
             err=None, stream=None)
    a.update(kw)
    return B.lib().moe_bf16_grouped_matmul(*a.values())


def _naive(**kw):
    a = dict(x=P0, per_pair=0, ldx=256, w=P0, ldw=256, bias=None, bias_f32=0, y=P0, ldy=128, act=0, weights=None, ids=P0, M=2,
             topk=2, E=8, K=256, N=128, err=None, stream=None)
    a.update(kw)
    return B.lib().moe_bf16_grouped_matmul_naive(*a.values())


def _route(**kw):
    a = dict(logits=P0, f32=1, ld=64, bias=None, scoring=0, renormalize=1, scale=1.0, groups=1, topk_groups=1, best=1, ids=P0,
             weights=P0, M=2, E=64, topk=4, stream=None)
    a.update(kw)
    return B.lib().moe_route(*a.values())


PRODUCT = [(INVALID, dict(M=-1)), (INVALID, dict(K=0)), (INVALID, dict(N=0)), (INVALID, dict(ldx=248)),
           (INVALID, dict(ldw=248)), (INVALID, dict(ldy=127)), (MISALIGNED, dict(ldx=260)), (MISALIGNED, dict(ldw=260)),
           (INVALID, dict(x=None)), (INVALID, dict(w=None)), (INVALID, dict(y=None)), (MISALIGNED, dict(x=P0 + 8)),
           (MISALIGNED, dict(w=P0 + 8)), (MISALIGNED, dict(y=P0 + 1)), (MISALIGNED, dict(bias=P0 + 1)),
           (MISALIGNED, dict(bias=P0 + 2, bias_f32=1)), (MISALIGNED, dict(err=P0 + 1)), (INVALID, dict(act=-1)),
           (INVALID, dict(act=5)), (UNSUPPORTED, dict(ldw=1 << 38)), (INVALID, dict(ldx=1 << 39)),
           (UNSUPPORTED, dict(K=(1 << 30) - 64, ldx=1 << 30, ldw=1 << 30)), (OK, dict(M=0)),
           (OK, dict(M=0, x=None, w=None, y=None))]


@pytest.mark.parametrize("call", [_dense, _naive, _grouped])
@pytest.mark.parametrize("want,kw", PRODUCT)
def test_products(call, want, kw):
    assert call(**kw) == want


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(res=P0, ldr=127)), (MISALIGNED, dict(res=P0 + 1, ldr=128)), (MISALIGNED, dict(y=P0 + 2, y_f32=1)),
    (MISALIGNED, dict(res=P0 + 2, ldr=128, y_f32=1)), (UNSUPPORTED, dict(M=(1 << 30) + 1)),
    (UNSUPPORTED, dict(M=1 << 29, N=1 << 22, ldy=1 << 22, ldw=256))])
def test_dense(want, kw):
    assert _dense(**kw) == want


@pytest.mark.parametrize("want,kw", [
    (UNSUPPORTED, dict(block=8)), (UNSUPPORTED, dict(block=256)), (INVALID, dict(cap=123)), (INVALID, dict(capb=7)),
    (INVALID, dict(sorted=None)), (INVALID, dict(experts=None)), (INVALID, dict(padded=None)),
    (MISALIGNED, dict(sorted=P0 + 2)), (WORKSPACE, dict(M=4096, cap=8192 + 8 * 15, capb=520, N=4096, ldy=4096)),
    (WORKSPACE, dict(M=4096, cap=8192 + 8 * 15, capb=520, N=4096, ldy=4096, ws_ptr=P0, ws_bytes=64)),
    (MISALIGNED, dict(M=4096, cap=8192 + 8 * 15, capb=520, N=4096, ldy=4096, ws_ptr=P0 + 8, ws_bytes=1 << 30))])
def test_grouped(want, kw):
    assert _grouped(**kw) == want


@pytest.mark.parametrize("call", [_grouped, _naive])
@pytest.mark.parametrize("want,kw", [
    (UNSUPPORTED, dict(E=1025, cap=1 << 20, capb=1 << 16)), (UNSUPPORTED, dict(topk=9, cap=1 << 20, capb=1 << 16)),
    (INVALID, dict(topk=0)), (INVALID, dict(E=0)), (MISALIGNED, dict(weights=P0 + 2)),
    (UNSUPPORTED, dict(M=1 << 30, cap=1 << 30, capb=1 << 30))])
def test_grouped_sizes(call, want, kw):
    if call is _naive:
        kw = {k: v for k, v in kw.items() if k not in ("cap", "capb")}
    assert call(**kw) == want


def test_naive_needs_ids():
    assert _naive(ids=None) == INVALID and _naive(ids=P0 + 2) == MISALIGNED


def test_grouped_workspace():
    need = B.bf16_grouped_workspace_bytes
    assert need(64, 2, 16, 256, 4096, 16) == 0                    # few pairs an expert: none
    n = need(8192, 2, 8, 4096, 128, 128)
    rows = (8192 * 2 + 8 * 127) // 128 * 128
    assert rows * 8192 < n < rows * 8192 * 1.1
    for bad in ((-1, 2, 8, 256, 128, 16), (4096, 9, 8, 256, 128, 16), (4096, 2, 0, 256, 128, 16), (4096, 2, 8, 0, 128, 16),
                (4096, 2, 8, 256, 0, 16), (4096, 2, 8, 256, 128, 24), (0, 2, 8, 256, 128, 16), (4096, 0, 8, 256, 128, 16)):
        assert need(*bad) == 0


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(M=-1)), (INVALID, dict(E=0)), (INVALID, dict(topk=0)), (INVALID, dict(scoring=2)),
    (INVALID, dict(scoring=-1)), (INVALID, dict(best=0)), (INVALID, dict(best=3)), (INVALID, dict(groups=0)),
    (INVALID, dict(topk_groups=0)), (INVALID, dict(groups=5)), (INVALID, dict(groups=4, topk_groups=5)),
    (INVALID, dict(topk=65, groups=1)), (INVALID, dict(groups=16, topk_groups=1, topk=5)), (INVALID, dict(ld=63)),
    (INVALID, dict(ld=1 << 39)), (UNSUPPORTED, dict(E=1025, ld=1025)), (UNSUPPORTED, dict(topk=33)),
    (UNSUPPORTED, dict(groups=64, topk_groups=64)), (INVALID, dict(logits=None)), (INVALID, dict(ids=None)),
    (INVALID, dict(weights=None)), (MISALIGNED, dict(logits=P0 + 2)), (MISALIGNED, dict(logits=P0 + 1, f32=0)),
    (MISALIGNED, dict(bias=P0 + 2)), (MISALIGNED, dict(ids=P0 + 2)), (MISALIGNED, dict(weights=P0 + 2)), (OK, dict(M=0)),
    (OK, dict(M=0, logits=None, ids=None, weights=None))])
def test_route(want, kw):
    if kw.get("topk") == 65:
        want = UNSUPPORTED      # (the limit is looked at first)
    assert _route(**kw) == want


# ------------------------------------------------------------------ the binding

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def test_binding_refuses_types_and_shapes():
    x, w, y = torch.zeros((2, 64), dtype=BF), torch.zeros((8, 64), dtype=BF), torch.zeros((2, 8), dtype=BF)
    with pytest.raises(ValueError):                       # host tensors
        B.moe_bf16_matmul(x, w, y)
    with pytest.raises(TypeError):
        B.moe_bf16_matmul(x, w, y.half())
    with pytest.raises(TypeError):
        B.moe_bf16_matmul(x.float(), w, y)
    with pytest.raises(ValueError):
        B.moe_bf16_matmul(x, w[:7], y)
    with pytest.raises(TypeError):
        B.moe_route(torch.zeros((2, 8), dtype=torch.float16), torch.zeros((2, 2), dtype=I32), torch.zeros((2, 2)))
    with pytest.raises(ValueError):
        B.moe_route(torch.zeros((2, 8)), torch.zeros((2, 2), dtype=I32), torch.zeros((2, 2)))
    ids = torch.zeros((2, 2), dtype=I32)
    with pytest.raises(ValueError):
        B.moe_bf16_grouped_matmul_naive(x, w[None], torch.zeros((2, 2, 8), dtype=BF), ids)


def test_constants_are_the_headers():
    import os
    import re
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe_lora.h")) as f:
        text = f.read()
    for name in ("ACT_NONE", "ACT_RELU", "ACT_SILU", "ACT_GELU", "ACT_GELU_TANH", "ROUTE_SOFTMAX", "ROUTE_SIGMOID"):
        assert int(re.search(r"#define MOE_%s (\d+)" % name, text).group(1)) == getattr(B, name)
