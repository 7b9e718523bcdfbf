"""The calls of the bf16 products and of the router refuse tensors and streams that are not on the current device (tensors
stood in for, on the host: no GPU needed)."""
import pytest
import torch

from lora_moe_gb300 import binding as B
from test_fp8_devices import Fake, Library

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
M, N, K, E, TOPK = 4, 128, 256, 8, 2
DENSE = dict(x=(BF, M, K), w=(BF, N, K), y=(BF, M, N), bias=(BF, N), residual=(BF, M, N), err_flag=(I32, 1))
GROUPED = dict(x=(BF, M, K), w=(BF, E, N, K), y=(BF, M, TOPK, N), bias=(F32, E, N), topk_weights=(F32, M, TOPK),
               err_flag=(I32, 1))
SORTED = dict(GROUPED, sorted_token_ids=(I32, 128), expert_ids=(I32, 8), num_tokens_post_padded=(I32, 1),
              workspace=(torch.uint8, 64))
NAIVE = dict(GROUPED, topk_ids=(I32, M, TOPK))
ROUTE = dict(logits=(F32, M, E), topk_ids=(I32, M, TOPK), topk_weights=(F32, M, TOPK), bias=(F32, E))
CALLS = [("moe_bf16_matmul", DENSE, {}), ("moe_bf16_grouped_matmul", SORTED, {"block_size": 16}),
         ("moe_bf16_grouped_matmul_naive", NAIVE, {}), ("moe_route", ROUTE, {})]


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(B, "_lib", lib)
    monkeypatch.setattr(B, "_fast", B._NoFast)
    monkeypatch.setattr(B, "_raw_current_stream", lambda index: 77)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return lib


def _call(name, spec, more, elsewhere=(), stream=None):
    tensors = {k: Fake(*v, device=1 if k in elsewhere else 0) for k, v in spec.items()}
    getattr(B, name)(**tensors, **more, stream=stream)


@pytest.mark.parametrize("name,spec,more", CALLS)
def test_on_the_current_device(library, name, spec, more):
    _call(name, spec, more)
    assert library.calls[-1] == name


@pytest.mark.parametrize("name,spec,more", CALLS)
def test_every_tensor_elsewhere(library, name, spec, more):
    for key in spec:
        with pytest.raises(ValueError, match="current device"):
            _call(name, spec, more, (key,))
    with pytest.raises(ValueError, match="current device"):
        _call(name, spec, more, tuple(spec))     # all of them on one device, which is not the current one
    assert name not in library.calls


@pytest.mark.parametrize("name,spec,more", CALLS)
def test_a_stream_of_another_device(library, monkeypatch, name, spec, more):
    class Stream:
        def __init__(self, index):
            self.device, self.cuda_stream = torch.device("cuda", index), 88

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    _call(name, spec, more, stream=Stream(0))
    assert library.calls[-1] == name
    library.calls.clear()
    with pytest.raises(ValueError, match="current device"):
        _call(name, spec, more, stream=Stream(1))
    assert name not in library.calls
