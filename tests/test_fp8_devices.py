"""The 8-bit operators' calls refuse tensors and streams that are not on the current device (tensors stood in for, on the
host: no GPU needed).  The library would launch on the current device, with another device's pointers."""
import pytest
import torch

from lora_moe_gb300 import binding as B

BF, F8, F32, I32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.int32


class Fake:
    """As much of a CUDA tensor as the binding looks at."""
    is_cuda = True

    def __init__(self, dtype, *shape, device=0):
        self.dtype, self.shape, self.index = dtype, torch.Size(shape), device
        self.device = torch.device("cuda", device)

    def get_device(self):
        return self.index

    def numel(self):
        return self.shape.numel()

    def stride(self, d=None):
        st = [1]
        for n in reversed(self.shape[1:]):
            st.insert(0, st[0] * n)
        return tuple(st) if d is None else st[d]

    def is_contiguous(self):
        return True

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return 1 << 12


class Library:
    """Records the calls that reach the library."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


M, H, N, K, E, TOPK = 4, 256, 128, 256, 8, 2
NORM = dict(x=(BF, M, H), weight=(BF, H), q=(F8, M, H), scales=(F32, M, 2), residual=(BF, M, H), residual_out=(BF, M, H),
            normed=(BF, M, H))
PARTS = dict(NORM, x=(BF, M, 3, H))
ACT = dict(x=(BF, M, 2 * H), q=(F8, M, H), scales=(F32, M, 2), act=(BF, M, H))
DENSE = dict(x=(F8, M, K), x_scales=(F32, M, 2), w=(F8, N, K), w_scales=(F32, 1, 2), y=(BF, M, N), err_flag=(I32, 1))
GROUPED = dict(x=(F8, M, K), x_scales=(F32, M, 2), w=(F8, E, N, K), w_scales=(F32, E, 1, 2), y=(BF, M, TOPK, N),
               topk_weights=(F32, M, TOPK), err_flag=(I32, 1))
SORTED = dict(GROUPED, sorted_token_ids=(I32, 128), expert_ids=(I32, 8), num_tokens_post_padded=(I32, 1),
              workspace=(torch.uint8, 64))
NAIVE = dict(GROUPED, topk_ids=(I32, M, TOPK))
CALLS = [("moe_add_rms_norm_fp8", NORM, {}), ("moe_add_rms_norm_fp8", PARTS, {}), ("moe_silu_mul_fp8", ACT, {}),
         ("moe_fp8_matmul", DENSE, {}), ("moe_fp8_grouped_matmul", SORTED, {"block_size": 16}),
         ("moe_fp8_grouped_matmul_naive", NAIVE, {})]


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
