"""Refusals of the 8-bit operators, on the host (no GPU needed)."""
import ctypes

import pytest
import torch

from lora_moe_gb300 import binding as B

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
_buf = ctypes.create_string_buffer(64)
P0 = (ctypes.addressof(_buf) + 15) & ~15      # host memory, never dereferenced


def _norm(**kw):
    a = dict(x=P0, ldx=256, ld_part=0, parts=1, res=None, ldr=0, weight=P0, eps=1e-6, out=None, ldo=0, normed=None,
             ldn=0, q=P0, ldq=256, scales=P0, M=2, H=256, stream=None)
    a.update(kw)
    return B.lib().moe_add_rms_norm_fp8(*a.values())


def _act(**kw):
    a = dict(x=P0, ldx=512, act=None, lda=0, q=P0, ldq=256, scales=P0, rows=2, I=256, stream=None)
    a.update(kw)
    return B.lib().moe_silu_mul_fp8(*a.values())


def _dense(**kw):
    a = dict(x=P0, ldx=256, xs=P0, w=P0, ldw=256, ws=P0, y=P0, ldy=128, M=2, N=128, K=256, err=None, stream=None)
    a.update(kw)
    return B.lib().moe_fp8_matmul(*a.values())


def _grouped(**kw):
    a = dict(x=P0, per_pair=0, ldx=256, xs=P0, w=P0, ldw=256, ws=P0, y=P0, ldy=128, weights=None, sorted=P0, experts=P0,
             padded=P0, M=2, topk=2, E=8, K=256, N=128, block=16, cap=124, capb=8, ws_ptr=None, ws_bytes=0, err=None, stream=None)
    a.update(kw)
    return B.lib().moe_fp8_grouped_matmul(*a.values())


def _naive(**kw):
    a = dict(x=P0, per_pair=0, ldx=256, xs=P0, w=P0, ldw=256, ws=P0, y=P0, ldy=128, weights=None, ids=P0, M=2, topk=2,
             E=8, K=256, N=128, err=None, stream=None)
    a.update(kw)
    return B.lib().moe_fp8_grouped_matmul_naive(*a.values())


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(M=-1)), (INVALID, dict(H=0)), (INVALID, dict(parts=0)), (INVALID, dict(eps=-1.0)),
    (INVALID, dict(eps=float("nan"))), (UNSUPPORTED, dict(H=16385, ldx=20000, ldq=20000)), (INVALID, dict(ldx=255)),
    (INVALID, dict(parts=2, ld_part=255)), (INVALID, dict(ldq=100)), (INVALID, dict(res=P0, ldr=255)),
    (INVALID, dict(out=P0, ldo=0)), (INVALID, dict(normed=P0, ldn=-1)), (INVALID, dict(x=None)),
    (INVALID, dict(weight=None)), (INVALID, dict(q=None)), (INVALID, dict(scales=None)), (MISALIGNED, dict(x=P0 + 1)),
    (MISALIGNED, dict(scales=P0 + 2)), (MISALIGNED, dict(res=P0 + 1, ldr=256)), (OK, dict(M=0))])
def test_norm(want, kw):
    assert _norm(**kw) == want


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(rows=-1)), (INVALID, dict(I=0)), (INVALID, dict(ldx=511)), (INVALID, dict(ldq=255)),
    (INVALID, dict(x=None)), (INVALID, dict(q=None)), (INVALID, dict(scales=None)), (MISALIGNED, dict(x=P0 + 1)),
    (MISALIGNED, dict(scales=P0 + 1)), (INVALID, dict(act=P0, lda=255)), (MISALIGNED, dict(act=P0 + 1, lda=256)),
    (OK, dict(rows=0))])
def test_act(want, kw):
    assert _act(**kw) == want


PRODUCT = [(INVALID, dict(M=-1)), (INVALID, dict(K=0)), (INVALID, dict(N=0)), (INVALID, dict(ldx=240)),
           (INVALID, dict(ldw=240)), (INVALID, dict(ldy=127)), (MISALIGNED, dict(ldx=264)), (MISALIGNED, dict(ldw=264)),
           (INVALID, dict(x=None)), (INVALID, dict(xs=None)), (INVALID, dict(w=None)), (INVALID, dict(ws=None)),
           (INVALID, dict(y=None)), (MISALIGNED, dict(x=P0 + 8)), (MISALIGNED, dict(w=P0 + 8)),
           (MISALIGNED, dict(y=P0 + 1)), (MISALIGNED, dict(xs=P0 + 2)), (MISALIGNED, dict(ws=P0 + 2)),
           (MISALIGNED, dict(err=P0 + 1)), (UNSUPPORTED, dict(ldw=1 << 39)), (OK, dict(M=0))]


@pytest.mark.parametrize("call", [_dense, _naive])
@pytest.mark.parametrize("want,kw", PRODUCT)
def test_products(call, want, kw):
    assert call(**kw) == want


@pytest.mark.parametrize("want,kw", PRODUCT + [
    (UNSUPPORTED, dict(block=8)), (UNSUPPORTED, dict(block=256)), (INVALID, dict(cap=123)), (INVALID, dict(capb=7)),
    (INVALID, dict(sorted=None)), (INVALID, dict(experts=None)), (INVALID, dict(padded=None)),
    (MISALIGNED, dict(sorted=P0 + 2))])
def test_grouped(want, kw):
    assert _grouped(**kw) == want


@pytest.mark.parametrize("call", [_grouped, _naive])
@pytest.mark.parametrize("want,kw", [(UNSUPPORTED, dict(E=1025, cap=1 << 20, capb=1 << 16)), (UNSUPPORTED, dict(topk=9, cap=1 << 20, capb=1 << 16)),
                                     (INVALID, dict(topk=0)), (INVALID, dict(E=0)), (MISALIGNED, dict(weights=P0 + 2)),
                                     (UNSUPPORTED, dict(M=1 << 30, cap=1 << 30, capb=1 << 30))])
def test_grouped_sizes(call, want, kw):
    if call is _naive:
        kw = {k: v for k, v in kw.items() if k not in ("cap", "capb")}
    assert call(**kw) == want


def test_grouped_workspace():
    need = B.fp8_grouped_workspace_bytes
    assert need(64, 2, 16, 256, 4096, 16) == 0                    # few pairs an expert: none
    n = need(8192, 2, 8, 4096, 128, 128)
    rows = (8192 * 2 + 8 * 127) // 128 * 128
    assert rows * 4096 < n < rows * 4096 * 1.1
    assert need(4096, 2, 8, 256, 128, 64) > 0 and need(64, 2, 8, 256, 128, 64) == 0
    for bad in ((-1, 2, 8, 256, 128, 16), (4096, 9, 8, 256, 128, 16), (4096, 2, 8, 0, 128, 16), (4096, 2, 8, 256, 0, 16),
                (4096, 2, 8, 256, 128, 8)):
        assert need(*bad) == 0
    big = dict(M=8192, cap=1 << 20, capb=1 << 16, block=128, ldx=4096, ldw=4096, K=4096)
    assert _grouped(**big) == 4 and _grouped(ws_ptr=P0, ws_bytes=n - 1, **big) == 4
    assert _grouped(ws_ptr=P0 + 8, ws_bytes=n, **big) == MISALIGNED


def test_naive_ids():
    assert _naive(ids=None) == INVALID and _naive(ids=P0 + 2) == MISALIGNED


def test_binding_refuses_host_tensors_and_wrong_layouts():
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    x, w = torch.zeros((2, 256), dtype=bf), torch.zeros(256, dtype=bf)
    q, s = torch.zeros((2, 256), dtype=f8), torch.zeros((2, 2))
    with pytest.raises(ValueError, match="CUDA"):
        B.moe_add_rms_norm_fp8(x, w, q, s)
    with pytest.raises(TypeError):
        B.moe_add_rms_norm_fp8(x.float(), w, q, s)
    with pytest.raises(ValueError):
        B.moe_add_rms_norm_fp8(x, w[:255], q, s)
    with pytest.raises(ValueError, match="CUDA"):
        B.moe_silu_mul_fp8(torch.zeros((2, 512), dtype=bf), q, s)
    with pytest.raises(ValueError):
        B.moe_silu_mul_fp8(torch.zeros((3, 512), dtype=bf), q, s)
    y = torch.zeros((2, 128), dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        B.moe_fp8_matmul(q, s, torch.zeros((128, 256), dtype=f8), torch.zeros((1, 2)), y)
    with pytest.raises(ValueError, match="inconsistent"):
        B.moe_fp8_matmul(q, s, torch.zeros((128, 256), dtype=f8), torch.zeros((1, 2)), torch.zeros((3, 128), dtype=bf))
    with pytest.raises(TypeError):
        B.moe_fp8_matmul(x, s, torch.zeros((128, 256), dtype=f8), torch.zeros((1, 2)), y)


def test_rows_layout():
    """Leading dimensions as the binding reads them from strides (checked on CUDA tensors only, so faked here)."""
    class Fake:
        is_cuda, dtype = True, torch.bfloat16

        def __init__(self, shape, stride):
            self.shape, self._s = torch.Size(shape), stride

        def stride(self, d=None):
            return self._s if d is None else self._s[d]

        def data_ptr(self):
            return 64

        def numel(self):
            return self.shape.numel()

        def is_contiguous(self):
            return False

    def ld(shape, stride):
        rows = 1
        for n in shape[:-1]:
            rows *= n
        return B._rows(Fake(shape, stride), torch.bfloat16, "t", rows, shape[-1])[1]
    assert ld((4, 8), (8, 1)) == 8 and ld((4, 8), (24, 1)) == 24
    assert ld((1, 8), (1, 1)) == 16               # one row: any will do
    assert ld((3, 2, 8), (32, 16, 1)) == 16
    assert ld((3, 1, 8), (32, 8, 1)) == 32
    assert ld((1, 1, 24), (5, 3, 1)) == 32
    assert ld((3, 1, 1, 8), (32, 2, 7, 1)) == 32
    for shape, stride in (((4, 8), (8, 2)), ((3, 2, 8), (20, 8, 1)), ((1, 8), (8, 2))):
        with pytest.raises(ValueError):
            ld(shape, stride)
