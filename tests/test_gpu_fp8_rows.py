"""The row operators of the 8-bit path against their definitions in 64 bits."""
import pytest
import torch

from fp8_helpers import F8, TINY, assert_bf16_close, assert_f8_close, groups, quantize64, strided
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


def _norm64(x, residual, weight, eps):
    h = x.double() if x.dim() == 2 else x.double().sum(1)
    mag = x.double().abs() if x.dim() == 2 else x.double().abs().sum(1)
    parts = 1 if x.dim() == 2 else x.shape[1]
    if residual is not None:
        h, mag = h + residual.double(), mag + residual.double().abs()
    r = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    return h, mag * (parts * 2.0 ** -24), h * r * weight.double(), r * weight.double().abs()


# fp32 sums of at most 16384 squares in trees of threads, then rsqrt and two products: 2^-24 times the longest chain
# (8 columns x 4 vectors + 5 + 16 levels), halved by the root, and 4 roundings
NORM_REL = 40 * 2.0 ** -24


def _check_norm(x, residual, weight, eps, out, normed, q, scales):
    h, hb, n, gain = _norm64(x, residual, weight, eps)
    if out is not None:
        assert_bf16_close(out, h, hb, "residual")
    # an error of h's own sum reaches n through the gain, and through the root mean square (at most as much again)
    nb = n.abs() * NORM_REL + gain * (hb + hb.amax(1, keepdim=True))
    if normed is not None:
        assert_bf16_close(normed, n, nb, "normed")
    rel = (nb.amax() / n.abs().amax()).item() + NORM_REL
    s64 = quantize64(n)
    s = scales.double()
    worst = torch.stack([nb[:, g * 128:(g + 1) * 128].amax(1) for g in range(groups(n.shape[1]))], 1) / 448
    assert ((s - s64).abs() <= worst + s64 * 2.0 ** -22).all(), "scales"
    se = s.repeat_interleave(128, 1)[:, :n.shape[1]]
    off = (q.double() * se - n).abs() - torch.maximum(n.abs() * 2.0 ** -4, se * 2.0 ** -10) * (1 + 1e-4) - 2 * nb - rel * n.abs()
    assert (off <= 0).all(), "q: %g over the bound" % off.max().item()


@pytest.mark.parametrize("M,H,parts", [(1, 1, 1), (3, 7, 1), (2, 128, 2), (5, 129, 1), (1, 2048, 8), (64, 2880, 4),
                                       (7, 1000, 3), (4, 4096, 2), (3, 4104, 1), (2, 8191, 1), (2, 8192, 5),
                                       (3, 16384, 2), (1, 16383, 1), (300, 256, 1)])
@pytest.mark.parametrize("pad", [0, 3, 16])
def test_norm(M, H, parts, pad):
    g = _gen(M * 7 + H + parts)
    x = torch.empty((M, parts, H + pad), dtype=BF, device="cuda").fill_(float("nan"))[:, :, :H]
    x.copy_(torch.randn((M, parts, H), generator=g, device="cuda"))
    residual = strided(M, H, BF, pad)
    residual.copy_(3 * torch.randn((M, H), generator=g, device="cuda"))
    weight = (1 + 0.3 * torch.randn(H, generator=g, device="cuda")).to(BF)
    out, normed, q = strided(M, H, BF, pad), strided(M, H, BF, pad), strided(M, H, F8, pad)
    scales = torch.full((M, groups(H)), float("nan"), device="cuda")
    B.moe_add_rms_norm_fp8(x, weight, q, scales, residual=residual, residual_out=out, normed=normed, eps=1e-5)
    _check_norm(x, residual, weight, 1e-5, out, normed, q, scales)
    if pad:   # nothing is written between the rows
        for t in (out, normed, q):
            raw = t.as_strided((M, H + pad), (H + pad, 1))[:, H:]
            assert torch.isnan(raw.float()).all()


@pytest.mark.parametrize("H", [96, 2880, 5000])
def test_norm_optional_operands(H):
    g = _gen(H)
    M = 5
    x = torch.randn((M, H), generator=g, device="cuda").to(BF)
    weight = torch.ones(H, dtype=BF, device="cuda")
    q, scales = torch.empty((M, H), dtype=F8, device="cuda"), torch.empty((M, groups(H)), device="cuda")
    B.moe_add_rms_norm_fp8(x, weight, q, scales)
    _check_norm(x, None, weight, 1e-6, None, None, q, scales)
    # the residual updated in place
    residual = torch.randn((M, H), generator=g, device="cuda").to(BF)
    before = residual.clone()
    B.moe_add_rms_norm_fp8(x, weight, q, scales, residual=residual, residual_out=residual)
    _check_norm(x, before, weight, 1e-6, residual, None, q, scales)


def test_norm_unaligned_pointers():
    g = _gen(3)
    M, H = 4, 640
    x, residual = strided(M, H, BF, 8, lead=1), strided(M, H, BF, 0, lead=3)
    x.copy_(torch.randn((M, H), generator=g, device="cuda"))
    residual.copy_(torch.randn((M, H), generator=g, device="cuda"))
    weight = torch.ones(H, dtype=BF, device="cuda")
    q, scales = strided(M, H, F8, 0, lead=5), torch.empty((M, groups(H)), device="cuda")
    B.moe_add_rms_norm_fp8(x, weight, q, scales, residual=residual)
    _check_norm(x, residual, weight, 1e-6, None, None, q, scales)


def test_norm_zero_nan_and_infinite_rows():
    M, H = 6, 384
    x = torch.randn((M, H), generator=_gen(1), device="cuda").to(BF)
    x[1] = 0
    x[2, 200] = float("nan")
    x[3, 0] = float("inf")
    x[4, 128:256] = 0
    weight = torch.ones(H, dtype=BF, device="cuda")
    q, scales = torch.empty((M, H), dtype=F8, device="cuda"), torch.empty((M, 3), device="cuda")
    normed = torch.empty((M, H), dtype=BF, device="cuda")
    B.moe_add_rms_norm_fp8(x, weight, q, scales, normed=normed, eps=1e-6)
    assert (q[1].float() == 0).all() and (scales[1] == TINY).all()
    assert torch.isnan(q[2].float()).all() and torch.isnan(scales[2]).all() and torch.isnan(normed[2]).all()
    # inf * 0 = NaN at the infinity, zero elsewhere
    assert torch.isnan(q[3, :128].float()).all() and torch.isnan(scales[3, 0])
    assert (q[3, 128:].float() == 0).all() and (normed[3, 1:] == 0).all()
    assert scales[4, 1] == TINY and (q[4, 128:256].float() == 0).all()
    keep = [0, 5]
    _check_norm(x[keep], None, weight, 1e-6, None, normed[keep], q.view(torch.uint8)[keep].view(F8), scales[keep])


def test_norm_zero_rows_and_zero_eps():
    weight = torch.ones(256, dtype=BF, device="cuda")
    B.moe_add_rms_norm_fp8(torch.empty((0, 256), dtype=BF, device="cuda"), weight,
                           torch.empty((0, 256), dtype=F8, device="cuda"), torch.empty((0, 2), device="cuda"))
    x = torch.full((1, 256), 2.0, dtype=BF, device="cuda")
    q, s = torch.empty((1, 256), dtype=F8, device="cuda"), torch.empty((1, 2), device="cuda")
    B.moe_add_rms_norm_fp8(x, weight, q, s, eps=0.0)
    assert torch.allclose(q.float() * s.repeat_interleave(128, 1), torch.ones(1, 256, device="cuda"), rtol=1e-6)


# exp with |argument| <= 89: CUDA's fast exponential is within 2 + |1.16 x| units of fp32 (its documented error), of
# which a gate below zero carries at most 1 + 89 * 1.16 units; a gate above zero e / (1 + e) of them.  Then a sum, a
# quotient (2 units) and a product.
ACT_REL = (2 + 1.16 * 89 + 4) * 2.0 ** -23


@pytest.mark.parametrize("rows,I", [(1, 1), (3, 7), (1, 128), (5, 129), (128, 768), (33, 1000), (3, 14336), (700, 192)])
@pytest.mark.parametrize("pad", [0, 3, 16])
def test_act(rows, I, pad):
    g = _gen(rows + I)
    x = strided(rows, 2 * I, BF, pad)
    x.copy_(4 * torch.randn((rows, 2 * I), generator=g, device="cuda"))
    q, scales = strided(rows, I, F8, pad), torch.full((rows, groups(I)), float("nan"), device="cuda")
    act = strided(rows, I, BF, pad) if rows != 33 else None
    B.moe_silu_mul_fp8(x, q, scales, act=act)
    gate, up = x[:, :I].double(), x[:, I:].double()
    v = gate / (1 + torch.exp(-gate)) * up
    assert_f8_close(q, scales, v, quantize64(v), ACT_REL, "act")
    if act is not None:
        assert_bf16_close(act, v, v.abs() * ACT_REL, "act")
    if pad:
        assert torch.isnan(q.as_strided((rows, I + pad), (I + pad, 1))[:, I:].float()).all()
        if act is not None:
            assert torch.isnan(act.as_strided((rows, I + pad), (I + pad, 1))[:, I:]).all()


def test_act_extremes():
    I = 256
    x = torch.zeros((5, 2 * I), dtype=BF, device="cuda")
    x[:, I:] = 1
    x[0, :I] = -300          # exp overflows: the activation is zero
    x[1, :I] = 300           # the gate itself
    x[2, 5] = float("nan")
    x[3, I + 200] = float("inf")
    x[3, 200] = 1
    x[4, :128] = 1e-38       # below the least scale
    q, s = torch.empty((5, I), dtype=F8, device="cuda"), torch.empty((5, 2), device="cuda")
    B.moe_silu_mul_fp8(x, q, s)
    assert (q[0].float() == 0).all() and (s[0] == TINY).all()
    assert torch.allclose(q[1].float() * s[1].repeat_interleave(128), torch.full((I,), 300.0, device="cuda"), rtol=1e-6)
    assert torch.isnan(q[2, :128].float()).all() and torch.isnan(s[2, 0]) and s[2, 1] == TINY
    assert torch.isinf(s[3, 1]) and torch.isnan(q[3, 200].float()) and (q[3, 128:200].float() == 0).all()
    assert (s[4] == TINY).all()


def test_act_three_dimensions_and_empty():
    x = torch.randn((4, 2, 512), generator=_gen(9), device="cuda").to(BF)
    q, s = torch.empty((8, 256), dtype=F8, device="cuda"), torch.empty((8, 2), device="cuda")
    B.moe_silu_mul_fp8(x, q, s)
    v = x.view(8, 512).double()
    v = v[:, :256] / (1 + torch.exp(-v[:, :256])) * v[:, 256:]
    assert_f8_close(q, s, v, quantize64(v), ACT_REL)
    B.moe_silu_mul_fp8(x[:0], q[:0], s[:0])


def test_rows_on_another_stream_and_twice_the_same():
    x = torch.randn((512, 4096), generator=_gen(2), device="cuda").to(BF)
    outs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        q, s = torch.empty((512, 2048), dtype=F8, device="cuda"), torch.empty((512, 16), device="cuda")
        n, r = torch.empty((512, 4096), dtype=F8, device="cuda"), torch.empty((512, 32), device="cuda")
        torch.cuda.synchronize()
        B.moe_silu_mul_fp8(x, q, s, stream=stream)
        B.moe_add_rms_norm_fp8(x, x[0], n, r, stream=stream)
        torch.cuda.synchronize()
        outs.append((q.view(torch.uint8), s, n.view(torch.uint8), r))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_rows_offsets_past_32_bits():
    """Rows 2^30 elements apart: the last one starts past 2^32."""
    M, H, ld = 6, 400, 1 << 30
    g = _gen(4)
    x = torch.empty(M * ld, dtype=BF, device="cuda").view(M, ld)[:, :2 * H]
    q8 = torch.empty(M * ld, dtype=torch.uint8, device="cuda").view(F8).view(M, ld)
    x.copy_(torch.randn((M, 2 * H), generator=g, device="cuda"))
    q, scales = q8[:, :H], torch.empty((M, groups(H)), device="cuda")
    weight = torch.ones(H, dtype=BF, device="cuda")
    B.moe_add_rms_norm_fp8(x[:, :H], weight, q, scales)
    _check_norm(x[:, :H], None, weight, 1e-6, None, None, q, scales)
    B.moe_silu_mul_fp8(x, q, scales)
    v = x[:, :H].double()
    v = v / (1 + torch.exp(-v)) * x[:, H:].double()
    assert_f8_close(q, scales, v, quantize64(v), ACT_REL)
