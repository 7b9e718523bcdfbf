"""The activations of every bf16 number, in relation to their values: the tails of gelu and silu too, which are tiny beside
the number."""
import pytest
import torch

from bf16_helpers import ACTS, BF, F32, act64, assert_rounded, operand
from lora_moe_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _act64(v, act):
    """In 64 bits; gelu by erfc, as 1 + erf(v), which torch.special.ndtr takes, has lost the tail below v = -8."""
    return 0.5 * v * torch.special.erfc(-v * 0.5 ** 0.5) if act == "gelu" else act64(v, act)


def _numbers():
    """All finite bf16 numbers."""
    v = torch.arange(1 << 16, device="cuda").to(torch.int32).to(torch.int16).view(BF)
    return v[torch.isfinite(v)]


@pytest.mark.parametrize("act", [a for a in ACTS if a != "none"])
@pytest.mark.parametrize("rows", [1 << 16, 64, 16])      # by the wide kernel, the narrow one, and the one for few rows
def test_every_number(act, rows):
    v = _numbers()
    # every k-th number where the calls are many
    v = v[torch.arange(0, v.numel(), 1 if rows > 64 else 1023 // rows, device="cuda")]
    x, w, one = operand(v[:, None]), operand(torch.ones((1, 1), device="cuda")), torch.empty((v.numel(), 1), dtype=BF, device="cuda")
    for at in range(0, v.numel(), rows):
        B.moe_bf16_matmul(x[at:at + rows], w, one[at:at + rows], activation=ACTS[act])
    d = v.double()[:, None]
    ref = _act64(d, act)
    # the header's bound
    bound = torch.maximum(torch.where(d < -5, 2.0 ** -14, 2.0 ** -16) * ref.abs(), torch.full_like(ref, 2.0 ** -118))
    big = d.abs() > 2.0 ** 100      # (a cube past the largest fp32, and y its own limit or nothing)
    assert_rounded(one[~big][:, None], ref[~big][:, None], bound[~big][:, None], act)
    got = one[big].double()
    want = torch.where(d[big] > 0, d[big], torch.zeros_like(d[big]))
    assert torch.equal(got, want)


def test_fp32_tails():
    """CUDA's functions keep them: expf and erfcf, whose argument is rounded (x^2 up to 88, twice 2^-24 of it)."""
    v = _numbers()
    v = v[(v.double().abs() < 13)]
    y = torch.empty((v.numel(), 1), dtype=F32, device="cuda")
    for act in ("silu", "gelu", "gelu_tanh"):
        B.moe_bf16_matmul(operand(v[:, None]), operand(torch.ones((1, 1), device="cuda")), y, activation=ACTS[act])
        ref = _act64(v.double()[:, None], act)
        off = (y.double() - ref).abs()
        assert (off <= 2.0 ** -14 * ref.abs() + 2.0 ** -118).all(), act
