"""The 8-bit outputs' scales and values where their quotients, amax / 448 and v / scale, lie on the rounding boundaries:
each quotient is a product with a reciprocal, within 2^-23 of its value (two roundings to fp32), so a value on a boundary
may take either of its neighbours and any other value has one answer.  On activations whose fp32 value is known exactly.

With a gate above 104, exp(-gate) is below the least fp32 value and silu(gate) is the gate itself; gate * up is then a
product of two numbers of at most 8 bits, exact in fp32."""
import pytest
import torch

from fp8_helpers import F8, TINY, groups, strided
from lora_moe_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _check(gate, up, pad=0):
    """gate, up: fp32 [rows, I] on the host, exact in bf16."""
    rows, I = gate.shape
    x = strided(rows, 2 * I, BF, pad)
    x.copy_(torch.cat((gate, up), 1))
    q, scales = strided(rows, I, F8, pad), torch.empty((rows, groups(I)), device="cuda")
    B.moe_silu_mul_fp8(x, q, scales)
    a = gate * up
    want_s = torch.stack([g.abs().amax(1).double() / 448 for g in a.split(128, 1)], 1).clamp_min(TINY)
    s = scales.cpu()
    assert ((s.double() - want_s).abs() <= 2.0 ** -23 * want_s).all()
    # the quotient by the scale that was returned; 2^-22: its own bound and the rounding of the two ends to fp32
    v = a.double() / s.double().repeat_interleave(128, 1)[:, :I]
    ends = [(v * (1 + d)).float().to(F8).view(torch.uint8) for d in (-2.0 ** -22, 2.0 ** -22)]
    got = q.contiguous().cpu().view(torch.uint8)
    assert ((got == ends[0]) | (got == ends[1])).all()
    assert not (ends[0] == ends[1]).all()     # (boundaries are among them)


def _grid(gates, copies=1):
    """A row for each gate c: a group with the largest value 448 c, so that its scale is c, and in it every value that 8
    bits hold and every one half way between two of them, times c."""
    steps = torch.tensor([k * 2.0 ** e for e in range(-14, 5) for k in range(16, 32)])     # 304 values up to 496
    steps = steps[steps <= 448]
    steps = torch.cat((torch.tensor([0.0, -0.0]), steps))
    body = torch.cat((steps, -steps))
    n = -(-body.numel() // 127)
    up = torch.zeros((n, 128))
    up[:, 0] = 448
    up[:, 1:] = torch.nn.functional.pad(body, (0, n * 127 - body.numel())).view(n, 127)
    up = up.reshape(1, -1)
    gate = torch.tensor(gates)[:, None].expand(len(gates), up.shape[1])
    return gate.repeat(copies, 1), up.expand(len(gates), -1).repeat(copies, 1)


@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("copies", [1, 130])     # 130: more than 38912 groups, the form of large calls
def test_quotients_at_the_rounding_boundaries(copies, pad):
    gate, up = _grid([float(c) for c in range(129, 256, 2)], copies)
    assert (up[:, ::128] == 448).all() and copies * 64 * groups(up.shape[1]) > (38912 if copies > 1 else 0)
    _check(gate, up, pad)


@pytest.mark.parametrize("exponent", [-132, -128, -120, -100, -60, 100, 111])
def test_quotients_of_small_and_large_groups(exponent):
    """Groups whose largest value is near the least scale's, subnormal, or near the largest fp32 value."""
    gate, up = _grid([129.0, 171.0, 233.0, 255.0])
    up = up.clone()
    ok = (up * 2.0 ** exponent).to(BF).float() == up * 2.0 ** exponent      # those that bf16 holds
    _check(gate, torch.where(ok, up * 2.0 ** exponent, torch.zeros(())))


def test_infinite_groups():
    """An infinity makes its group's scale infinite: finite values over it are zero, with their sign."""
    gate = torch.full((2, 256), 128.0)
    up = torch.linspace(-4, 4, 512).view(2, 256).to(BF).float()
    up[0, 7] = float("inf")
    up[1, 200] = float("-inf")
    x = torch.cat((gate, up), 1).to(BF).cuda()
    q, scales = torch.empty((2, 256), dtype=F8, device="cuda"), torch.empty((2, 2), device="cuda")
    B.moe_silu_mul_fp8(x, q, scales)
    s, v = scales.cpu(), q.cpu()
    assert s[0, 0] == float("inf") and s[1, 1] == float("inf") and torch.isfinite(s[0, 1]) and torch.isfinite(s[1, 0])
    for r, c in ((0, 7), (1, 200)):
        assert torch.isnan(v[r, c].float())
        group = slice(c // 128 * 128, c // 128 * 128 + 128)
        keep = torch.arange(group.start, group.stop) != c
        assert torch.equal(v[r, group].view(torch.uint8)[keep], torch.where(up[r, group] < 0, 0x80, 0).to(torch.uint8)[keep])
