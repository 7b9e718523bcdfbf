"""The example MoE layer (base experts in 8 bits, adapters in bf16) against the same layer in 64 bits."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer_fp8.py")
    spec = importlib.util.spec_from_file_location("moe_layer_fp8", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _layer64(layer, seen, lora):
    """The layer's rows for the example's own x, routing and activations: each stage's input is what the stage before it
    wrote, so that a bf16 or 8-bit rounding is made once on each side."""
    def weight(q, s):
        return q.double() * s.double().repeat_interleave(128, 1)[:, :q.shape[1]].repeat_interleave(128, 2)[:, :, :q.shape[2]]

    x, ids, act = seen["x"].double(), seen["ids"].long(), seen["act"].double()
    M, topk = ids.shape
    w13, w2 = weight(layer.w13, layer.s13), weight(layer.w2, layer.s2)
    gated = torch.zeros_like(act)
    rows = torch.zeros((M, topk, layer.H), dtype=torch.float64, device="cuda")
    for m in range(M):
        for k in range(topk):
            e, l, f = ids[m, k].item(), lora[m].item(), m * topk + k
            y = w13[e] @ x[m]
            z = w2[e] @ act[f]
            if l >= 0:
                for s in range(2):
                    y[s * layer.I:(s + 1) * layer.I] += layer.b13[s][l, e].double() @ (layer.a13[s][l, e].double() @ x[m])
                z = z + layer.b2[l, e].double() @ (layer.a2[l, e].double() @ act[f])
            gated[f] = torch.nn.functional.silu(y[:layer.I]) * y[layer.I:]
            rows[m, k] = z * seen["weights"][m, k].double()
    return gated, rows


@pytest.mark.parametrize("M,naive", [(1, None), (3, None), (8, False), (20, None), (20, True), (65, None)])
def test_layer(example, M, naive):
    layer = example.MoELayer(H=320, I=192, E=6, topk=2, max_loras=2, rank=8, seed=M)
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    rows = torch.randn((M, 3, layer.H), generator=g, device="cuda").to(BF)
    residual = torch.randn((M, layer.H), generator=g, device="cuda").to(BF)
    lora = (torch.arange(M, device="cuda") % 3 - 1).to(torch.int32)
    want = residual.double() + rows.double().sum(1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, seen = layer.step(rows, residual, lora, naive=naive, err=err)
    assert err.item() == 0
    assert ((residual.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5).all()
    n = want / torch.sqrt(want.square().mean(1, keepdim=True) + 1e-6) * layer.norm.double()
    assert ((seen["x"].double() - n).abs() <= 2.0 ** -8 * n.abs() + 1e-4).all()
    gated, ref = _layer64(layer, seen, lora)
    # An e4m3 rounding of an input is off by 2^-4 of it at most, uniformly over steps of up to 2^-3: 2^-3 / sqrt(12) =
    # 0.036 of it in the mean square at most.  Products of many such inputs are off by that share of their norm; the
    # activation multiplies two of them.
    assert (seen["act"].double() - gated).norm() <= 2 * 0.036 * gated.norm() * 1.1
    assert (y.double() - ref).norm() <= 0.036 * ref.norm() * 1.1


def test_layer_forms_agree(example):
    """The naive and the sorted forms of one batch differ by roundings of sums only."""
    layer = example.MoELayer(H=512, I=256, E=8, topk=2, max_loras=2, rank=16)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    rows = torch.randn((12, 1, layer.H), generator=g, device="cuda").to(BF)
    lora = (torch.arange(12, device="cuda") % 3 - 1).to(torch.int32)
    out = []
    for naive in (True, False):
        residual = torch.zeros((12, layer.H), dtype=BF, device="cuda")
        out.append(layer.step(rows, residual, lora, naive=naive)[0].double())
    assert (out[0] - out[1]).norm() <= 0.02 * out[0].norm()


def test_example_runs(example, capsys, monkeypatch):
    for argv in (["x", "5"], ["x", "40"]):
        monkeypatch.setattr("sys.argv", argv)
        example.main()
    assert "4 layers of 40 tokens" in capsys.readouterr().out
