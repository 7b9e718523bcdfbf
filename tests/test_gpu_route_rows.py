"""The router with as many rows as an int holds."""
import pytest
import torch

from lora_moe_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("M", [(1 << 31) - 1, (1 << 31) - 4])
def test_the_most_rows(M):
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("26 GB of rows")
    logits = torch.zeros((M, 2), dtype=torch.bfloat16, device="cuda")
    logits[-1, 1] = 1
    logits[M // 2, 1] = 1
    ids = torch.full((M, 1), -7, dtype=torch.int32, device="cuda")
    weights = torch.full((M, 1), -7.0, device="cuda")
    B.moe_route(logits, ids, weights)
    assert ids[-1].item() == ids[M // 2].item() == 1 and ids.sum(dtype=torch.int64).item() == 2
    assert (weights == 1).all()
