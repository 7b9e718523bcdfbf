"""The tensor-core kernels of the 8-bit products leave nothing on its way when they exit: copies, stage hand-backs and
commits are waited for, in rings that end at every slot.  A wait for a phase that never comes would show as its limit of
4 seconds; an arrival in the shared memory of the next kernel's CTA as a wrong result there."""
import time

import pytest
import torch

from fp8_helpers import F8, groups
from lora_moe_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _whole(gen, *shape):
    return torch.randint(-2, 3, shape, generator=gen, device="cuda").to(F8)


def _run(calls, outputs, want):
    """Many calls back to back (each may start while the one before finishes), timed against the wait limit."""
    for f in calls:
        f()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(20):
        for f in calls:
            f()
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 2
    for y, w in zip(outputs, want):
        assert torch.equal(y, w)


# rows: the wide kernel on pairs of CTAs; 40 and 17 the narrow one; N of one and of several tiles
@pytest.mark.parametrize("M,N", [(5000, 260), (2000, 1500), (40, 700), (17, 130)])
def test_dense_rings(M, N):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(M)
    calls, outputs, want = [], [], []
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for kb in list(range(1, 15)) + [23, 24, 25]:
        x, w = _whole(gen, M, kb * 128), _whole(gen, N, kb * 128)
        y = torch.empty((M, N), dtype=BF, device="cuda")
        xs, ws = torch.ones((M, kb), device="cuda"), torch.ones((groups(N), kb), device="cuda")
        calls.append(lambda a=(x, xs, w, ws, y): B.moe_fp8_matmul(*a, err_flag=err))
        outputs.append(y)
        want.append((x.double() @ w.double().t()).to(BF))
    _run(calls, outputs, want)
    assert err.item() == 0


# (tokens, experts, block): the wide kernel, the narrow one with and without clusters, single pairs in clusters
@pytest.mark.parametrize("M,E,block", [(1500, 4, 128), (700, 8, 64), (60, 16, 16), (3, 4, 32), (1, 4, 0)])
def test_grouped_rings(M, E, block):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(M)
    calls, outputs, want = [], [], []
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    N = 300 if block else 1100
    # (single pairs: weights too large for the kernel that streams them through registers)
    for kb in range(1, 13) if block else (116, 117, 130, 133):
        x, w = _whole(gen, M, kb * 128), _whole(gen, E, N, kb * 128)
        y = torch.empty((M, 2, N), dtype=BF, device="cuda")
        xs, ws = torch.ones((M, kb), device="cuda"), torch.ones((E, groups(N), kb), device="cuda")
        ids = torch.argsort(torch.rand((M, E), generator=gen, device="cuda"), 1)[:, :2].to(torch.int32).contiguous()
        if block:
            buf = B.AlignBuffers(M, 2, E, 1, 1, block)

            def call(a=(x, xs, w, ws, y), ids=ids, buf=buf):
                B.moe_align_block_size(ids, E, block, buf.sorted_token_ids, buf.expert_ids, buf.num_tokens_post_padded,
                                       workspace=buf.workspace, err_flag=err)
                B.moe_fp8_grouped_matmul(*a, buf.sorted_token_ids, buf.expert_ids, buf.num_tokens_post_padded, block,
                                         err_flag=err)
        else:
            def call(a=(x, xs, w, ws, y), ids=ids):
                B.moe_fp8_grouped_matmul_naive(*a, ids, err_flag=err)
        calls.append(call)
        outputs.append(y)
        every = torch.einsum("mk,enk->men", x.double(), w.double()).to(BF)
        want.append(every.gather(1, ids.long()[:, :, None].expand(M, 2, N)))
    _run(calls, outputs, want)
    assert err.item() == 0
