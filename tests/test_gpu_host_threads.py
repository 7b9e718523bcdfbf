"""Calls of different sizes from several host threads at once, each on its own stream: every call is launched and right.
(A launch limit that belongs to a kernel must not follow one call's size under another's launch.)"""
import concurrent.futures

import pytest
import torch

from fp8_helpers import F8, groups
from helpers import DeviceInputs
from lora_moe_gb300 import binding as B
from lora_moe_gb300 import inputs as gen

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
ROUNDS = 1500


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.lib()


def _in_threads(jobs):
    """Each job, a list of calls that take a stream, on a thread and a stream of its own, all at once.  (A call that
    names its stream goes through ctypes, which lets the other threads run.)"""
    torch.cuda.synchronize()

    def work(calls):
        stream = torch.cuda.Stream()
        torch.zeros(1, device="cuda")       # (the thread has a context)
        for _ in range(ROUNDS):
            for f in calls:
                f(stream)
        stream.synchronize()
    with concurrent.futures.ThreadPoolExecutor(len(jobs)) as ex:
        for f in [ex.submit(work, calls) for calls in jobs]:
            f.result()
    torch.cuda.synchronize()


@pytest.mark.parametrize("which", ["dense, narrow", "dense, wide", "dense, few rows", "norm", "align", "adapters, tensor cores", "adapters, streaming"])
def test_first_call_of_a_thread(which):
    """A thread whose first CUDA call this is: no context is current in it yet."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    M, N, K = {"dense, narrow": (40, 300, 256), "dense, wide": (5000, 300, 256)}.get(which, (4, 300, 256))
    x, w = (torch.randint(-2, 3, (n, K), generator=g, device="cuda").to(F8) for n in (M, N))
    xs, ws = torch.ones((M, 2), device="cuda"), torch.ones((3, 2), device="cuda")
    y, q = torch.zeros((M, N), dtype=BF, device="cuda"), torch.zeros((M, K), dtype=F8, device="cuda")
    rows, gain = torch.ones((M, K), dtype=BF, device="cuda"), torch.ones(K, dtype=BF, device="cuda")
    w_ = gen.Workload("thread", M=64, K=256, N=512, E=4, topk=2, max_loras=2, num_active_loras=2, rank=16,
                      block_size=32, mapping="uniform", experts="uniform")
    d = DeviceInputs(gen.make_inputs(w_))
    align = lambda s: B.moe_lora_align(  # noqa: E731
        d.topk_ids, d.mapping, d.lora_ids, w_.E, w_.max_loras, w_.block_size, d.buf.sorted_token_ids, d.buf.expert_ids,
        d.buf.num_tokens_post_padded, workspace=d.buf.workspace, stream=s)
    align(None)
    stream = torch.cuda.current_stream()
    torch.cuda.synchronize()

    def call():
        if which == "norm":
            B.moe_add_rms_norm_fp8(rows, gain, q, xs, stream=stream)
        elif which == "align":
            align(stream)
        elif which.startswith("adapters"):
            B.moe_lora_fused_shrink_expand(d.x, d.a, d.b, d.y_in, d.buf.sorted_token_ids, d.buf.expert_ids,
                                           d.buf.num_tokens_post_padded, d.lora_ids, w_.topk, w_.block_size,
                                           path=B.PATH_TCGEN05 if "tensor" in which else B.PATH_CUDA_CORE_STREAM,
                                           stream=stream)
        else:
            B.moe_fp8_matmul(x, xs, w, ws, y, stream=stream)
    call()       # (whatever is done once a process is done in this thread)
    torch.cuda.synchronize()
    y.zero_()
    torch.cuda.synchronize()
    with concurrent.futures.ThreadPoolExecutor(1) as ex:
        ex.submit(call).result()
    torch.cuda.synchronize()
    if which.startswith("dense"):
        assert torch.equal(y, (x.double() @ w.double().t()).to(BF))


def test_fp8_products():
    g = torch.Generator(device="cuda")
    g.manual_seed(0)

    def whole(*shape):
        return torch.randint(-2, 3, shape, generator=g, device="cuda").to(F8)

    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    jobs, checks = [], []
    # one kernel instance: rings of 4 stages (more items than SMs) and of 2, and clusters that split K
    for M, N, K in ((40, 20000, 256), (40, 300, 256), (50, 20100, 256), (64, 200, 250), (36, 19900, 130), (40, 128, 256),
                    (40, 4096, 4096), (33, 640, 6000)):
        x, w = whole(M, -(-K // 16) * 16)[:, :K], whole(N, -(-K // 16) * 16)[:, :K]
        xs, ws = torch.ones((M, groups(K)), device="cuda"), torch.ones((groups(N), groups(K)), device="cuda")
        y = torch.full((M, N), float("nan"), dtype=BF, device="cuda")
        jobs.append([lambda s, a=(x, xs, w, ws, y): B.moe_fp8_matmul(*a, err_flag=err, stream=s)])
        checks.append((y, (x.double() @ w.double().t()).to(BF)))
    _in_threads(jobs)
    assert err.item() == 0
    for y, want in checks:
        assert torch.equal(y, want)


# (M, K, N, E, rank): calls of one kernel instance whose shared memory differs
SHAPES = {B.PATH_CUDA_CORE_CLUSTER: ((96, 2048, 1536, 16, 64), (60, 4096, 4096, 6, 64), (40, 6144, 6144, 4, 64), (4, 256, 512, 8, 64)),
          B.PATH_TCGEN05: ((96, 2048, 1536, 16, 16), (60, 4096, 4096, 6, 128), (40, 2048, 2048, 4, 64), (4, 256, 512, 8, 32))}


@pytest.mark.parametrize("path", list(SHAPES))
def test_adapters(path):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    jobs, checks, sizes = [], [], set()
    for i, (M, K, N, E, rank) in enumerate(SHAPES[path]):
        w = gen.Workload("threads%d" % i, M=M, K=K, N=N, E=E, topk=2, max_loras=2, num_active_loras=2, rank=rank,
                         block_size=32, mapping="uniform", experts="uniform", seed=i)
        sizes.add(B.fused_plan(M, 2, E, K, N, rank, 2, 32, path=path)["smem_bytes"])
        d = DeviceInputs(gen.make_inputs(w))
        y = torch.zeros_like(d.y_in)
        B.moe_lora_align(d.topk_ids, d.mapping, d.lora_ids, w.E, w.max_loras, w.block_size, d.buf.sorted_token_ids,
                         d.buf.expert_ids, d.buf.num_tokens_post_padded, workspace=d.buf.workspace, err_flag=err)

        def fused(s, w=w, d=d, y=y):
            B.moe_lora_fused_shrink_expand(d.x, d.a, d.b, y, d.buf.sorted_token_ids, d.buf.expert_ids,
                                           d.buf.num_tokens_post_padded, d.lora_ids, w.topk, w.block_size,
                                           add_inputs=False, path=path, err_flag=err, stream=s)
        fused(None)
        checks.append((y, y.clone()))
        y.zero_()
        jobs.append([fused])
    assert len(sizes) > 1
    _in_threads(jobs)
    assert err.item() == 0
    for y, want in checks:
        assert torch.equal(y.view(torch.int16), want.view(torch.int16))


def test_align():
    """The shared-memory variant's counters: 32 warps of 400 to 1000 experts."""
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    jobs, checks = [], []
    for E in (400, 500, 700, 1000):
        M, topk = 2000, 2
        ids = torch.randint(0, E, (M, topk), device="cuda", dtype=torch.int32)
        buf = B.AlignBuffers(M, topk, E, 1, 1, 16, variant=B.ALIGN_SMEM)

        def align(s, E=E, ids=ids, buf=buf):
            B.moe_align_block_size(ids, E, 16, buf.sorted_token_ids, buf.expert_ids, buf.num_tokens_post_padded,
                                   workspace=buf.workspace, variant=B.ALIGN_SMEM, err_flag=err, stream=s)
        align(None)
        n = int(buf.num_tokens_post_padded.reshape(-1)[0])
        checks.append((buf, n, buf.sorted_token_ids.reshape(-1)[:n].clone()))
        buf.sorted_token_ids.fill_(-5)
        jobs.append([align])
    _in_threads(jobs)
    assert err.item() == 0
    for buf, n, want in checks:
        assert int(buf.num_tokens_post_padded.reshape(-1)[0]) == n
        assert torch.equal(buf.sorted_token_ids.reshape(-1)[:n], want)
