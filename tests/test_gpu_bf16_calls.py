"""How the bf16 products and the router are called: captured into graphs and replayed, on other streams, from several host
threads at once, back to back with rings that end at every slot, and with offsets past 32 bits."""
import concurrent.futures
import time

import pytest
import torch

from bf16_helpers import BF, F32, I32, align, err_flag, experts, gen, grouped64, operand, routes, whole
from lora_moe_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class Layer:
    """The router's projection, routing, align and an expert product of one MoE layer, on whole numbers."""

    def __init__(self, M, seed, E=8, topk=2, K=192, N=256, block=64):
        g = gen(seed)
        self.x, self.gate = operand(whole(g, M, K)), operand(whole(g, E, K))
        self.w = experts(whole(g, E, N, K))
        self.bias = whole(g, E, N, most=9).to(BF)
        self.logits = torch.empty((M, E), device="cuda")
        self.ids, self.weights = torch.empty((M, topk), dtype=I32, device="cuda"), torch.empty((M, topk), device="cuda")
        self.buf = B.AlignBuffers(M, topk, E, 1, 1, block)
        self.y = torch.empty((M, topk, N), dtype=BF, device="cuda")
        n = B.bf16_grouped_workspace_bytes(M, topk, E, K, N, block)
        self.space = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
        self.E, self.block, self.err = E, block, err_flag()

    def run(self, stream=None):
        B.moe_bf16_matmul(self.x, self.gate, self.logits, err_flag=self.err, stream=stream)
        B.moe_route(self.logits, self.ids, self.weights, stream=stream)
        B.moe_align_block_size(self.ids, self.E, self.block, self.buf.sorted_token_ids, self.buf.expert_ids,
                               self.buf.num_tokens_post_padded, workspace=self.buf.workspace, err_flag=self.err, stream=stream)
        B.moe_bf16_grouped_matmul(self.x, self.w, self.y, self.buf.sorted_token_ids, self.buf.expert_ids,
                                  self.buf.num_tokens_post_padded, self.block, bias=self.bias, workspace=self.space,
                                  err_flag=self.err, stream=stream)

    def check(self):
        logits = self.x.double() @ self.gate.double().t()
        assert torch.equal(self.logits.double(), logits) and self.err.item() == 0
        want = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :self.ids.shape[1]]
        assert torch.equal(self.ids.long(), want)
        p = torch.softmax(logits, 1).gather(1, want)
        p = p / p.sum(1, keepdim=True)
        # the header's bound of the weights
        assert ((self.weights.double() - p).abs() <= 2.0 ** -19 * p + 2.0 ** -140).all()
        y = grouped64(self.x, self.w, self.ids, False, self.bias)[0]
        assert torch.equal(self.y.view(-1, self.y.shape[2]), y.to(BF))


@pytest.mark.parametrize("M", [1, 40, 1500])
def test_layer(M):
    layer = Layer(M, M)
    layer.run()
    layer.check()


@pytest.mark.parametrize("M", [3, 1500])
def test_captured_and_replayed(M):
    """Two graphs that share a workspace, replayed in turn on inputs that change in between."""
    a, b = Layer(M, 1), Layer(M, 2)
    if b.space is not None:
        b.space = a.space
    side = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(side):
        for layer in (a, b):
            layer.run()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                layer.run()
            graphs.append(graph)
    for turn in range(3):
        for layer, graph in ((a, graphs[0]), (b, graphs[1])):
            g = gen(10 * turn + M)
            layer.x.copy_(whole(g, *layer.x.shape))
            layer.y.fill_(float("nan"))
            graph.replay()
        torch.cuda.synchronize()
        a.check()
        b.check()


@pytest.mark.parametrize("M", [3, 1500])
def test_on_another_stream(M):
    """A call that names its stream, while the current one is busy with something else."""
    layer, side = Layer(M, 5), torch.cuda.Stream()
    layer.space = None                     # (taken from torch's allocator, for that stream)
    torch.cuda.synchronize()
    busy = torch.randn((4096, 4096), device="cuda")
    for _ in range(5):
        busy = busy @ busy * 1e-2
        layer.run(side)
    side.synchronize()
    layer.check()


def test_from_several_threads():
    """Calls of different sizes at once, each on a stream of its own."""
    layers = [Layer(M, M, N=N, K=K) for M, N, K in ((1, 256, 192), (30, 700, 320), (100, 260, 64), (900, 520, 192),
                                                    (3000, 256, 128))]
    torch.cuda.synchronize()

    def work(layer):
        stream = torch.cuda.Stream()
        torch.zeros(1, device="cuda")       # (the thread has a context)
        for _ in range(200):
            layer.run(stream)
        stream.synchronize()
    with concurrent.futures.ThreadPoolExecutor(len(layers)) as ex:
        for f in [ex.submit(work, layer) for layer in layers]:
            f.result()
    torch.cuda.synchronize()
    for layer in layers:
        layer.check()


@pytest.mark.parametrize("which", ["few rows", "narrow", "wide", "wide, split", "route"])
def test_first_call_of_a_thread(which):
    """A thread whose first CUDA call this is: no context is current in it yet."""
    M, N = {"few rows": (4, 300), "narrow": (40, 300), "wide": (3000, 3000), "wide, split": (100, 300), "route": (40, 64)}[which]
    g = gen(1)
    x, w = operand(whole(g, M, 2048)), operand(whole(g, N, 2048))
    y = torch.zeros((M, N), dtype=BF, device="cuda")
    ids, weights = torch.zeros((M, 2), dtype=I32, device="cuda"), torch.zeros((M, 2), device="cuda")
    stream = torch.cuda.current_stream()

    def call():
        if which == "route":
            B.moe_route(x[:, :N], ids, weights, stream=stream)
        else:
            B.moe_bf16_matmul(x, w, y, stream=stream)
    call()       # (whatever is done once a process is done in this thread)
    torch.cuda.synchronize()
    y.zero_()
    ids.fill_(-1)
    torch.cuda.synchronize()
    with concurrent.futures.ThreadPoolExecutor(1) as ex:
        ex.submit(call).result()
    torch.cuda.synchronize()
    if which == "route":
        assert torch.equal(ids.long(), torch.sort(x[:, :N].double(), dim=1, descending=True, stable=True).indices[:, :2])
    else:
        assert torch.equal(y, (x.double() @ w.double().t()).to(BF))


# ------------------------------------------------------------------ exits

def _run(calls, outputs, want):
    """Many calls back to back (each may start while the one before finishes), timed against the limit of a wait."""
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


# rows and columns: the wide kernel on pairs of CTAs (all of K in one accumulator, in chunks), in clusters that split K,
# the narrow one, alone and in clusters
@pytest.mark.parametrize("M,N,dtype", [(5000, 2500, BF), (5000, 1500, F32), (300, 700, BF), (100, 300, F32), (40, 20000, BF),
                                       (40, 700, BF), (17, 130, F32)])
def test_dense_rings(M, N, dtype):
    g = gen(M)
    calls, outputs, want = [], [], []
    err = err_flag()
    for kb in list(range(1, 15)) + [23, 24, 25, 40, 61]:
        x, w = operand(whole(g, M, kb * 64)), operand(whole(g, N, kb * 64))
        y = torch.empty((M, N), dtype=dtype, device="cuda")
        calls.append(lambda a=(x, w, y): B.moe_bf16_matmul(*a, err_flag=err))
        outputs.append(y)
        want.append((x.double() @ w.double().t()).to(dtype))
    _run(calls, outputs, want)
    assert err.item() == 0


# (tokens, experts, block): the wide kernel with high and low tiles, the narrow one with and without clusters, single pairs
@pytest.mark.parametrize("M,E,block", [(1500, 4, 128), (700, 8, 64), (300, 16, 16), (60, 16, 16), (3, 4, 32), (1, 4, 0)])
def test_grouped_rings(M, E, block):
    g = gen(M)
    calls, outputs, want = [], [], []
    err = err_flag()
    N = 700
    for kb in list(range(1, 13)) + [31, 32, 33]:
        x, w = operand(whole(g, M, kb * 64)), experts(whole(g, E, N, kb * 64))
        y = torch.empty((M, 2, N), dtype=BF, device="cuda")
        ids = routes(M, 2, E, g)
        if block:
            buf = align(ids, E, block)
            calls.append(lambda a=(x, w, y, *buf): B.moe_bf16_grouped_matmul(*a, block, err_flag=err))
        else:
            calls.append(lambda a=(x, w, y, ids): B.moe_bf16_grouped_matmul_naive(*a, err_flag=err))
        outputs.append(y)
        want.append(grouped64(x, w, ids, False)[0].to(BF).view(M, 2, N))
    _run(calls, outputs, want)
    assert err.item() == 0


# ------------------------------------------------------------------ reach

@pytest.mark.parametrize("M", [3, 40, 100, 1000])
def test_offsets_past_32_bits(M):
    """Rows of x, w, y and the residual far apart."""
    g = gen(M)
    K, N = 128, 96
    far = (1 << 33) // M // 8 * 8          # elements between rows: M of them pass 2^32 elements

    def apart(rows, columns, dtype):
        raw = torch.empty((rows - 1) * far + columns, dtype=dtype, device="cuda")
        return raw.as_strided((rows, columns), (far, 1))
    x = apart(M, K, BF).copy_(whole(g, M, K))
    w = operand(whole(g, N, K))
    y = apart(M, N, BF)
    B.moe_bf16_matmul(x, w, y, residual=x[:, :N])
    want = x.double() @ w.double().t() + x[:, :N].double()
    assert torch.equal(y, want.to(BF))
    ids, weights = torch.empty((M, 4), dtype=I32, device="cuda"), torch.empty((M, 4), device="cuda")
    B.moe_route(x, ids, weights)
    assert torch.equal(ids.long(), torch.sort(x.double(), dim=1, descending=True, stable=True).indices[:, :4])


@pytest.mark.parametrize("M", [1, 16])
def test_weights_too_large_to_stream(M):
    g = gen(M)
    K, N = 8192, 17000
    x = operand(whole(g, M, K, most=1))
    w = torch.randint(-1, 2, (N, K), generator=g, device="cuda", dtype=torch.int8).to(BF)
    y = torch.empty((M, N), dtype=BF, device="cuda")
    B.moe_bf16_matmul(x, w, y)
    assert torch.equal(y, (x.double() @ w.double().t()).to(BF))


def test_single_pairs_too_many_to_stream():
    g = gen(7)
    M, topk, E, K, N = 16, 8, 8, 2048, 1030
    ids = routes(M, topk, E, g)
    x, w = operand(whole(g, M * topk, K)), experts(whole(g, E, N, K))
    y, err = torch.empty((M, topk, N), dtype=BF, device="cuda"), err_flag()
    B.moe_bf16_grouped_matmul_naive(x, w, y, ids, x_per_pair=True, err_flag=err)
    assert torch.equal(y.view(M * topk, N), grouped64(x, w, ids, True)[0].to(BF)) and err.item() == 0


@pytest.mark.parametrize("M,topk", [(4, 2), (40, 2), (300, 4)])
def test_adapters_behind_a_product(M, topk):
    """Slots' indexes and flags that are written just before a product, whose end the adapters' kernel starts beside."""
    g = gen(M)
    E, L, r, K, N, block = 8, 2, 8, 256, 256, 16
    x, w = operand(whole(g, M, K)), operand(whole(g, N, K))
    a, b = whole(g, L, E, r, K, most=1).to(BF), whole(g, L, E, N, r, most=1).to(BF)
    ids = routes(M, topk, E, g)
    lora = torch.arange(M, device="cuda", dtype=I32) % L
    slots = [torch.tensor(v, dtype=I32, device="cuda") for v in ([0, 1], [-1, 1], [0, -1], [0, 1])]
    flags = [torch.tensor(v, dtype=I32, device="cuda") for v in ([1, 1], [1, 1], [1, 1], [1, 0])]
    blocks = B.AlignBuffers(M, topk, E, L, L, block)
    now, on = slots[0].clone(), flags[0].clone()
    B.moe_lora_align(ids, lora, now, E, L, block, blocks.sorted_token_ids, blocks.expert_ids, blocks.num_tokens_post_padded,
                     workspace=blocks.workspace)
    base, err = torch.empty((M, N), dtype=BF, device="cuda"), err_flag()

    def call(i, y, apart):
        now.copy_(slots[i])
        on.copy_(flags[i])
        if apart:
            torch.cuda.synchronize()
        B.moe_bf16_matmul(x, w, base, err_flag=err)
        if apart:
            torch.cuda.synchronize()
        B.moe_lora_fused_shrink_expand_ex(x, a, b, y, blocks.sorted_token_ids, blocks.expert_ids,
                                          blocks.num_tokens_post_padded, now, topk, block, adapter_enabled=on, err_flag=err)
        if apart:
            torch.cuda.synchronize()
    want = [torch.zeros((M, topk, N), dtype=BF, device="cuda") for _ in slots]
    for i, y in enumerate(want):
        call(i, y, True)
    assert not torch.equal(want[0], want[1]) and not torch.equal(want[0], want[2]) and not torch.equal(want[0], want[3])
    got = [torch.zeros((M, topk, N), dtype=BF, device="cuda") for _ in range(80)]
    for i, y in enumerate(got):
        call(i * 7 // 4 % 4, y, False)
    for i, y in enumerate(got):
        assert torch.equal(y, want[i * 7 // 4 % 4])
    assert err.item() == 2      # MOE_LORA_DEVERR_LORA_ID: slots without an adapter are reported, and nothing else


@pytest.mark.parametrize("M,E,N,K,block", [(3, 4, 70, 100, 0), (3, 4, 70, 100, 16), (50, 6, 260, 200, 64), (900, 4, 300, 256, 128),
                                           (5, 1, 33, 64, 32)])
def test_the_same_expert_twice(M, E, N, K, block):
    """Pairs of one token that name one expert are pairs of their own."""
    g = gen(M + N)
    ids = torch.randint(0, E, (M, 1), generator=g, device="cuda").expand(M, min(E, 3)).to(I32).contiguous()
    x, w = operand(whole(g, ids.numel(), K)), experts(whole(g, E, N, K))
    y, err = torch.empty((*ids.shape, N), dtype=BF, device="cuda"), err_flag()
    if block:
        B.moe_bf16_grouped_matmul(x, w, y, *align(ids, E, block), block, x_per_pair=True, err_flag=err)
    else:
        B.moe_bf16_grouped_matmul_naive(x, w, y, ids, x_per_pair=True, err_flag=err)
    assert torch.equal(y.view(-1, N), grouped64(x, w, ids, True)[0].to(BF)) and err.item() == 0


@pytest.mark.parametrize("M,topk,block", [(1, 32, 0), (20, 32, 16), (700, 32, 64), (13000, 1, 128)])
def test_1024_experts(M, topk, block):
    g = gen(M)
    E, N, K = 1024, 136, 72
    ids = routes(M, topk, E, g, "skew" if M > 1000 else "even")
    x, w = operand(whole(g, M, K)), experts(whole(g, E, N, K))
    y, err = torch.empty((M, topk, N), dtype=BF, device="cuda"), err_flag()
    if block:
        B.moe_bf16_grouped_matmul(x, w, y, *align(ids, E, block), block, err_flag=err)
    else:
        B.moe_bf16_grouped_matmul_naive(x, w, y, ids, err_flag=err)
    assert torch.equal(y.view(-1, N), grouped64(x, w, ids, False)[0].to(BF)) and err.item() == 0


def test_two_graphs_share_a_workspace():
    """One after the other on a stream, in any order."""
    layers = [Layer(1500, 3), Layer(1400, 4)]
    space = max((a.space for a in layers), key=torch.Tensor.numel)
    graphs = []
    for a in layers:
        a.space = space
        a.run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            a.run()
        graphs.append(graph)
    for order in ((0, 1), (1, 0), (0, 0, 1, 1)):
        for a in layers:
            a.y.fill_(float("nan"))
        for i in order:
            graphs[i].replay()
        for a in layers:
            a.check()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_rows(dtype):
    """More rows than tiles of any grid, few columns."""
    g = gen(5)
    M, N, K = 700001, 24, 40
    x, w = operand(whole(g, M, K)), operand(whole(g, N, K))
    y, err = torch.empty((M, N), dtype=dtype, device="cuda"), err_flag()
    B.moe_bf16_matmul(x, w, y, err_flag=err)
    assert torch.equal(y, (x.double() @ w.double().t()).to(dtype)) and err.item() == 0
    ids, weights = torch.empty((M, 3), dtype=I32, device="cuda"), torch.empty((M, 3), device="cuda")
    B.moe_route(y, ids, weights)
    assert torch.equal(ids.long(), torch.sort(y.double(), dim=1, descending=True, stable=True).indices[:, :3])
    B.moe_route(y, ids, weights, num_groups=6, topk_groups=2, group_best=1)
    best = torch.sort(y.double().view(M, 6, 4).amax(2), dim=1, descending=True, stable=True).indices[:, :2]
    inside = torch.zeros((M, 6), dtype=torch.bool, device="cuda").scatter_(1, best, True).repeat_interleave(4, 1)
    masked = y.double().masked_fill(~inside, -float("inf"))
    assert torch.equal(ids.long(), torch.sort(masked, dim=1, descending=True, stable=True).indices[:, :3])
