"""Inputs and 64-bit definitions of the bf16 products, for their tests."""
import torch

from lora_moe_gb300 import binding as B

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
ACTS = {"none": B.ACT_NONE, "relu": B.ACT_RELU, "silu": B.ACT_SILU, "gelu": B.ACT_GELU, "gelu_tanh": B.ACT_GELU_TANH}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def err_flag():
    return torch.zeros(1, dtype=I32, device="cuda")


def strided(rows, columns, dtype, pad=0, lead=0):
    """A [rows, columns] view whose rows are columns + pad apart, `lead` elements into a buffer of NaN."""
    raw = torch.full((rows * (columns + pad) + lead,), float("nan"), dtype=dtype, device="cuda")
    return raw[lead:].view(rows, columns + pad)[:, :columns]


def operand(v, pad=0):
    """v in bf16; its rows start on 16 bytes, with NaN behind them."""
    rows, k = v.shape
    return strided(rows, k, BF, -(-(k + pad) // 8) * 8 - k).copy_(v)


def experts(v, pad=0):
    e, n, k = v.shape
    t = operand(v.reshape(e * n, k), pad)
    return t.as_strided((e, n, k), (n * t.stride(0), t.stride(0), 1))


def whole(g, *shape, most=2):
    """Whole numbers: their products, and sums of fewer than 2^24 / most^2 of them, are exact."""
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda").double()


def act64(v, name):
    if name == "relu":
        return v.clamp_min(0)
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return v * torch.special.ndtr(v)
    if name == "gelu_tanh":
        return v * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (v + 0.044715 * v ** 3))
    return v


def assert_rounded(got, ref, bound, what=""):
    """got: roundings (to its type) of values within `bound` of ref."""
    half = torch.finfo(got.dtype).eps / 2
    g = got.double()
    assert torch.isfinite(g).all(), what
    off = (g - ref).abs() - (bound + half * (ref.abs() + bound) + 2.0 ** -133)
    assert (off <= 0).all(), "%s: %g over the bound" % (what, off.max().item())


def align(ids, E, block):
    M, topk = ids.shape
    buf = B.AlignBuffers(M, topk, E, 1, 1, block)
    B.moe_align_block_size(ids, E, block, buf.sorted_token_ids, buf.expert_ids, buf.num_tokens_post_padded,
                           workspace=buf.workspace)
    return buf.sorted_token_ids, buf.expert_ids, buf.num_tokens_post_padded


def routes(M, topk, E, g, kind="even"):
    if kind == "one":                       # every token to the same experts
        ids = torch.arange(topk, device="cuda").expand(M, topk) % E
    else:
        p = torch.ones(E, device="cuda") if kind == "even" else 1.0 / torch.arange(1, E + 1, device="cuda") ** 1.5
        ids = torch.multinomial(p.expand(max(M, 1), E), topk, generator=g)[:M]
    return ids.to(I32).contiguous()


def grouped64(x, w, ids, per_pair, bias=None, act="none", weights=None):
    """[M * topk, N] in 64 bits, zeros for pairs whose expert does not exist; and the sums of magnitudes."""
    M, topk = ids.shape
    flat = ids.reshape(-1).long()
    y = torch.zeros((M * topk, w.shape[1]), dtype=torch.float64, device="cuda")
    size = torch.zeros_like(y)
    for e in flat.unique().tolist():
        if not 0 <= e < w.shape[0]:
            continue
        f = torch.nonzero(flat == e)[:, 0]
        rows = x[f if per_pair else f // topk].double()
        v = rows @ w[e].double().t()
        size[f] = rows.abs() @ w[e].double().abs().t()
        y[f] = act64(v if bias is None else v + bias[e].double(), act)
    if weights is not None:
        y, size = y * weights.reshape(-1, 1).double(), size * weights.reshape(-1, 1).double().abs()
    return y, size
