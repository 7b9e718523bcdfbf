"""Timed cases of the 8-bit serving operators around the MoE adapters.

Four operators, in the order in which a decoder layer's MoE block calls them:

  norm     residual addition (with the sum over a token's top-k expert rows), root-mean-square norm, and the
           normalised row in bf16 and in 8 bits with one scale for each 128 columns;
  dense    8-bit matrix product with a scale for each 1 x 128 group of the input and each 128 x 128 block of the weight;
  grouped  the same product over the experts that the router chose for each (token, top-k) pair, on the blocks of the
           plain align ("sorted") or with one item per pair and no align ("naive");
  act      the gated activation silu(gate) * up between the experts' two products, in 8 bits with the same scales.

The plain forms are elementary torch operations in 32 bits.  Sizes are those of this repository's workloads
(Qwen3-, gpt-oss- and Mixtral-shaped decode and prefill, the large-E hidden size) or generic.
"""
import math

import torch

own = False

EPS = 1e-6
GROUP = 128
F8_MAX = 448.0
TINY = 2.0 ** -126      # the least scale
F8 = torch.float8_e4m3fn


def listed():
    return [
        # the norm before a decode step's next layer: one token, its eight expert rows summed (Qwen3-shaped)
        {"name": "norm 1x2048 of 8", "op": "norm", "M": 1, "H": 2048, "parts": 8},
        # a decode batch; 2880 columns end in half a group (gpt-oss-shaped)
        {"name": "norm 64x2880 of 4", "op": "norm", "M": 64, "H": 2880, "parts": 4},
        # prefill (Mixtral-shaped)
        {"name": "norm 8192x4096 of 2", "op": "norm", "M": 8192, "H": 4096, "parts": 2},
        # the activations of a decode batch of 16 tokens with 8 experts each (Qwen3-shaped)
        {"name": "act 128x768", "op": "act", "rows": 128, "I": 768},
        # prefill (Mixtral-shaped)
        {"name": "act 16384x14336", "op": "act", "rows": 16384, "I": 14336},
        # one token through a projection of the large-E hidden size: bound by the weight's bytes
        {"name": "dense 1x7168x4096", "op": "dense", "M": 1, "K": 7168, "N": 4096},
        # an odd decode batch; K and N end in half a block
        {"name": "dense 37x2880x2880", "op": "dense", "M": 37, "K": 2880, "N": 2880},
        # prefill through a square projection: bound by the tensor cores
        {"name": "dense 8192x4096x4096", "op": "dense", "M": 8192, "K": 4096, "N": 4096},
        # one token and its eight experts, no align (Qwen3-shaped gate and up projections)
        {"name": "naive 1 of 128x2048x1536", "op": "grouped", "mode": "naive", "M": 1, "topk": 8, "E": 128, "K": 2048,
         "N": 1536, "block": 16, "per_pair": False, "weights": False, "skew": 1.1},
        # a decode batch with a skewed router (Qwen3-shaped gate and up projections)
        {"name": "sorted 16 of 128x2048x1536", "op": "grouped", "mode": "sorted", "M": 16, "topk": 8, "E": 128,
         "K": 2048, "N": 1536, "block": 16, "per_pair": False, "weights": False, "skew": 1.1},
        # a decode batch's down projection: a row for each pair, times the router's weight (gpt-oss-shaped)
        {"name": "sorted 64 of 128x2880x2880", "op": "grouped", "mode": "sorted", "M": 64, "topk": 4, "E": 128,
         "K": 2880, "N": 2880, "block": 16, "per_pair": True, "weights": True, "skew": 0.0},
        # prefill (Mixtral-shaped gate and up projections): bound by the tensor cores
        {"name": "sorted 8192 of 8x4096x28672", "op": "grouped", "mode": "sorted", "M": 8192, "topk": 2, "E": 8,
         "K": 4096, "N": 28672, "block": 128, "per_pair": False, "weights": False, "skew": 0.0},
    ]


def draw(rng):
    def log(lo, hi, whole=0.0):
        """A size between lo and hi, even in its logarithm; with probability `whole` a multiple of 16."""
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        if rng.random() < whole:
            v = max(lo, v // 16 * 16)
        return v if v != 3 * 1024 else v + 16   # (no size of this repository's workloads)

    op = rng.choice(("norm", "act", "dense", "dense", "grouped", "grouped", "grouped"))
    if op == "norm":
        H, parts = log(64, 8192, 0.7), rng.choice((1, 2, 4, 8))
        return {"op": op, "M": min(log(1, 8192), 8192 * 4096 * 2 // (H * parts)), "H": H, "parts": parts}
    if op == "act":
        return {"op": op, "rows": log(1, 16384), "I": log(64, 14336, 0.7)}
    K, N = log(128, 8192, 0.8), log(64, 8192, 0.8)
    if op == "dense":
        return {"op": op, "M": log(1, 8192), "K": K, "N": N}
    mode = rng.choice(("naive", "sorted", "sorted"))
    E, topk = rng.choice((8, 16, 60, 128, 256)), rng.choice((1, 2, 4, 8))
    M = log(1, 16) if mode == "naive" else log(1, 8192)
    # no more weight, and no more work with every expert's rows padded to M, than the largest listed case
    E = max(8, min(E, 8 * 4096 * 28672 // (K * N)))
    M = max(1, min(M, 4 * 8 * 2048 * 4096 * 28672 // (E * K * N), 16384 // topk))
    return {"op": op, "mode": mode, "M": M, "topk": topk, "E": E, "K": K, "N": N,
            "block": 16 if mode == "naive" else rng.choice((16, 32, 64, 128)), "per_pair": rng.random() < 0.5,
            "weights": rng.random() < 0.5, "skew": rng.choice((0.0, 1.1))}


# ------------------------------------------------------------------ inputs

def _groups(n):
    return -(-n // GROUP)


def _padded(t, *sizes):
    """t with zeros up to `sizes` in its last dimensions."""
    pad = []
    for have, want in zip(reversed(t.shape), reversed(sizes)):
        pad += [0, want - have]
    return torch.nn.functional.pad(t, pad)


def _quantize_rows(v):
    """8-bit rows, padded to whole 16 bytes, and their [rows, groups] scales."""
    rows, k = v.shape
    g = _groups(k)
    b = _padded(v, g * GROUP).view(rows, g, GROUP)
    s = (b.abs().amax(-1) / F8_MAX).clamp_min(TINY)
    q = (b / s[..., None]).to(F8).view(torch.uint8).view(rows, g * GROUP)
    ld = -(-k // 16) * 16
    return q[:, :ld].contiguous().view(F8)[:, :k], s


def _quantize_weight(v):
    """8-bit [N, ld] rows of one expert, padded to whole 16 bytes, and their [N / 128, K / 128] scales."""
    n, k = v.shape
    gn, gk = _groups(n), _groups(k)
    b = _padded(v, gn * GROUP, gk * GROUP).view(gn, GROUP, gk, GROUP)
    s = (b.abs().amax((1, 3)) / F8_MAX).clamp_min(TINY)
    q = (b / s[:, None, :, None]).to(F8).view(torch.uint8).view(gn * GROUP, gk * GROUP)
    return q[:n, :-(-k // 16) * 16].contiguous().view(F8), s


def _weights(count, n, k, gen):
    """Random experts of unit gain, whose rows differ in size (as a trained weight's do)."""
    q = torch.empty((count, n, -(-k // 16) * 16), dtype=F8, device="cuda")
    s = torch.empty((count, _groups(n), _groups(k)), dtype=torch.float32, device="cuda")
    for e in range(count):
        v = torch.randn((n, k), generator=gen, device="cuda") / math.sqrt(k)
        v *= torch.exp(0.3 * torch.randn((n, 1), generator=gen, device="cuda"))
        q[e], s[e] = _quantize_weight(v)
    return q[:, :, :k], s


def _activations(rows, k, gen):
    """Normal rows with a few large channels."""
    v = torch.randn((rows, k), generator=gen, device="cuda")
    return v * torch.exp(0.5 * torch.randn((1, k), generator=gen, device="cuda"))


def _routing(c, gen):
    """Distinct experts for each token, uniform or with a Zipf-like skew, and router weights that sum to one."""
    M, E, topk = c["M"], c["E"], c["topk"]
    p = torch.arange(1, E + 1, dtype=torch.float32, device="cuda") ** -c["skew"]
    p = p[torch.randperm(E, generator=gen, device="cuda")]
    ids = torch.multinomial(p.expand(M, E), topk, generator=gen).to(torch.int32)
    w = torch.softmax(torch.randn((M, topk), generator=gen, device="cuda"), -1)
    return ids, w


def _align(ids, E, block):
    """The blocks of the plain align: pairs by expert in ascending order, each expert padded to whole blocks with the
    sentinel (the number of pairs)."""
    flat = ids.reshape(-1).long()
    P = flat.numel()
    counts = torch.bincount(flat, minlength=E)
    blocks = (counts + block - 1) // block
    first = torch.cumsum(blocks, 0) - blocks
    order = torch.argsort(flat, stable=True)
    rank = torch.arange(P, device="cuda") - (torch.cumsum(counts, 0) - counts)[flat[order]]
    cap = P + E * (block - 1)
    sorted_ids = torch.full((cap,), P, dtype=torch.int32, device="cuda")
    sorted_ids[first[flat[order]] * block + rank] = order.to(torch.int32)
    expert_ids = torch.zeros(-(-cap // block), dtype=torch.int32, device="cuda")
    n = int(blocks.sum())
    expert_ids[:n] = torch.repeat_interleave(torch.arange(E, device="cuda"), blocks).to(torch.int32)
    return sorted_ids, expert_ids, (blocks.sum() * block).to(torch.int32).reshape(1), int(counts.max())


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    bf = torch.bfloat16
    s = {"case": c}
    if c["op"] == "norm":
        M, H, parts = c["M"], c["H"], c["parts"]
        s["x"] = (torch.randn((M, parts, H), generator=gen, device="cuda") / math.sqrt(parts)).to(bf)
        s["residual"] = (4 * _activations(M, H, gen)).to(bf)
        s["weight"] = (1 + 0.2 * torch.randn(H, generator=gen, device="cuda")).to(bf)
        s["residual_out"], s["normed"] = torch.empty((M, H), dtype=bf, device="cuda"), torch.empty((M, H), dtype=bf, device="cuda")
        s["q"] = torch.empty((M, -(-H // 16) * 16), dtype=F8, device="cuda")[:, :H]
        s["scales"] = torch.empty((M, _groups(H)), dtype=torch.float32, device="cuda")
    elif c["op"] == "act":
        rows, I = c["rows"], c["I"]
        s["x"] = torch.empty((rows, 2 * I), dtype=bf, device="cuda")
        for r in range(0, rows, 4096):
            s["x"][r:r + 4096] = (1.5 * torch.randn((min(4096, rows - r), 2 * I), generator=gen, device="cuda")).to(bf)
        s["q"] = torch.empty((rows, -(-I // 16) * 16), dtype=F8, device="cuda")[:, :I]
        s["scales"] = torch.empty((rows, _groups(I)), dtype=torch.float32, device="cuda")
    else:
        M, K, N = c["M"], c["K"], c["N"]
        grouped = c["op"] == "grouped"
        rows = M * c["topk"] if grouped and c["per_pair"] else M
        s["x"], s["x_scales"] = _quantize_rows(_activations(rows, K, gen))
        w, ws = _weights(c["E"] if grouped else 1, N, K, gen)
        s["w"], s["w_scales"] = (w, ws) if grouped else (w[0], ws[0])
        s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if grouped:
            s["ids"], weights = _routing(c, gen)
            s["weights"] = weights if c["weights"] else None
            s["sorted"], s["experts"], s["padded"], s["most"] = _align(s["ids"], c["E"], c["block"])
            s["y"] = torch.empty((M, c["topk"], N), dtype=bf, device="cuda")
        else:
            s["y"] = torch.empty((M, N), dtype=bf, device="cuda")
    return s


# ------------------------------------------------------------------ the plain forms, in 32 bits

def _plain_quantize(v):
    rows, n = v.shape
    g = _groups(n)
    b = _padded(v, g * GROUP).view(rows, g, GROUP)
    s = (b.abs().amax(-1) / F8_MAX).clamp_min(TINY)
    return (b / s[..., None]).view(rows, g * GROUP)[:, :n].to(F8), s


def _plain_rows(q, s):
    return q.float() * s.repeat_interleave(GROUP, -1)[:, :q.shape[1]]


def _plain_weight(q, s):
    return q.float() * s.repeat_interleave(GROUP, -2)[..., :q.shape[-2], :].repeat_interleave(GROUP, -1)[..., :q.shape[-1]]


def _plain(s):
    c = s["case"]
    if c["op"] == "norm":
        h = s["residual"].float() + s["x"].float().sum(1)
        n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"].float()
        q, scales = _plain_quantize(n)
        return {"residual": h.to(torch.bfloat16), "normed": n.to(torch.bfloat16), "q": q, "scales": scales}
    if c["op"] == "act":
        gate, up = s["x"][:, :c["I"]].float(), s["x"][:, c["I"]:].float()
        q, scales = _plain_quantize(gate / (1 + torch.exp(-gate)) * up)
        return {"q": q, "scales": scales}
    x = _plain_rows(s["x"], s["x_scales"])
    if c["op"] == "dense":
        return (x @ _plain_weight(s["w"], s["w_scales"]).t()).to(torch.bfloat16)
    flat = s["ids"].reshape(-1).long()
    x = x if c["per_pair"] else x.repeat_interleave(c["topk"], 0)
    if flat.numel() < c["E"]:
        # few pairs: each with its expert's weight
        y = torch.bmm(_plain_weight(s["w"][flat], s["w_scales"][flat]), x[:, :, None])[:, :, 0]
    else:
        # every expert's rows side by side, padded to the most that one expert has: one batched product
        rank = torch.nn.functional.one_hot(flat, c["E"]).cumsum(0).gather(1, flat[:, None])[:, 0] - 1
        rows = torch.zeros((c["E"], s["most"], c["K"]), device="cuda")
        rows[flat, rank] = x
        y = torch.bmm(rows, _plain_weight(s["w"], s["w_scales"]).transpose(1, 2))[flat, rank]
    if s["weights"] is not None:
        y = y * s["weights"].reshape(-1, 1)
    return y.to(torch.bfloat16).view(c["M"], c["topk"], c["N"])


def run(state):
    if not own:
        return _plain(state)
    from lora_moe_gb300 import binding as B
    s, c = state, state["case"]
    if c["op"] == "norm":
        B.moe_add_rms_norm_fp8(s["x"], s["weight"], s["q"], s["scales"], residual=s["residual"],
                               residual_out=s["residual_out"], normed=s["normed"], eps=EPS)
        return {"residual": s["residual_out"], "normed": s["normed"], "q": s["q"], "scales": s["scales"]}
    if c["op"] == "act":
        B.moe_silu_mul_fp8(s["x"], s["q"], s["scales"])
        return {"q": s["q"], "scales": s["scales"]}
    if c["op"] == "dense":
        B.moe_fp8_matmul(s["x"], s["x_scales"], s["w"], s["w_scales"], s["y"], err_flag=s["err"])
    elif c["mode"] == "naive":
        B.moe_fp8_grouped_matmul_naive(s["x"], s["x_scales"], s["w"], s["w_scales"], s["y"], s["ids"],
                                       topk_weights=s["weights"], x_per_pair=c["per_pair"], err_flag=s["err"])
    else:
        B.moe_fp8_grouped_matmul(s["x"], s["x_scales"], s["w"], s["w_scales"], s["y"], s["sorted"], s["experts"],
                                 s["padded"], c["block"], topk_weights=s["weights"], x_per_pair=c["per_pair"],
                                 err_flag=s["err"])
    return s["y"]


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["M"] * c["H"]
        # the parts and the residual in; the residual, the bf16 row, the 8-bit row and its scales out
        return {"bytes": n * (2 * c["parts"] + 2 + 2 + 2 + 1) + 4 * c["M"] * _groups(c["H"]) + 2 * c["H"],
                "flops": n * (c["parts"] + 6)}
    if c["op"] == "act":
        return {"bytes": c["rows"] * (5 * c["I"] + 4 * _groups(c["I"])), "flops": 6 * c["rows"] * c["I"]}
    M, K, N = c["M"], c["K"], c["N"]
    blocks = _groups(N) * _groups(K)
    if c["op"] == "dense":
        return {"bytes": M * (K + 4 * _groups(K)) + N * K + 4 * blocks + 2 * M * N, "flops": 2 * M * N * K}
    pairs = M * c["topk"]
    rows = pairs if c["per_pair"] else M
    # each expert that a token chose, once: their expected number (each token's experts taken as drawn independently)
    p = [(e + 1) ** -c["skew"] for e in range(c["E"])]
    used = sum(1 - (1 - v / sum(p)) ** pairs for v in p)
    return {"bytes": int(rows * (K + 4 * _groups(K)) + used * (N * K + 4 * blocks) + 2 * pairs * N + 4 * pairs
                         + (4 * pairs if c["weights"] else 0)), "flops": 2 * pairs * N * K}


# ------------------------------------------------------------------ the definitions, in 64 bits

def exact(case, seed):
    c, s = case, prepare(case, seed)
    f64 = torch.float64
    if c["op"] in ("norm", "act"):
        if c["op"] == "norm":
            h = s["residual"].to(f64)
            for p in range(c["parts"]):
                h = h + s["x"][:, p].to(f64)
            v = h / torch.sqrt((h ** 2).sum(1, keepdim=True) / c["H"] + EPS) * s["weight"].to(f64)
        else:
            v = s["x"].to(f64)
            v = v[:, :c["I"]] * torch.sigmoid(v[:, :c["I"]]) * v[:, c["I"]:]
        q, scales = torch.empty_like(v), torch.empty((v.shape[0], _groups(v.shape[1])), dtype=f64, device="cuda")
        for g in range(_groups(v.shape[1])):
            part = v[:, g * GROUP:(g + 1) * GROUP]
            scales[:, g] = torch.clamp(part.abs().max(1).values / F8_MAX, min=TINY)
            q[:, g * GROUP:(g + 1) * GROUP] = part / scales[:, g:g + 1]     # the value that 8 bits round
        return {"residual": h, "normed": v, "q": q, "scales": scales} if c["op"] == "norm" else {"q": q, "scales": scales}

    def product(rows, scales, w, w_scales):
        y = torch.zeros((rows.shape[0], c["N"]), dtype=f64, device="cuda")
        n_block = torch.arange(c["N"], device="cuda") // GROUP
        for g in range(_groups(c["K"])):
            k = slice(g * GROUP, min((g + 1) * GROUP, c["K"]))
            y += (rows[:, k].to(f64) @ w[:, k].to(f64).t()) * scales[:, g:g + 1].to(f64) * w_scales[n_block, g].to(f64)
        return y

    if c["op"] == "dense":
        return product(s["x"], s["x_scales"], s["w"], s["w_scales"])
    flat = s["ids"].reshape(-1)
    y = torch.empty((flat.numel(), c["N"]), dtype=f64, device="cuda")
    for e in range(c["E"]):
        pairs = torch.nonzero(flat == e)[:, 0]
        if pairs.numel():
            rows = pairs if c["per_pair"] else pairs // c["topk"]
            x = s["x"].view(torch.uint8)[rows].view(F8)
            y[pairs] = product(x, s["x_scales"][rows], s["w"][e], s["w_scales"][e])
    if s["weights"] is not None:
        y *= s["weights"].reshape(-1, 1).to(f64)
    return y.view(c["M"], c["topk"], c["N"])
