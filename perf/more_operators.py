"""Timed cases of the router and of the bf16 products around the MoE adapters.

Three operators, in the order in which a MoE layer whose base weights are bf16 calls them:

  dense    y = act(x . w^T + bias) + residual: the router's projection (fp32 logits) and the layer's other projections;
  route    from a token's logits its top-k experts and their weights: softmax or sigmoid scores, a bias that balances
           the choice, groups of experts, renormalised weights;
  grouped  y = weight * act(x . w[e]^T + bias[e]) over the experts that the router chose for each (token, top-k) pair, on
           the blocks of the plain align ("sorted") or with one item per pair and no align ("naive").

The plain forms are elementary torch operations in 32 bits; the router's scores, which decide between neighbours, in 64.
Sizes are those of this repository's workloads (Qwen3-, gpt-oss- and Mixtral-shaped decode and prefill, the large-E
hidden size and expert count) or generic.
"""
import math

import torch

own = False

BF, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32


def listed():
    return [
        # one token's choice among 128 experts (Qwen3-shaped decode): latency alone
        {"name": "route 1x128 of 8", "op": "route", "M": 1, "E": 128, "topk": 8, "scoring": "softmax", "f32": True,
         "bias": False, "renormalize": True, "scale": 1.0, "groups": 1, "topk_groups": 1, "best": 1, "masked": 0},
        # a decode batch, bf16 logits with many ties (gpt-oss-shaped)
        {"name": "route 64x128 of 4", "op": "route", "M": 64, "E": 128, "topk": 4, "scoring": "softmax", "f32": False,
         "bias": False, "renormalize": True, "scale": 1.0, "groups": 1, "topk_groups": 1, "best": 1, "masked": 0},
        # a large prefill with balancing bias and groups (the large-E expert count)
        {"name": "route 16384x256 of 8 in groups", "op": "route", "M": 16384, "E": 256, "topk": 8, "scoring": "sigmoid",
         "f32": True, "bias": True, "renormalize": True, "scale": 2.5, "groups": 8, "topk_groups": 4, "best": 2,
         "masked": 0},
        # the router's projection of one token (Qwen3-shaped)
        {"name": "dense 1x2048x128 to f32", "op": "dense", "M": 1, "K": 2048, "N": 128, "f32": True, "bias": "",
         "act": "none", "residual": False},
        # a decode batch's output projection of 64 heads of 64, with bias and residual (gpt-oss-shaped)
        {"name": "dense 64x4096x2880 bias residual", "op": "dense", "M": 64, "K": 4096, "N": 2880, "f32": False,
         "bias": "bf16", "act": "none", "residual": True},
        # the router's projection in a prefill (the large-E hidden size and expert count): x is read once
        {"name": "dense 4096x7168x256 to f32", "op": "dense", "M": 4096, "K": 7168, "N": 256, "f32": True, "bias": "f32",
         "act": "none", "residual": False},
        # prefill through an up projection with its activation: bound by the tensor cores
        {"name": "dense 8192x4096x14336 silu", "op": "dense", "M": 8192, "K": 4096, "N": 14336, "f32": False, "bias": "",
         "act": "silu", "residual": False},
        # one token and its eight experts, no align (Qwen3-shaped gate and up projections)
        {"name": "naive 1 of 128x2048x1536", "op": "grouped", "mode": "naive", "M": 1, "topk": 8, "E": 128, "K": 2048,
         "N": 1536, "block": 16, "per_pair": False, "weights": False, "skew": 1.1, "bias": "", "act": "none"},
        # a decode batch with a skewed router (Qwen3-shaped gate and up projections)
        {"name": "sorted 16 of 128x2048x1536", "op": "grouped", "mode": "sorted", "M": 16, "topk": 8, "E": 128,
         "K": 2048, "N": 1536, "block": 16, "per_pair": False, "weights": False, "skew": 1.1, "bias": "", "act": "none"},
        # a decode batch's down projection: a row for each pair, an expert's bias, the router's weight (gpt-oss-shaped)
        {"name": "sorted 64 of 128x2880x2880 bias", "op": "grouped", "mode": "sorted", "M": 64, "topk": 4, "E": 128,
         "K": 2880, "N": 2880, "block": 16, "per_pair": True, "weights": True, "skew": 0.0, "bias": "bf16", "act": "none"},
        # a batch between decode and prefill, 64 pairs an expert (Qwen3-shaped gate and up projections)
        {"name": "sorted 1024 of 128x2048x1536", "op": "grouped", "mode": "sorted", "M": 1024, "topk": 8, "E": 128,
         "K": 2048, "N": 1536, "block": 64, "per_pair": False, "weights": False, "skew": 0.0, "bias": "", "act": "none"},
        # prefill (Mixtral-shaped gate and up projections): bound by the tensor cores
        {"name": "sorted 8192 of 8x4096x28672", "op": "grouped", "mode": "sorted", "M": 8192, "topk": 2, "E": 8,
         "K": 4096, "N": 28672, "block": 128, "per_pair": False, "weights": False, "skew": 0.0, "bias": "", "act": "none"},
    ]


ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def draw(rng):
    def log(lo, hi, whole=0.0):
        """A size between lo and hi, even in its logarithm; with probability `whole` a multiple of 16."""
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return max(lo, v // 16 * 16) if rng.random() < whole else v

    op = rng.choice(("route", "route", "dense", "dense", "dense", "grouped", "grouped", "grouped"))
    if op == "route":
        E = rng.choice((8, 16, 60, 64, 128, 160, 256, 384, 512, rng.randint(2, 1024)))
        groups = rng.choice([g for g in (1, 1, 2, 4, 8, 16) if E % g == 0 and E // g >= 2])
        topk_groups = rng.randint(1, groups)
        return {"op": op, "M": log(1, 16384), "E": E,
                "topk": min(rng.choice((1, 2, 4, 6, 8, 10)), topk_groups * (E // groups)),
                "scoring": rng.choice(("softmax", "sigmoid")), "f32": rng.random() < 0.6, "bias": rng.random() < 0.5,
                "renormalize": rng.random() < 0.7, "scale": rng.choice((1.0, 2.5)), "groups": groups,
                "topk_groups": topk_groups, "best": rng.choice((1, 2)), "masked": rng.choice((0, 0, 0, 0.1))}
    bias, act = rng.choice(("", "bf16", "f32")), rng.choice(("none", "none") + ACTS)
    K = log(64, 8192, 0.8)
    if op == "dense":
        f32 = rng.random() < 0.3
        N = log(8, 1024, 0.5) if f32 else log(64, 16384, 0.8)     # fp32: logits
        M = max(1, min(log(1, 8192), 8192 * 4096 * 14336 // (K * N)))
        return {"op": op, "M": M, "K": K, "N": N, "f32": f32, "bias": bias, "act": "none" if f32 else act,
                "residual": rng.random() < 0.4}
    mode = rng.choice(("naive", "sorted", "sorted"))
    N = log(64, 8192, 0.8)
    E, topk = rng.choice((8, 16, 60, 128, 256)), rng.choice((1, 2, 4, 8))
    M = log(1, 16) if mode == "naive" else log(1, 8192)
    # no more weight, and no more work with every expert's rows padded to M, than the largest listed case
    E = max(8, min(E, 8 * 4096 * 28672 // (K * N)))
    M = max(1, min(M, 4 * 8 * 2048 * 4096 * 28672 // (E * K * N), 16384 // topk))
    return {"op": op, "mode": mode, "M": M, "topk": topk, "E": E, "K": K, "N": N,
            "block": 16 if mode == "naive" else rng.choice((16, 32, 64, 128)), "per_pair": rng.random() < 0.5,
            "weights": rng.random() < 0.5, "skew": rng.choice((0.0, 1.1)), "bias": bias, "act": act}


# ------------------------------------------------------------------ inputs

def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _bf_rows(v):
    """v in bf16, its rows padded to whole 16 bytes."""
    rows, k = v.shape
    t = torch.zeros((rows, -(-k // 8) * 8), dtype=BF, device="cuda")[:, :k]
    return t.copy_(v)


def _weights(count, n, k, gen):
    """Random matrices of unit gain, whose rows differ in size (as a trained weight's do)."""
    w = torch.zeros((count, n, -(-k // 8) * 8), dtype=BF, device="cuda")[:, :, :k]
    for e in range(count):
        w[e] = _randn(gen, n, k) * torch.exp(0.3 * _randn(gen, n, 1)) / math.sqrt(k)
    return w


def _activations(rows, k, gen):
    """Normal rows with a few large channels."""
    return _bf_rows(_randn(gen, rows, k) * torch.exp(0.5 * _randn(gen, 1, k)))


def _bias(kind, gen, *shape):
    return (0.2 * _randn(gen, *shape)).to(BF if kind == "bf16" else F32) if kind else None


def _routing(c, gen):
    """Distinct experts for each token, uniform or with a Zipf-like skew, and router weights that sum to one."""
    M, E, topk = c["M"], c["E"], c["topk"]
    p = torch.arange(1, E + 1, dtype=F32, device="cuda") ** -c["skew"]
    p = p[torch.randperm(E, generator=gen, device="cuda")]
    ids = torch.multinomial(p.expand(M, E), topk, generator=gen).to(I32)
    return ids, torch.softmax(_randn(gen, M, topk), -1)


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
    sorted_ids = torch.full((cap,), P, dtype=I32, device="cuda")
    sorted_ids[first[flat[order]] * block + rank] = order.to(I32)
    expert_ids = torch.zeros(-(-cap // block), dtype=I32, device="cuda")
    n = int(blocks.sum())
    expert_ids[:n] = torch.repeat_interleave(torch.arange(E, device="cuda"), blocks).to(I32)
    return sorted_ids, expert_ids, (blocks.sum() * block).to(I32).reshape(1), int(counts.max())


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "route":
        M, E = c["M"], c["E"]
        # logits spread over a few units, some experts liked by most tokens
        logits = 1.5 * _randn(gen, M, E) + 0.7 * _randn(gen, 1, E)
        if c["masked"]:     # experts that are switched off
            logits[:, torch.rand(E, generator=gen, device="cuda") < c["masked"]] = -math.inf
        s["logits"] = logits.to(F32 if c["f32"] else BF)
        s["bias"] = 0.1 * _randn(gen, E) if c["bias"] else None
        s["ids"] = torch.empty((M, c["topk"]), dtype=I32, device="cuda")
        s["weights"] = torch.empty((M, c["topk"]), dtype=F32, device="cuda")
        return s
    M, K, N = c["M"], c["K"], c["N"]
    grouped = c["op"] == "grouped"
    s["x"] = _activations(M * c["topk"] if grouped and c["per_pair"] else M, K, gen)
    w = _weights(c["E"] if grouped else 1, N, K, gen)
    s["w"] = w if grouped else w[0]
    s["bias"] = _bias(c["bias"], gen, c["E"], N) if grouped else _bias(c["bias"], gen, N)
    s["err"] = torch.zeros(1, dtype=I32, device="cuda")
    if grouped:
        s["ids"], weights = _routing(c, gen)
        s["weights"] = weights if c["weights"] else None
        s["sorted"], s["experts"], s["padded"], s["most"] = _align(s["ids"], c["E"], c["block"])
        s["y"] = torch.empty((M, c["topk"], N), dtype=BF, device="cuda")
    else:
        kind = F32 if c["f32"] else BF
        s["residual"] = (2 * _randn(gen, M, N)).to(kind) if c["residual"] else None
        s["y"] = torch.empty((M, N), dtype=kind, device="cuda")
    return s


# ------------------------------------------------------------------ the plain forms

def _plain_act(v, act):
    if act == "relu":
        return v.clamp_min(0)
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _plain_route(s):
    """Scores in 64 bits: they decide between neighbours."""
    c, x = s["case"], s["logits"].double()
    M, E = x.shape
    if c["scoring"] == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-x))
    choice = score if s["bias"] is None else score + s["bias"].double()
    choice = choice.masked_fill(x == -math.inf, -math.inf)
    if c["groups"] > 1:
        best = choice.view(M, c["groups"], -1).sort(dim=-1, descending=True).values[:, :, :c["best"]]
        # a group of one candidate counts that one, and one of none is last
        total = best.masked_fill(best == -math.inf, 0).sum(-1).masked_fill(best[:, :, 0] == -math.inf, -math.inf)
        kept = total.sort(dim=-1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        open_ = torch.zeros((M, c["groups"]), dtype=torch.bool, device="cuda").scatter_(1, kept, True)
        choice = choice.masked_fill(~open_.repeat_interleave(E // c["groups"], 1), -math.inf)
    top, ids = (t[:, :c["topk"]] for t in choice.sort(dim=-1, descending=True, stable=True))
    weights = score.gather(1, ids).masked_fill(top == -math.inf, 0)
    if c["renormalize"]:
        total = weights.sum(1, keepdim=True)
        weights = torch.where(total > 0, weights / total, weights)
    return {"ids": ids.to(I32), "weights": (weights * c["scale"]).float()}


def _plain(s):
    c = s["case"]
    if c["op"] == "route":
        return _plain_route(s)
    x = s["x"].float()
    if c["op"] == "dense":
        y = x @ s["w"].float().t()
        y = _plain_act(y if s["bias"] is None else y + s["bias"].float(), c["act"])
        return (y if s["residual"] is None else y + s["residual"].float()).to(s["y"].dtype)
    flat = s["ids"].reshape(-1).long()
    x = x if c["per_pair"] else x.repeat_interleave(c["topk"], 0)
    if flat.numel() < c["E"]:
        # few pairs: each with its expert's weight
        y = torch.bmm(s["w"][flat].float(), x[:, :, None])[:, :, 0]
    else:
        # every expert's rows side by side, padded to the most that one expert has: one batched product
        rank = torch.nn.functional.one_hot(flat, c["E"]).cumsum(0).gather(1, flat[:, None])[:, 0] - 1
        rows = torch.zeros((c["E"], s["most"], c["K"]), device="cuda")
        rows[flat, rank] = x
        y = torch.bmm(rows, s["w"].float().transpose(1, 2))[flat, rank]
    y = _plain_act(y if s["bias"] is None else y + s["bias"].float()[flat], c["act"])
    if s["weights"] is not None:
        y = y * s["weights"].reshape(-1, 1)
    return y.to(BF).view(c["M"], c["topk"], c["N"])


def run(state):
    if not own:
        return _plain(state)
    from lora_moe_gb300 import binding as B
    s, c = state, state["case"]
    if c["op"] == "route":
        B.moe_route(s["logits"], s["ids"], s["weights"], bias=s["bias"],
                    scoring=B.ROUTE_SOFTMAX if c["scoring"] == "softmax" else B.ROUTE_SIGMOID,
                    renormalize=c["renormalize"], scale=c["scale"], num_groups=c["groups"],
                    topk_groups=c["topk_groups"], group_best=c["best"])
        return {"ids": s["ids"], "weights": s["weights"]}
    act = getattr(B, "ACT_" + c["act"].upper())
    if c["op"] == "dense":
        B.moe_bf16_matmul(s["x"], s["w"], s["y"], bias=s["bias"], residual=s["residual"], activation=act,
                          err_flag=s["err"])
    elif c["mode"] == "naive":
        B.moe_bf16_grouped_matmul_naive(s["x"], s["w"], s["y"], s["ids"], bias=s["bias"], activation=act,
                                        topk_weights=s["weights"], x_per_pair=c["per_pair"], err_flag=s["err"])
    else:
        B.moe_bf16_grouped_matmul(s["x"], s["w"], s["y"], s["sorted"], s["experts"], s["padded"], c["block"],
                                  bias=s["bias"], activation=act, topk_weights=s["weights"],
                                  x_per_pair=c["per_pair"], err_flag=s["err"])
    return s["y"]


def work(case):
    c = case
    if c["op"] == "route":
        # the logits in, ids and weights out; an exponential and a few comparisons a logit
        return {"bytes": c["M"] * (c["E"] * (4 if c["f32"] else 2) + 8 * c["topk"]) + (4 * c["E"] if c["bias"] else 0),
                "flops": c["M"] * c["E"] * (4 + c["topk"])}
    M, K, N = c["M"], c["K"], c["N"]
    bias = {"": 0, "bf16": 2 * N, "f32": 4 * N}[c["bias"]]
    if c["op"] == "dense":
        out = (4 if c["f32"] else 2) * M * N
        return {"bytes": 2 * (M * K + N * K) + bias + out * (2 if c["residual"] else 1), "flops": 2 * M * N * K}
    pairs = M * c["topk"]
    rows = pairs if c["per_pair"] else M
    # each expert that a token chose, once: their expected number (each token's experts taken as drawn independently)
    p = [(e + 1) ** -c["skew"] for e in range(c["E"])]
    used = sum(1 - (1 - v / sum(p)) ** pairs for v in p)
    return {"bytes": int(2 * rows * K + used * (2 * N * K + bias) + 2 * pairs * N + 4 * pairs
                         + (4 * pairs if c["weights"] else 0)), "flops": 2 * pairs * N * K}


# ------------------------------------------------------------------ the definitions, in 64 bits

def _exact_act(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "gelu_tanh":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "route":
        x = s["logits"].to(F64)
        score = torch.softmax(x, 1) if c["scoring"] == "softmax" else torch.sigmoid(x)
        choice = (score + (0 if s["bias"] is None else s["bias"].to(F64))).where(x > -math.inf, x)
        if c["groups"] > 1:
            size = c["E"] // c["groups"]
            worth = []
            for g in range(c["groups"]):
                top = choice[:, g * size:(g + 1) * size].topk(c["best"], 1).values
                worth.append(torch.where(top[:, 0] > -math.inf, top.clamp_min(-1e300).where(top > -math.inf, 0 * score[:, :1]).sum(1), top[:, 0]))
            worth = torch.stack(worth, 1)
            for g in range(c["groups"]):
                before = (worth > worth[:, g:g + 1]).sum(1) + (worth[:, :g] == worth[:, g:g + 1]).sum(1)
                choice[:, g * size:(g + 1) * size].masked_fill_((before >= c["topk_groups"])[:, None], -math.inf)
        weights = torch.empty((c["M"], c["topk"]), dtype=F64, device="cuda")
        for k in range(c["topk"]):
            top = choice.amax(1, keepdim=True)
            # the first expert that has it (those taken, and those that are no candidates, weigh nothing)
            at = (choice == top).to(torch.uint8).argmax(1, keepdim=True)
            weights[:, k] = torch.where(top > -math.inf, score.gather(1, at), 0.0)[:, 0]
            choice.scatter_(1, at, -math.inf)
        if c["renormalize"]:
            weights /= weights.sum(1, keepdim=True).where(weights.sum(1, keepdim=True) > 0, torch.ones_like(weights[:, :1]))
        return {"ids": None, "weights": weights * c["scale"]}
    if c["op"] == "dense":
        y = torch.empty((c["M"], c["N"]), dtype=F64, device="cuda")
        w = s["w"].to(F64).t()
        for r in range(0, c["M"], 2048):
            y[r:r + 2048] = s["x"][r:r + 2048].to(F64) @ w
        y = _exact_act(y if s["bias"] is None else y + s["bias"].to(F64), c["act"])
        return y if s["residual"] is None else y + s["residual"].to(F64)
    flat = s["ids"].reshape(-1)
    y = torch.empty((flat.numel(), c["N"]), dtype=F64, device="cuda")
    for e in range(c["E"]):
        pairs = torch.nonzero(flat == e)[:, 0]
        if pairs.numel():
            rows = pairs if c["per_pair"] else pairs // c["topk"]
            v = s["x"][rows].to(F64) @ s["w"][e].to(F64).t()
            y[pairs] = _exact_act(v if s["bias"] is None else v + s["bias"][e].to(F64), c["act"])
    if s["weights"] is not None:
        y *= s["weights"].reshape(-1, 1).to(F64)
    return y.view(c["M"], c["topk"], c["N"])
