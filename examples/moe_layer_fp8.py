"""One MoE layer of a multi-LoRA served model, on this library alone.

The base experts are held in 8 bits (e4m3 with a scale for each block of 128 x
128), the adapters in bf16:

    residual, x, x8 = norm(residual + the last layer's rows)
    ids, weights    = router(x)
    y13             = w13[e] x8   + adapters(x)
    act, act8       = silu(gate) * up
    y2              = weights * (w2[e] act8) + weights * adapters(act)

and the next norm sums each token's rows of y2.  A batch of a few tokens takes
the forms without an align ("naive"), a larger one the blocks of two aligns:
one of all pairs for the base experts, one for each adapter.

Run:  python examples/moe_layer_fp8.py [tokens]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from lora_moe_gb300 import binding as B  # noqa: E402

F8, BF = torch.float8_e4m3fn, torch.bfloat16


def quantize_weight(w):
    """[E, N, K] experts as 8 bits and one scale for each block of 128 x 128."""
    E, N, K = w.shape
    n, k = B.fp8_groups(N), B.fp8_groups(K)
    blocks = torch.zeros((E, n * 128, k * 128), device=w.device)
    blocks[:, :N, :K] = w.float()
    blocks = blocks.view(E, n, 128, k, 128)
    scales = (blocks.abs().amax((2, 4)) / 448).clamp_min(2.0 ** -126)
    q = (blocks / scales[:, :, None, :, None]).view(E, n * 128, k * 128)[:, :N, :K]
    return q.to(F8).contiguous(), scales


class MoELayer:
    """Weights of one layer, and its step for a batch of tokens."""

    def __init__(self, H=1024, I=512, E=16, topk=4, max_loras=3, rank=16, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(*shape, scale):
            return torch.randn(shape, generator=g, device=device) * scale

        self.H, self.I, self.E, self.topk, self.L, self.r = H, I, E, topk, max_loras, rank
        self.norm = (1 + 0.1 * normal(H, scale=1)).to(BF)
        self.router = normal(H, E, scale=H ** -0.5).to(BF)
        self.w13, self.s13 = quantize_weight(normal(E, 2 * I, H, scale=H ** -0.5))
        self.w2, self.s2 = quantize_weight(normal(E, H, I, scale=I ** -0.5))
        # adapters: one slice each for gate and up, one for w2
        self.a13 = [normal(max_loras, E, rank, H, scale=H ** -0.5).to(BF) for _ in range(2)]
        self.b13 = [normal(max_loras, E, I, rank, scale=0.3 * rank ** -0.5).to(BF) for _ in range(2)]
        self.a2 = normal(max_loras, E, rank, I, scale=I ** -0.5).to(BF)
        self.b2 = normal(max_loras, E, H, rank, scale=0.3 * rank ** -0.5).to(BF)
        self.lora_ids = torch.arange(max_loras, dtype=torch.int32, device=device)

    def route(self, x):
        """Top-k experts of each token and their renormalised probabilities."""
        p, ids = torch.softmax((x @ self.router).float(), -1).topk(self.topk, -1)
        return ids.to(torch.int32), p / p.sum(-1, keepdim=True)

    def step(self, rows, residual, lora, naive=None, err=None):
        """rows: bf16 [M, parts, H], the last layer's output rows (summed by the norm); residual: bf16 [M, H], updated
        in place; lora: int32 [M], each token's adapter or -1.  Returns the layer's rows, bf16 [M, topk, H], and what
        it computed on the way."""
        M, topk, H, I, E = rows.shape[0], self.topk, self.H, self.I, self.E
        naive = M * topk <= 32 if naive is None else naive
        new = lambda *shape, dtype=BF: torch.empty(shape, dtype=dtype, device=rows.device)  # noqa: E731
        x, x8, xs = new(M, H), new(M, H, dtype=F8), new(M, B.fp8_groups(H), dtype=torch.float32)
        B.moe_add_rms_norm_fp8(rows, self.norm, x8, xs, residual=residual, residual_out=residual, normed=x)
        ids, weights = self.route(x)

        # every id is one of this layer's experts, so every row is written (a rank that holds some of them zeroes these)
        y13, y2 = new(M, topk, 2 * I), new(M, topk, H)
        act, act8 = new(M * topk, I), new(M * topk, I, dtype=F8)
        act_s = new(M * topk, B.fp8_groups(I), dtype=torch.float32)
        if naive:
            def base(*a, **kw):
                B.moe_fp8_grouped_matmul_naive(*a, ids, err_flag=err, **kw)

            def adapters(x, a, b, y, **kw):
                B.moe_lora_fused_shrink_expand_naive(x, a, b, y, ids, lora, self.lora_ids, self.L, err_flag=err, **kw)
        else:
            block = 16 if M * topk < 16 * E else 64
            plain = B.AlignBuffers(M, topk, E, 1, 1, block)
            B.moe_align_block_size(ids, E, block, plain.sorted_token_ids, plain.expert_ids, plain.num_tokens_post_padded,
                                   workspace=plain.workspace, err_flag=err)
            per_lora = B.AlignBuffers(M, topk, E, self.L, self.L, 16)
            B.moe_lora_align(ids, lora, self.lora_ids, E, self.L, 16, per_lora.sorted_token_ids, per_lora.expert_ids,
                             per_lora.num_tokens_post_padded, workspace=per_lora.workspace, err_flag=err)

            def base(*a, **kw):
                B.moe_fp8_grouped_matmul(*a, plain.sorted_token_ids, plain.expert_ids, plain.num_tokens_post_padded,
                                         block, err_flag=err, **kw)

            def adapters(x, a, b, y, **kw):
                B.moe_lora_fused_shrink_expand_ex(x, a, b, y, per_lora.sorted_token_ids, per_lora.expert_ids,
                                                  per_lora.num_tokens_post_padded, self.lora_ids, topk, 16,
                                                  err_flag=err, **kw)
        base(x8, xs, self.w13, self.s13, y13)
        adapters(x, self.a13, self.b13, y13)
        B.moe_silu_mul_fp8(y13.view(M * topk, 2 * I), act8, act_s, act=act)
        base(act8, act_s, self.w2, self.s2, y2, topk_weights=weights, x_per_pair=True)
        adapters(act, self.a2, self.b2, y2, topk_weights=weights, x_per_pair=True)
        return y2, {"x": x, "ids": ids, "weights": weights, "act": act}


def main():
    M = int(sys.argv[1]) if len(sys.argv) > 1 else 48
    layer = MoELayer()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rows = torch.randn((M, 1, layer.H), generator=g, device="cuda").to(BF)
    residual = torch.zeros((M, layer.H), dtype=BF, device="cuda")
    lora = (torch.arange(M, device="cuda") % (layer.L + 1) - 1).to(torch.int32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(4):      # the same weights for each layer
        rows, seen = layer.step(rows, residual, lora, err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    print("4 layers of %d tokens: residual rms %.3f, last rows rms %.3f" % (
        M, residual.float().square().mean().sqrt().item(), rows.float().square().mean().sqrt().item()))


if __name__ == "__main__":
    main()
