"""GB300-native multi-LoRA Mixture-of-Experts adapter path.

Two stages of adapters, both CUDA kernels for sm_103a behind a C-ABI library
(include/moe_lora.h):
  * moe_lora_align: per active LoRA slot, count (token, top-k) pairs per
    expert, pad to block_size, prefix-sum and scatter them in order;
  * moe_lora_fused_shrink_expand: y[m,k,:] (+)= (x[m] A[l,e]^T) B[l,e]^T with
    the rank-r intermediate kept on chip.

Beside them, the 8-bit serving path of the same MoE layer: residual addition
with root-mean-square norm, the gated activation, and block-scaled products of
the base model's experts (moe_add_rms_norm_fp8, moe_silu_mul_fp8,
moe_fp8_matmul, moe_fp8_grouped_matmul and its naive form); the router
(moe_route); and the products of bf16 weights with bias, activation and
residual (moe_bf16_matmul, moe_bf16_grouped_matmul and its naive form).

The Python binding (lora_moe_gb300.binding) only marshals arguments; importing
this package loads nothing.
"""

__all__ = ["binding", "inputs"]
